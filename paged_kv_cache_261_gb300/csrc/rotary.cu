// Rotary positions of a step's queries and keys, and, fused with them, the scatter of the
// rotated keys and of the values into a paged cache.
//
// The rotation is not on the pages; the slot arithmetic is that of "PagedAttention实现" write_kv
// and "04 - Paged Attention 实现进度" B.2. Pair j of a head's first rotary_dim channels, either
// (x[j], x[j + rotary_dim / 2]) or (x[2 j], x[2 j + 1]), is turned by the angle a = position *
// inv_freq[j]:
//   (x1, x2) -> factor * (x1 cos a - x2 sin a, x2 cos a + x1 sin a)
// in float32, rounded once to the type; the other channels are copied.
//
// Angles of far positions: inv_freq / 2 pi, in 64 bits, becomes a fixed-point number of 2^-64
// turns, and its product with the position, modulo 2^64, the angle's fraction of a turn: whole
// turns drop out exactly, whatever the position. The fraction, less its nearest quarter, is
// short enough for float32 (an error of 2^-28 turns at most), and sincospif takes it.
// The angle is off by position * inv_freq * 2^-52 and that, nothing else.
//
// A CTA takes one or two tokens: its threads first make the tokens' cosines and sines, in shared
// memory, then each takes units of 16 channels, the 8 pairs of which lie in one thread for both
// kinds of pairs. The first units are loaded before the angles are made. What bounds it is HBM:
// every row is read and written once.
#include "common.cuh"
#include "f32x2.cuh"
#include "kernels_step.h"

#include <algorithm>

namespace pa {
namespace {

constexpr int kThreads = 128;
constexpr int kUnits = 2;                        // of a thread, in flight together
constexpr int kMaxTokens = 2;                    // of a CTA
constexpr int64_t kManyTokens = 1200;            // from here on a CTA takes kMaxTokens

// inv_freq radians as a number of 2^-64 turns, modulo one turn.
__device__ __forceinline__ uint64_t turn_step(double inv_freq) {
    double turns = inv_freq * 0.15915494309189533577;      // 1 / (2 pi)
    turns -= floor(turns);
    return __double2ull_rn(turns * 18446744073709551616.0);
}
// Cosine and sine of position * step.
__device__ __forceinline__ float2 cos_sin(uint64_t step, int position) {
    const uint32_t at = (uint32_t)((step * (uint64_t)(int64_t)position) >> 32);
    const uint32_t quarter = (at + 0x20000000u) >> 30;
    float s, c;
    sincospif((float)(int)(at - (quarter << 30)) * 0x1p-31f, &s, &c);        // half turns, at most 1/4
    if (quarter & 1) {
        const float t = c;
        c = -s;
        s = t;
    }
    return quarter & 2 ? make_float2(-c, -s) : make_float2(c, s);
}

// Eight channels as loaded.
template <typename T> struct Run8 {
    uint4 raw[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T *src) {
#pragma unroll
        for (int u = 0; u < (int)sizeof(T) / 2; ++u) raw[u] = reinterpret_cast<const uint4 *>(src)[u];
    }
    __device__ __forceinline__ void store(T *dst) const {
#pragma unroll
        for (int u = 0; u < (int)sizeof(T) / 2; ++u) reinterpret_cast<uint4 *>(dst)[u] = raw[u];
    }
    __device__ __forceinline__ void values(float *x) const {
#pragma unroll
        for (int u = 0; u < (int)sizeof(T) / 2; ++u) Vec16<T>::unpack(raw[u], x + u * Vec16<T>::N);
    }
    __device__ __forceinline__ void round(const float *x) {
        T *v = reinterpret_cast<T *>(raw);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = Elem<T>::from_f(x[i]);
    }
};

template <typename T, bool kInterleaved>
__global__ __launch_bounds__(kThreads) void rotary_kernel(const RotaryParams p, int tokens) {
    extern __shared__ __align__(16) float turn[];          // [tokens][2][half] cosines, sines; then the steps [half]
    // launched as a dependent of the kernel before; a kernel launched after this one may start
    // its set-up once everything before this one has finished
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int half = p.rotary_dim / 2, D = p.head_dim, parts = D / 16;
    const int64_t t0 = (int64_t)blockIdx.x * tokens;
    const int n = (int)min((int64_t)tokens, p.num_tokens - t0);
    const int H = p.num_heads, Hk = p.num_kv_heads, heads = H + Hk * (p.slots ? 2 : 1);
    // this thread's part of a row's channels, and its place among the CTA's rows
    const int part = threadIdx.x % parts, rows = kThreads / parts;
    const bool turned = part * 8 < half;
    const int a = kInterleaved || !turned ? part * 16 : part * 8, b = kInterleaved || !turned ? a + 8 : a + half;
    const int h0 = threadIdx.x / parts;

    struct Unit {
        Run8<T> x[2];
        T *dst;                                            // null: none
        bool turns;
    };
    // head h of the queries, keys and values in turn, of token t; cache: its row there, -1: none
    auto load = [&](Unit &u, int h, int64_t t, int64_t cache) {
        u.dst = nullptr;
        if (h >= heads) return;
        const T *src;
        if (h < H) {
            src = static_cast<const T *>(p.q) + t * p.q_stride + h * D;
            u.dst = static_cast<T *>(p.q_out) + t * p.q_out_stride + h * D;
            u.turns = turned;
        } else {
            const bool is_v = h >= H + Hk;
            const int at = (h - H - (is_v ? Hk : 0)) * D;
            if (cache < 0) return;
            src = (is_v ? static_cast<const T *>(p.v) + t * p.v_stride : static_cast<const T *>(p.k) + t * p.k_stride) + at;
            u.dst = static_cast<T *>(is_v ? p.v_out : p.k_out) + cache + at;
            u.turns = turned && !is_v;
        }
        u.x[0].load(src + a);
        u.x[1].load(src + b);
    };
    auto finish = [&](Unit &u, const float *cs) {
        if (!u.dst) return;
        if (u.turns) {
            float x[16], y[16];
            u.x[0].values(x);
            u.x[1].values(x + 8);
            float c[8], s[8];
#pragma unroll
            for (int j = 0; j < 8; j += 4) {
                *reinterpret_cast<float4 *>(c + j) = *reinterpret_cast<const float4 *>(cs + j);
                *reinterpret_cast<float4 *>(s + j) = *reinterpret_cast<const float4 *>(cs + half + j);
            }
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                // channels of the pairs j and j + 1: (one, two) of each
                const int i1 = kInterleaved ? 2 * j : j, i2 = kInterleaved ? i1 + 1 : 8 + j, next = kInterleaved ? 2 : 1;
                const float2 one = make_float2(x[i1], x[i1 + next]), two = make_float2(x[i2], x[i2 + next]);
                const float2 cj = make_float2(c[j], c[j + 1]), sj = make_float2(s[j], s[j + 1]);
                const float2 y1 = fma2(one, cj, mul2(two, make_float2(-sj.x, -sj.y))), y2 = fma2(two, cj, mul2(one, sj));
                y[i1] = y1.x;
                y[i1 + next] = y1.y;
                y[i2] = y2.x;
                y[i2 + next] = y2.y;
            }
            u.x[0].round(y);
            u.x[1].round(y + 8);
        }
        u.x[0].store(u.dst + a);
        u.x[1].store(u.dst + b);
    };
    // where a token's keys and values go, in elements from the outputs' start
    auto cache_row = [&](int64_t t) {
        if (!p.slots) return t * p.k_out_stride;
        const int64_t slot = p.slots[t];
        if (slot >= 0 && slot < p.num_slots) return slot * Hk * D;
        if (slot != -1 && threadIdx.x == 0) raise_error(p.err, PA_DEVERR_SLOT);
        return (int64_t)-1;
    };
    const bool works = h0 < rows;                          // threads that a row's parts do not divide are idle
    int64_t cache = cache_row(t0);
    Unit u[kUnits];
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
        u[k].dst = nullptr;
        if (works) load(u[k], h0 + k * rows, t0, cache);   // on their way while the angles are made
    }

    uint64_t *steps = reinterpret_cast<uint64_t *>(turn + 2 * tokens * half);
    for (int j = threadIdx.x; j < half; j += kThreads) steps[j] = turn_step(p.inv_freq[j]);
    __syncthreads();
    for (int e = threadIdx.x; e < n * half; e += kThreads) {
        const int i = e / half, j = e - i * half;
        const float2 cs = cos_sin(steps[j], p.positions[t0 + i]);
        turn[2 * i * half + j] = cs.x * p.factor;
        turn[(2 * i + 1) * half + j] = cs.y * p.factor;
    }
    __syncthreads();
    if (!works) return;

    for (int i = 0; i < n; ++i) {
        const float *cs = turn + 2 * i * half + part * 8;
        const int64_t t = t0 + i, next = i + 1 < n ? cache_row(t + 1) : -1;
        for (int h = h0; h < heads; h += kUnits * rows) {
#pragma unroll
            for (int k = 0; k < kUnits; ++k) finish(u[k], cs);
            // the next ones of this token, or the first of the next
            const bool same = h + kUnits * rows < heads;
#pragma unroll
            for (int k = 0; k < kUnits; ++k) {
                if (same) load(u[k], h + (kUnits + k) * rows, t, cache);
                else if (i + 1 < n) load(u[k], h0 + k * rows, t + 1, next);
            }
        }
        cache = next;
    }
}

template <typename T>
int launch_t(const RotaryParams &p, cudaStream_t stream) {
    const int tokens = p.num_tokens >= kManyTokens ? kMaxTokens : 1;
    const int64_t grid = (p.num_tokens + tokens - 1) / tokens;
    return launch_pdl(p.interleaved ? rotary_kernel<T, true> : rotary_kernel<T, false>, dim3((unsigned)grid),
                      dim3(kThreads), (size_t)(tokens + 1) * p.rotary_dim * sizeof(float), stream, p, tokens);
}

}  // namespace

int launch_rotary(const RotaryParams &p, int dtype, cudaStream_t stream) {
    switch (dtype) {
    case PA_DTYPE_F32: return launch_t<float>(p, stream);
    case PA_DTYPE_F16: return launch_t<__half>(p, stream);
    case PA_DTYPE_BF16: return launch_t<__nv_bfloat16>(p, stream);
    default: return -2;
    }
}

}  // namespace pa
