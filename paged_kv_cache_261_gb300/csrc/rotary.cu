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
// The angle is off by that, by position * inv_freq * 2^-52 (the quotient's two roundings) and by position * 2^-65 turns
// (the fixed point's, 2^-34 turns at most).
//
// A CTA takes a few tokens: its threads first make the tokens' cosines and sines, in shared
// memory, then take units of 16 channels, the 8 pairs of which lie in one thread for both kinds
// of pairs. The first units are loaded before the angles are made.
//
// What bounds it (one GB300, inputs and outputs not in L2): HBM, every row being read and written
// once. 8192 tokens of 32 + 8 + 8 heads, 201 MB, 32.4 us, 6.2 TB/s; 4096 of 128 + 8 + 8, 302 MB, 47.9;
// 2047 of 64 + 8, 75 MB, 14.7. Three units a thread in flight: with two 33.4 us (the 8192 tokens). With all of a
// CTA's rows copied asynchronously into shared memory, so more on its way: 46.6. The streaming hints gain
// 2 to 3 %, on the loads or the stores alone nothing.
#include "common.cuh"
#include "f32x2.cuh"
#include "kernels_step.h"

#include <algorithm>

namespace pa {
namespace {

constexpr int kThreads = 128;
constexpr int kUnits = 3;                        // of a thread, in flight together
constexpr int kTurns = 4;                        // units of a thread that a CTA's tokens are chosen for
constexpr int kMaxTokens = 8;                    // of a CTA
// Up to here a CTA takes one token (8 + 1 + 1 heads of 64 channels, us with one and 6: 200 tokens 2.9, 3.4,
// 1100 3.7, 3.5, 2000 5.8, 3.7).
constexpr int64_t kManyTokens = 1200;

// inv_freq radians as a number of 2^-64 turns, modulo one turn. Of a negative one the magnitude is taken and the
// number negated: the rest of a small one less a whole turn would keep its bits from 2^-54 turns on alone.
__device__ __forceinline__ uint64_t turn_step(double inv_freq) {
    double turns = fabs(inv_freq) * 0.15915494309189533577;      // 1 / (2 pi)
    turns -= floor(turns);
    const uint64_t step = __double2ull_rn(turns * 18446744073709551616.0);
    return inv_freq < 0.0 ? 0 - step : step;
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
        for (int u = 0; u < (int)sizeof(T) / 2; ++u) raw[u] = __ldcs(reinterpret_cast<const uint4 *>(src) + u);
    }
    __device__ __forceinline__ void store(T *dst) const {
#pragma unroll
        for (int u = 0; u < (int)sizeof(T) / 2; ++u) __stcs(reinterpret_cast<uint4 *>(dst) + u, raw[u]);
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
    // [tokens][2][half] cosines and sines, and the tokens' rows in the cache [tokens]
    extern __shared__ __align__(16) float turn[];
    // launched as a dependent of the kernel before; a kernel launched after this one may start
    // its set-up once everything before this one has finished
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int half = p.rotary_dim / 2, D = p.head_dim, parts = D / 16;
    int64_t *cache = reinterpret_cast<int64_t *>(turn + 2 * tokens * half);
    const int64_t t0 = (int64_t)blockIdx.x * tokens;
    const int n = (int)min((int64_t)tokens, p.num_tokens - t0);
    const int H = p.num_heads, Hk = p.num_kv_heads, heads = H + Hk * (p.slots ? 2 : 1);
    // this thread's part of a row's channels, and its place among the CTA's rows
    const int part = threadIdx.x % parts, rows = kThreads / parts;
    const bool turned = part * 8 < half;
    const int a = kInterleaved || !turned ? part * 16 : part * 8, b = kInterleaved || !turned ? a + 8 : a + half;

    struct Unit {
        Run8<T> x[2];
        int i, h;                                          // token, head of the queries, keys and values in turn
    };
    // the next row of this thread
    int i = 0, h = threadIdx.x / parts;
    if (h >= rows) i = n;                                  // threads that a row's parts do not divide are idle
    auto load = [&](Unit &u) {
        while (h >= heads) {
            h -= heads;
            ++i;
        }
        u.i = i;
        u.h = h;
        h += rows;
        if (u.i >= n) return;
        const int64_t t = t0 + u.i;
        const T *src = u.h < H        ? static_cast<const T *>(p.q) + t * p.q_stride + u.h * D
                       : u.h < H + Hk ? static_cast<const T *>(p.k) + t * p.k_stride + (u.h - H) * D
                                      : static_cast<const T *>(p.v) + t * p.v_stride + (u.h - H - Hk) * D;
        u.x[0].load(src + a);
        u.x[1].load(src + b);
    };
    Unit u[kUnits];
#pragma unroll
    for (int k = 0; k < kUnits; ++k) load(u[k]);           // on their way while the angles are made

    // where a token's keys and values go, in elements from the outputs' start; -1: nowhere
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const int64_t t = t0 + i;
        int64_t row = t * p.k_out_stride;
        if (p.slots) {
            const int64_t slot = p.slots[t];
            const bool good = slot >= 0 && slot < p.num_slots;
            if (!good && slot != -1) raise_error(p.err, PA_DEVERR_SLOT);
            row = good ? slot * Hk * D : -1;
        }
        cache[i] = row;
    }
    // a thread has a frequency and every groups-th token
    const int groups = max(1, kThreads / half);
    for (int e = threadIdx.x; e < groups * half; e += kThreads) {
        const int g = e / half, j = e - g * half;
        const uint64_t step = turn_step(p.inv_freq[j]);
        for (int t = g; t < n; t += groups) {
            const float2 cs = cos_sin(step, p.positions[t0 + t]);
            turn[2 * t * half + j] = cs.x * p.factor;
            turn[(2 * t + 1) * half + j] = cs.y * p.factor;
        }
    }
    __syncthreads();

    auto finish = [&](Unit &u) {
        if (u.i >= n) return;
        const bool is_v = u.h >= H + Hk;
        T *dst;
        if (u.h < H) {
            dst = static_cast<T *>(p.q_out) + (t0 + u.i) * p.q_out_stride + u.h * D;
        } else {
            if (cache[u.i] < 0) return;
            dst = static_cast<T *>(is_v ? p.v_out : p.k_out) + cache[u.i] + (u.h - H - (is_v ? Hk : 0)) * D;
        }
        if (turned && !is_v) {
            const float *cs = turn + 2 * u.i * half + part * 8;
            float x[16], y[16], c[8], s[8];
            u.x[0].values(x);
            u.x[1].values(x + 8);
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
        u.x[0].store(dst + a);
        u.x[1].store(dst + b);
    };
    while (u[0].i < n) {
#pragma unroll
        for (int k = 0; k < kUnits; ++k) finish(u[k]);
#pragma unroll
        for (int k = 0; k < kUnits; ++k) load(u[k]);
    }
}

template <typename T>
int launch_t(const RotaryParams &p, cudaStream_t stream) {
    const int rows = kThreads / (p.head_dim / 16), heads = p.num_heads + p.num_kv_heads * (p.slots ? 2 : 1);
    const int tokens = p.num_tokens < kManyTokens ? 1 : std::max(1, std::min(kMaxTokens, kTurns * rows / heads));
    const size_t smem = tokens * (p.rotary_dim * sizeof(float) + sizeof(int64_t));
    return launch_pdl(p.interleaved ? rotary_kernel<T, true> : rotary_kernel<T, false>,
                      dim3((unsigned)((p.num_tokens + tokens - 1) / tokens)), dim3(kThreads), smem, stream, p, tokens);
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
