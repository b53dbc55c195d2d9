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
// A CTA takes a few tokens: its threads first make the tokens' cosines and sines, in shared
// memory, then each takes units of 16 channels, the 8 pairs of which lie in one thread for
// both kinds of pairs. What bounds it is HBM: every row is read and written once.
#include "common.cuh"
#include "kernels_step.h"

#include <algorithm>

namespace pa {
namespace {

constexpr int kThreads = 256;

// Cosine and sine of position * inv_freq.
__device__ __forceinline__ float2 cos_sin(double inv_freq, int position) {
    double turns = inv_freq * 0.15915494309189533577;      // 1 / (2 pi)
    turns -= floor(turns);
    const uint64_t step = __double2ull_rn(turns * 18446744073709551616.0);   // of 2^-64 turns
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

template <typename T> __device__ __forceinline__ void load8(const T *src, float *x) {
    constexpr int N = Vec16<T>::N;
#pragma unroll
    for (int u = 0; u < 8 / N; ++u) Vec16<T>::unpack(reinterpret_cast<const uint4 *>(src)[u], x + u * N);
}
template <typename T> __device__ __forceinline__ void store8(T *dst, const float *x) {
    alignas(16) T v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = Elem<T>::from_f(x[i]);
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4 *>(dst)[i] = reinterpret_cast<const uint4 *>(v)[i];
}

template <typename T, bool kInterleaved>
__global__ __launch_bounds__(kThreads) void rotary_kernel(const RotaryParams p, int tokens) {
    extern __shared__ float2 turn[];                       // [tokens][rotary_dim / 2]
    // launched as a dependent of the kernel before; a kernel launched after this one may start
    // its set-up once everything before this one has finished
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int half = p.rotary_dim / 2, D = p.head_dim;
    const int64_t t0 = (int64_t)blockIdx.x * tokens;
    const int n = (int)min((int64_t)tokens, p.num_tokens - t0);
    for (int i = threadIdx.x; i < n * half; i += kThreads) {
        const float2 cs = cos_sin(p.inv_freq[i % half], p.positions[t0 + i / half]);
        turn[i] = make_float2(cs.x * p.factor, cs.y * p.factor);
    }
    __syncthreads();

    const int parts = D / 16, heads = p.num_heads + p.num_kv_heads * (p.slots ? 2 : 1);
    const int units = n * heads * parts;
    for (int u = threadIdx.x; u < units; u += kThreads) {
        const int row = u / parts, part = u - row * parts, i = row / heads, h = row - i * heads;
        const int64_t t = t0 + i;
        const bool is_q = h < p.num_heads, is_v = h >= p.num_heads + p.num_kv_heads;
        const int hh = is_q ? h : h - p.num_heads - (is_v ? p.num_kv_heads : 0);
        int64_t dst_row;
        if (is_q) {
            dst_row = t * p.q_out_stride;
        } else if (p.slots) {
            const int64_t slot = p.slots[t];
            if (slot < 0 || slot >= p.num_slots) {
                if (slot != -1 && part == 0 && hh == 0 && !is_v) raise_error(p.err, PA_DEVERR_SLOT);
                continue;
            }
            dst_row = slot * p.num_kv_heads * D;
        } else {
            dst_row = t * p.k_out_stride;
        }
        const T *src = static_cast<const T *>(is_q ? p.q : (is_v ? p.v : p.k)) +
                       t * (is_q ? p.q_stride : (is_v ? p.v_stride : p.k_stride)) + hh * D;
        T *dst = static_cast<T *>(is_q ? p.q_out : (is_v ? p.v_out : p.k_out)) + dst_row + hh * D;
        const bool turned = !is_v && part * 8 < half;
        const int a = kInterleaved || !turned ? part * 16 : part * 8, b = kInterleaved || !turned ? a + 8 : a + half;
        float x[16];
        load8(src + a, x);
        load8(src + b, x + 8);
        if (turned) {
            const float2 *cs = turn + i * half + part * 8;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float &x1 = kInterleaved ? x[2 * j] : x[j], &x2 = kInterleaved ? x[2 * j + 1] : x[8 + j];
                const float2 w = cs[j];
                const float y1 = x1 * w.x - x2 * w.y, y2 = x2 * w.x + x1 * w.y;
                x1 = y1;
                x2 = y2;
            }
        }
        store8(dst + a, x);
        store8(dst + b, x + 8);
    }
}

template <typename T>
int launch_t(const RotaryParams &p, cudaStream_t stream) {
    const int tokens = 1;
    const int64_t grid = (p.num_tokens + tokens - 1) / tokens;
    return launch_pdl(p.interleaved ? rotary_kernel<T, true> : rotary_kernel<T, false>, dim3((unsigned)grid),
                      dim3(kThreads), (size_t)tokens * p.rotary_dim / 2 * sizeof(float2), stream, p, tokens);
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
