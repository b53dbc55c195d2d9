// Scatter into an 8-bit paged cache with a scale for each block of tokens and kv head, and
// its read-back.
//
// The slot arithmetic is that of "PagedAttention实现" write_kv and "04 - Paged Attention
// 实现进度" B.2 (slot = block * block_size + offset). The format is not on the pages: E4M3 codes
// [num_blocks, num_kv_heads, block_size, head_dim] and, per block and kv head, a float32 scale
// for K and one for V; a channel stands for code * scale. The scatter makes a scale the
// smallest power of two 2^e, e >= -100, for which the largest finite magnitude in the block is
// at most 448 * 2^e (E4M3 is a floating-point format, so a scale between two powers of two would
// buy no precision, and dividing by a power of two is exact). When new tokens make it grow, the
// codes that the block held are re-encoded: exact, but for those that come to lie below E4M3's
// normal numbers. A call that writes a block's first slot starts the block anew: what else it
// held, its scales too, counts no more.
//
// Tokens of one block stand next to each other in slot_mapping, so a block's new tokens are a
// run of it, which starts where the block of the token before is another. A team of warps takes
// a run of one kv head and of K or V: it finds the run's largest magnitude, then the scale,
// re-encodes the block's older codes where the scale grew, and writes the new ones. (Atomic
// maxima over all tokens, whatever their order, would need the old scales kept beside the new
// ones and two more launches.)
#include "common.cuh"
#include "kernels_fp8_block.h"

namespace pa {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMinScaleExp = -100;

// 16 channels of a row as floats.
template <typename T> __device__ __forceinline__ void load16(const T *src, float *x) {
    constexpr int N = Vec16<T>::N;
#pragma unroll
    for (int u = 0; u < 16 / N; ++u) Vec16<T>::unpack(reinterpret_cast<const uint4 *>(src)[u], x + u * N);
}

// Codes of x[0..15] / scale (code i in byte i): nearest, ties to the even code, saturating at
// +-448, NaN to a NaN code. inv: 1 / scale where scale is a power of two (the product is then
// the quotient), else 0.
__device__ __forceinline__ uint4 encode16(const float *x, float scale, float inv) {
    float y[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = inv != 0.f ? x[i] * inv : __fdiv_rn(x[i], scale);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint16_t lo, hi;
        // the first source operand lands in the upper byte
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(y[4 * i + 1]), "f"(y[4 * i]));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(y[4 * i + 3]), "f"(y[4 * i + 2]));
        w[i] = (uint32_t)lo | ((uint32_t)hi << 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Four codes as floats (exact).
__device__ __forceinline__ void decode4(uint32_t w, float *x) {
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
    const float2 p = __half22float2(*reinterpret_cast<__half2 *>(&lo)), q = __half22float2(*reinterpret_cast<__half2 *>(&hi));
    x[0] = p.x; x[1] = p.y; x[2] = q.x; x[3] = q.y;
}
__device__ __forceinline__ void decode16(const uint4 &c, float *x) {
    decode4(c.x, x);
    decode4(c.y, x + 4);
    decode4(c.z, x + 8);
    decode4(c.w, x + 12);
}

// The smallest 2^e, e >= kMinScaleExp, with amax <= 448 * 2^e = 1.75 * 2^(e + 8).
__device__ __forceinline__ float scale_for(float amax) {
    const uint32_t b = __float_as_uint(amax);
    const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return __uint_as_float((uint32_t)(max(e, kMinScaleExp) + 127) << 23);
}
// 1 / s where s is a power of two whose reciprocal is exact, else 0.
__device__ __forceinline__ float exact_inverse(float s) {
    const uint32_t b = __float_as_uint(s), e = b >> 23;
    return (b & 0x7FFFFFu) == 0 && e >= 1 && e <= 253 ? __uint_as_float((254 - e) << 23) : 0.f;
}

// The block of a slot, or -1: no token.
__device__ __forceinline__ int64_t block_of(const Fp8BlockCache &c, int64_t slot) {
    return slot < 0 || slot >= c.num_slots ? -1 : slot >> c.log2_block_size;
}

// team: warps that share a run (a power of two, at most kWarps); chunk: tokens of
// slot_mapping whose runs a CTA column takes (at most 32).
template <typename T, int D>
__global__ __launch_bounds__(kThreads) void kv_write_fp8_block_kernel(const T *__restrict__ k, const T *__restrict__ v,
                                                                      int64_t k_stride, int64_t v_stride,
                                                                      const int32_t *__restrict__ slots,
                                                                      int64_t num_tokens, const Fp8BlockCache c,
                                                                      int team, int chunk, unsigned int *err) {
    constexpr int kLanes = D / 16, kRows = 32 / kLanes;   // lanes of a row; rows of a warp
    __shared__ float maxima[kWarps];
    // launched as a dependent of the kernel before; a kernel launched after this one may start
    // its set-up once everything before this one has finished
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = warp / team, member = warp - group * team, groups = kWarps / team;
    const int row0 = member * kRows + lane / kLanes, part = (lane % kLanes) * 16;
    const int row_step = team * kRows;
    const int Hk = c.num_kv_heads, bs = 1 << c.log2_block_size;
    auto sync = [&] {
        if (team == 1) __syncwarp();
        else asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(team * 32) : "memory");
    };

    // the runs that start in this CTA's tokens
    const int64_t t0 = (int64_t)blockIdx.x * chunk;
    uint32_t starts;
    {
        const int64_t t = t0 + lane;
        const bool in = lane < chunk && t < num_tokens;
        const int64_t slot = in ? slots[t] : -1, b = block_of(c, slot);
        if (in && b < 0 && slot != -1 && blockIdx.y == 0 && warp == 0) raise_error(err, PA_DEVERR_SLOT);
        starts = __ballot_sync(0xffffffffu, b >= 0 && (t == 0 || block_of(c, slots[t - 1]) != b));
    }
    const int64_t units = (int64_t)__popc(starts) * Hk * 2;
    for (int64_t u = (int64_t)blockIdx.y * groups + group; u < units; u += (int64_t)gridDim.y * groups) {
        const int r = (int)(u / (2 * Hk)), kvh = (int)(u - (int64_t)r * 2 * Hk) >> 1;
        const bool is_v = u & 1;
        uint32_t m = starts;
        for (int i = 0; i < r; ++i) m &= m - 1;
        const int64_t first = t0 + __ffs(m) - 1, block = block_of(c, slots[first]);
        // its length, and whether it starts the block
        int64_t n = 0;
        bool fresh = false;
        for (int len = 32; len == 32; n += len) {
            const int64_t t = first + n + lane;
            const int64_t slot = t < num_tokens ? slots[t] : -1;
            const uint32_t other = ~__ballot_sync(0xffffffffu, block_of(c, slot) == block);
            len = other ? __ffs(other) - 1 : 32;
            fresh |= __any_sync(0xffffffffu, lane < len && (slot & (bs - 1)) == 0);
        }
        const T *src = (is_v ? v + first * v_stride : k + first * k_stride) + kvh * D + part;
        const int64_t stride = is_v ? v_stride : k_stride;
        float amax = 0.f;
        for (int64_t i = row0; i < n; i += row_step) {
            float x[16];
            load16(src + i * stride, x);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float a = fabsf(x[j]);
                amax = fmaxf(amax, a < INFINITY ? a : 0.f);
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        float *scale_at = reinterpret_cast<float *>(c.scales + block * Hk + kvh) + is_v;
        const float old = *scale_at;
        if (lane == 0) maxima[warp] = amax;
        sync();
        for (int w = 0; w < team; ++w) amax = fmaxf(amax, maxima[group * team + w]);
        const bool held = !fresh && old > 0.f && old < INFINITY;
        const float scale = held ? fmaxf(old, scale_for(amax)) : scale_for(amax), inv = exact_inverse(scale);
        uint4 *codes = reinterpret_cast<uint4 *>(static_cast<unsigned char *>(is_v ? c.value : c.key) +
                                                 ((block * Hk + kvh) << c.log2_block_size) * D + part);
        if (held && scale > old) {
            const float ratio = __fdiv_rn(old, scale);
            for (int i = row0; i < bs; i += row_step) {
                float x[16];
                decode16(codes[i * kLanes], x);
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] *= ratio;
                codes[i * kLanes] = encode16(x, 1.f, 1.f);
            }
        }
        sync();                                        // older codes before new ones; the old scale is read
        for (int64_t i = row0; i < n; i += row_step) {
            float x[16];
            load16(src + i * stride, x);
            codes[(slots[first + i] & (bs - 1)) * kLanes] = encode16(x, scale, inv);
        }
        if (member == 0 && lane == 0) *scale_at = scale;
    }
}

template <typename T> __device__ __forceinline__ void store16(T *dst, const float *x) {
    alignas(16) T v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = Elem<T>::from_f(x[i]);
#pragma unroll
    for (int i = 0; i < (int)sizeof(T); ++i) reinterpret_cast<uint4 *>(dst)[i] = reinterpret_cast<const uint4 *>(v)[i];
}

// A lane has 16 channels of a row; a K row and its V row are side by side.
template <typename T, int D>
__global__ __launch_bounds__(kThreads) void kv_read_fp8_block_kernel(T *__restrict__ k, T *__restrict__ v,
                                                                     const int32_t *__restrict__ slots,
                                                                     uint32_t num_tokens, const Fp8BlockCache c,
                                                                     unsigned int *err) {
    constexpr int kLanes = D / 16, kPairs = kThreads / kLanes / 2;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int part = threadIdx.x % kLanes;
    const bool is_v = (threadIdx.x / kLanes) & 1;
    const uint32_t th = blockIdx.x * kPairs + threadIdx.x / (2 * kLanes);   // (token, kv head) pair
    const uint32_t t = th / (uint32_t)c.num_kv_heads;
    const int h = (int)(th - t * c.num_kv_heads);
    if (t >= num_tokens) return;
    const int64_t slot = slots[t], block = block_of(c, slot);
    if (block < 0) {
        if (slot != -1 && part == 0 && h == 0 && !is_v) raise_error(err, PA_DEVERR_SLOT);
        return;
    }
    const int64_t run = block * c.num_kv_heads + h;
    const int64_t row = (run << c.log2_block_size) + (slot & ((1 << c.log2_block_size) - 1));
    const float2 s = c.scales[run];
    const float scale = is_v ? s.y : s.x;
    float x[16];
    decode16(__ldcs(static_cast<const uint4 *>(is_v ? c.value : c.key) + row * kLanes + part), x);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] *= scale;
    store16((is_v ? v : k) + (int64_t)th * D + part * 16, x);
}

// scales[dst] = scales[src] for each pair of blocks.
__global__ __launch_bounds__(kThreads) void copy_scales_kernel(float2 *scales, const int32_t *__restrict__ pairs,
                                                               int64_t num_blocks, int num_kv_heads,
                                                               unsigned int *err) {
    const int64_t src = pairs[2 * (int64_t)blockIdx.x], dst = pairs[2 * (int64_t)blockIdx.x + 1];
    if (src < 0 || src >= num_blocks || dst < 0 || dst >= num_blocks) {
        if (threadIdx.x == 0) raise_error(err, PA_DEVERR_COPY_PAIR);
        return;
    }
    for (int i = threadIdx.x; i < num_kv_heads; i += kThreads)
        scales[dst * num_kv_heads + i] = scales[src * num_kv_heads + i];
}

template <typename T, int D>
int write_t(const void *k, const void *v, int64_t ks, int64_t vs, const int32_t *slots, int64_t n,
            const Fp8BlockCache &c, unsigned int *err, cudaStream_t s) {
    // a warp per 16 rows of a block
    const int team = std::max(1, std::min(kWarps, (1 << c.log2_block_size) / 16));
    const int chunk = 32;
    const int64_t units = (int64_t)chunk * 2 * c.num_kv_heads, groups = kWarps / team;
    const int64_t x = (n + chunk - 1) / chunk;
    const int64_t y = std::min<int64_t>((units + groups - 1) / groups, 2 * c.num_kv_heads);
    return launch_pdl(kv_write_fp8_block_kernel<T, D>, dim3((unsigned)x, (unsigned)std::min<int64_t>(y, 65535)),
                      dim3(kThreads), 0, s, (const T *)k, (const T *)v, ks, vs, slots, n, c, team, chunk, err);
}

template <typename T, int D>
int read_t(void *k, void *v, const int32_t *slots, int64_t n, const Fp8BlockCache &c, unsigned int *err,
           cudaStream_t s) {
    const int pairs = kThreads / (D / 16) / 2;         // of a CTA
    return launch_pdl(kv_read_fp8_block_kernel<T, D>, dim3((unsigned)((n * c.num_kv_heads + pairs - 1) / pairs)),
                      dim3(kThreads), 0, s, (T *)k, (T *)v, slots, (uint32_t)n, c, err);
}

template <typename T>
int write_d(const void *k, const void *v, int64_t ks, int64_t vs, const int32_t *slots, int64_t n,
            const Fp8BlockCache &c, unsigned int *err, cudaStream_t s) {
    return c.head_dim == 128 ? write_t<T, 128>(k, v, ks, vs, slots, n, c, err, s)
                             : write_t<T, 64>(k, v, ks, vs, slots, n, c, err, s);
}
template <typename T>
int read_d(void *k, void *v, const int32_t *slots, int64_t n, const Fp8BlockCache &c, unsigned int *err,
           cudaStream_t s) {
    return c.head_dim == 128 ? read_t<T, 128>(k, v, slots, n, c, err, s) : read_t<T, 64>(k, v, slots, n, c, err, s);
}

}  // namespace

int launch_kv_write_fp8_block(const void *k, const void *v, int64_t k_stride, int64_t v_stride, int src_dtype,
                              const int32_t *slot_mapping, int64_t num_tokens, const Fp8BlockCache &c,
                              unsigned int *err, cudaStream_t stream) {
    switch (src_dtype) {
    case PA_DTYPE_F32: return write_d<float>(k, v, k_stride, v_stride, slot_mapping, num_tokens, c, err, stream);
    case PA_DTYPE_F16: return write_d<__half>(k, v, k_stride, v_stride, slot_mapping, num_tokens, c, err, stream);
    case PA_DTYPE_BF16:
        return write_d<__nv_bfloat16>(k, v, k_stride, v_stride, slot_mapping, num_tokens, c, err, stream);
    default: return -2;
    }
}

int launch_kv_read_fp8_block(void *k, void *v, int dst_dtype, const int32_t *slot_mapping, int64_t num_tokens,
                             const Fp8BlockCache &c, unsigned int *err, cudaStream_t stream) {
    switch (dst_dtype) {
    case PA_DTYPE_F32: return read_d<float>(k, v, slot_mapping, num_tokens, c, err, stream);
    case PA_DTYPE_F16: return read_d<__half>(k, v, slot_mapping, num_tokens, c, err, stream);
    case PA_DTYPE_BF16: return read_d<__nv_bfloat16>(k, v, slot_mapping, num_tokens, c, err, stream);
    default: return -2;
    }
}

int launch_copy_scales_fp8_block(float2 *scales, const int32_t *pairs, int64_t num_pairs, int64_t num_blocks,
                                 int num_kv_heads, unsigned int *err, cudaStream_t stream) {
    copy_scales_kernel<<<(unsigned)num_pairs, kThreads, 0, stream>>>(scales, pairs, num_blocks, num_kv_heads, err);
    return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace pa
