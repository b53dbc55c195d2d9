// Scatter into a 4-bit paged cache, and its read-back.
//
// The slot arithmetic is that of "PagedAttention实现" write_kv and "04 - Paged
// Attention 实现进度" B.2 (slot = block * block_size + offset). The 4-bit format is not
// on the pages. Per token, kv head and tensor, a row x of head_dim channels becomes
//   zero  = f16(min x),  scale = f16((max x - min x) / 15)      (x clamped to +-65504)
//   code  = clamp(rint((x - zero) / scale), 0, 15), 0 where scale is 0
// in float32 with IEEE division, and stands for code * scale + zero. A row that holds a
// NaN gets NaN parameters, so it reads as NaN throughout. Codes are packed two to a
// byte (channel 2i low, 2i + 1 high); a block of one kv head is one contiguous run of
// block_size rows, and so are its (K scale, K zero, V scale, V zero) float16 quadruples.
//
// Both kernels: a row is head_dim / 8 lanes of 8 channels, so a lane moves 16 bytes of a
// 16-bit row and 4 bytes of codes; a K row and its V row sit side by side in a warp, and
// the extrema are butterfly shuffles inside a row's lanes.
#include "common.cuh"
#include "kernels_compress.h"

namespace pa {
namespace {

constexpr int kThreads = 256;

template <typename T> __device__ __forceinline__ void load8(const T *src, float *x);
template <> __device__ __forceinline__ void load8<float>(const float *src, float *x) {
    Vec16<float>::unpack(__ldcs(reinterpret_cast<const uint4 *>(src)), x);
    Vec16<float>::unpack(__ldcs(reinterpret_cast<const uint4 *>(src) + 1), x + 4);
}
template <> __device__ __forceinline__ void load8<__half>(const __half *src, float *x) {
    Vec16<__half>::unpack(__ldcs(reinterpret_cast<const uint4 *>(src)), x);
}
template <> __device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16 *src, float *x) {
    Vec16<__nv_bfloat16>::unpack(__ldcs(reinterpret_cast<const uint4 *>(src)), x);
}

template <typename T> __device__ __forceinline__ void store8(T *dst, const float *x) {
    alignas(16) T v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = Elem<T>::from_f(x[i]);
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4 *>(dst)[i] = reinterpret_cast<const uint4 *>(v)[i];
}

// min and max that give NaN when either operand is one
__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Row of the cache (in rows of one kv head's token) of a slot, or -1: skip the token.
__device__ __forceinline__ int64_t cache_row(const Int4Cache &c, int64_t slot, int h, bool first, unsigned int *err) {
    if (slot == -1) return -1;
    if (slot < 0 || slot >= c.num_slots) {
        if (first) raise_error(err, PA_DEVERR_SLOT);
        return -1;
    }
    const int64_t bs = int64_t(1) << c.log2_block_size;
    return (((slot >> c.log2_block_size) * c.num_kv_heads + h) << c.log2_block_size) + (slot & (bs - 1));
}

template <typename T, int D>
__global__ __launch_bounds__(kThreads) void kv_write_int4_kernel(const T *__restrict__ k, const T *__restrict__ v,
                                                                 const int32_t *__restrict__ slots,
                                                                 int64_t num_tokens, const Int4Cache c,
                                                                 unsigned int *err) {
    constexpr int kLanes = D / 8;                       // lanes per row
    // a decode launched after this kernel may start its set-up now; it waits for this
    // grid to finish before reading the cache
    asm volatile("griddepcontrol.launch_dependents;");
    const int64_t idx = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int part = (int)(idx % kLanes);               // which 8 channels
    const int64_t row = idx / kLanes;                   // ((token, kv head), K or V)
    const bool is_v = row & 1;
    const int64_t th = row >> 1;
    const int64_t t = th / c.num_kv_heads;
    const int h = (int)(th - t * c.num_kv_heads);
    const bool live = t < num_tokens;
    float x[8] = {};
    if (live) load8((is_v ? v : k) + th * D + part * 8, x);
    const int64_t dst = live ? cache_row(c, slots[t], h, part == 0 && h == 0 && !is_v, err) : -1;
    float lo = x[0], hi = x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        lo = min_nan(lo, x[i]);
        hi = max_nan(hi, x[i]);
    }
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) {
        lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    lo = max_nan(min_nan(lo, 65504.f), -65504.f);
    hi = max_nan(min_nan(hi, 65504.f), -65504.f);
    const __half zero_h = __float2half_rn(lo);
    const __half scale_h = __float2half_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.f));
    const float zero = __half2float(zero_h), scale = __half2float(scale_h);
    uint32_t codes = 0;
    if (scale > 0.f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float n = rintf(__fdiv_rn(__fsub_rn(x[i], zero), scale));
            codes |= (uint32_t)fminf(fmaxf(n, 0.f), 15.f) << (4 * i);
        }
    }
    const uint32_t mine = (uint32_t)__half_as_ushort(scale_h) | ((uint32_t)__half_as_ushort(zero_h) << 16);
    const uint32_t other = __shfl_xor_sync(0xffffffffu, mine, kLanes);   // the V row's, for the K row's lanes
    if (dst < 0) return;
    reinterpret_cast<uint32_t *>(is_v ? c.value : c.key)[dst * kLanes + part] = codes;
    if (part == 0 && !is_v) reinterpret_cast<uint2 *>(c.params)[dst] = make_uint2(mine, other);
}

template <typename T, int D>
__global__ __launch_bounds__(kThreads) void kv_read_int4_kernel(T *__restrict__ k, T *__restrict__ v,
                                                                const int32_t *__restrict__ slots,
                                                                int64_t num_tokens, const Int4Cache c,
                                                                unsigned int *err) {
    constexpr int kLanes = D / 8;
    const int64_t idx = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int part = (int)(idx % kLanes);
    const int64_t row = idx / kLanes;
    const bool is_v = row & 1;
    const int64_t th = row >> 1;
    const int64_t t = th / c.num_kv_heads;
    const int h = (int)(th - t * c.num_kv_heads);
    if (t >= num_tokens) return;
    const int64_t src = cache_row(c, slots[t], h, part == 0 && h == 0 && !is_v, err);
    if (src < 0) return;
    const uint32_t codes = reinterpret_cast<const uint32_t *>(is_v ? c.value : c.key)[src * kLanes + part];
    const float2 sz = __half22float2(reinterpret_cast<const __half2 *>(c.params)[src * 2 + is_v]);
    float x[8] = {};
    // code * scale is exact in float32 (4 + 11 bits), so the fused form rounds once
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = fmaf((float)((codes >> (4 * i)) & 15u), sz.x, sz.y);
    store8((is_v ? v : k) + th * D + part * 8, x);
}

// params[dst] = params[src] for each pair, in 16-byte vectors.
__global__ __launch_bounds__(kThreads) void copy_params_kernel(uint4 *params, const int32_t *__restrict__ pairs,
                                                               int64_t num_blocks, int64_t block_vecs,
                                                               unsigned int *err) {
    const int64_t src = pairs[2 * (int64_t)blockIdx.x], dst = pairs[2 * (int64_t)blockIdx.x + 1];
    if (src < 0 || src >= num_blocks || dst < 0 || dst >= num_blocks) {
        if (threadIdx.x == 0) raise_error(err, PA_DEVERR_COPY_PAIR);
        return;
    }
    for (int64_t i = threadIdx.x; i < block_vecs; i += kThreads)
        params[dst * block_vecs + i] = params[src * block_vecs + i];
}

int64_t row_grid(const Int4Cache &c, int64_t num_tokens) {
    const int64_t rows = num_tokens * 2 * c.num_kv_heads;
    return (rows * (c.head_dim / 8) + kThreads - 1) / kThreads;
}

template <typename T>
int write_t(const void *k, const void *v, const int32_t *slots, int64_t n, const Int4Cache &c, unsigned int *err,
            cudaStream_t s) {
    const int64_t grid = row_grid(c, n);
    if (grid > 0x7FFFFFFF) return -2;
    if (c.head_dim == 128)
        kv_write_int4_kernel<T, 128><<<(unsigned)grid, kThreads, 0, s>>>((const T *)k, (const T *)v, slots, n, c, err);
    else
        kv_write_int4_kernel<T, 64><<<(unsigned)grid, kThreads, 0, s>>>((const T *)k, (const T *)v, slots, n, c, err);
    return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

template <typename T>
int read_t(void *k, void *v, const int32_t *slots, int64_t n, const Int4Cache &c, unsigned int *err,
           cudaStream_t s) {
    const int64_t grid = row_grid(c, n);
    if (grid > 0x7FFFFFFF) return -2;
    if (c.head_dim == 128)
        kv_read_int4_kernel<T, 128><<<(unsigned)grid, kThreads, 0, s>>>((T *)k, (T *)v, slots, n, c, err);
    else
        kv_read_int4_kernel<T, 64><<<(unsigned)grid, kThreads, 0, s>>>((T *)k, (T *)v, slots, n, c, err);
    return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace

int launch_kv_write_int4(const void *k, const void *v, int src_dtype, const int32_t *slot_mapping,
                         int64_t num_tokens, const Int4Cache &c, unsigned int *err, cudaStream_t stream) {
    switch (src_dtype) {
    case PA_DTYPE_F32: return write_t<float>(k, v, slot_mapping, num_tokens, c, err, stream);
    case PA_DTYPE_F16: return write_t<__half>(k, v, slot_mapping, num_tokens, c, err, stream);
    case PA_DTYPE_BF16: return write_t<__nv_bfloat16>(k, v, slot_mapping, num_tokens, c, err, stream);
    default: return -2;
    }
}

int launch_kv_read_int4(void *k, void *v, int dst_dtype, const int32_t *slot_mapping, int64_t num_tokens,
                        const Int4Cache &c, unsigned int *err, cudaStream_t stream) {
    switch (dst_dtype) {
    case PA_DTYPE_F32: return read_t<float>(k, v, slot_mapping, num_tokens, c, err, stream);
    case PA_DTYPE_F16: return read_t<__half>(k, v, slot_mapping, num_tokens, c, err, stream);
    case PA_DTYPE_BF16: return read_t<__nv_bfloat16>(k, v, slot_mapping, num_tokens, c, err, stream);
    default: return -2;
    }
}

int launch_copy_params_int4(void *params, const int32_t *pairs, int64_t num_pairs, int64_t num_blocks,
                            int64_t block_bytes, unsigned int *err, cudaStream_t stream) {
    copy_params_kernel<<<(unsigned)num_pairs, kThreads, 0, stream>>>(static_cast<uint4 *>(params), pairs, num_blocks,
                                                                     block_bytes / 16, err);
    return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace pa
