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
// In both kernels a row is shared by a few lanes, and a K row and its V row sit side by
// side in a warp; the extrema are butterfly shuffles inside a row's lanes.
#include "common.cuh"
#include "kernels_compress.h"

#include <type_traits>

namespace pa {
namespace {

constexpr int kThreads = 128;

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

// The smallest and largest of some channels. In 16 bits packed as (min, -max), so that one
// packed min takes both further.
template <typename T> struct Extrema;
template <> struct Extrema<float> {
    float lo, hi;
    __device__ __forceinline__ void merge(const Extrema &o) {
        lo = min_nan(lo, o.lo);
        hi = max_nan(hi, o.hi);
    }
    __device__ __forceinline__ Extrema of_lane(int mask) const {
        return {__shfl_xor_sync(0xffffffffu, lo, mask), __shfl_xor_sync(0xffffffffu, hi, mask)};
    }
    __device__ __forceinline__ float2 values() const { return make_float2(lo, hi); }
};
template <typename T2> __device__ __forceinline__ T2 as2(uint32_t u) { return *reinterpret_cast<T2 *>(&u); }
template <typename T2> __device__ __forceinline__ uint32_t bits2(T2 v) { return *reinterpret_cast<uint32_t *>(&v); }
template <typename T, typename T2> struct PackedExtrema {
    uint32_t both;
    __device__ __forceinline__ void merge_bits(uint32_t o) { both = bits2(__hmin2_nan(as2<T2>(both), as2<T2>(o))); }
    __device__ __forceinline__ float2 values() const {
        float f[8];
        Vec16<T>::unpack(make_uint4(both, 0, 0, 0), f);
        return make_float2(f[0], -f[1]);
    }
};
template <> struct Extrema<__half> : PackedExtrema<__half, __half2> {
    using T2 = __half2;
    __device__ __forceinline__ void merge(const Extrema &o) { merge_bits(o.both); }
    __device__ __forceinline__ Extrema of_lane(int mask) const {
        Extrema e;
        e.both = __shfl_xor_sync(0xffffffffu, both, mask);
        return e;
    }
};
template <> struct Extrema<__nv_bfloat16> : PackedExtrema<__nv_bfloat16, __nv_bfloat162> {
    using T2 = __nv_bfloat162;
    __device__ __forceinline__ void merge(const Extrema &o) { merge_bits(o.both); }
    __device__ __forceinline__ Extrema of_lane(int mask) const {
        Extrema e;
        e.both = __shfl_xor_sync(0xffffffffu, both, mask);
        return e;
    }
};

// Eight channels of a row as loaded.
template <typename T> struct Run8 {
    uint4 raw;
    __device__ __forceinline__ void load(const T *src) { raw = *reinterpret_cast<const uint4 *>(src); }
    __device__ __forceinline__ void clear() { raw = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void values(float *x) const { Vec16<T>::unpack(raw, x); }
    __device__ __forceinline__ Extrema<T> extrema() const {
        using T2 = typename Extrema<T>::T2;
        const T2 a = as2<T2>(raw.x), b = as2<T2>(raw.y), c = as2<T2>(raw.z), d = as2<T2>(raw.w);
        const uint32_t mn = bits2(__hmin2_nan(__hmin2_nan(a, b), __hmin2_nan(c, d)));
        const uint32_t mx = bits2(__hmax2_nan(__hmax2_nan(a, b), __hmax2_nan(c, d)));
        // (mn.lo, -mx.lo) and (mn.hi, -mx.hi)
        Extrema<T> e;
        e.both = __byte_perm(mn, mx, 0x5410) ^ 0x80000000u;
        e.merge_bits(__byte_perm(mn, mx, 0x7632) ^ 0x80000000u);
        return e;
    }
};
template <> struct Run8<float> {
    uint4 raw[2];
    __device__ __forceinline__ void load(const float *src) {
        raw[0] = reinterpret_cast<const uint4 *>(src)[0];
        raw[1] = reinterpret_cast<const uint4 *>(src)[1];
    }
    __device__ __forceinline__ void clear() { raw[0] = raw[1] = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void values(float *x) const {
        Vec16<float>::unpack(raw[0], x);
        Vec16<float>::unpack(raw[1], x + 4);
    }
    __device__ __forceinline__ Extrema<float> extrema() const {
        float x[8];
        values(x);
        Extrema<float> e{x[0], x[0]};
#pragma unroll
        for (int i = 1; i < 8; ++i) e.merge({x[i], x[i]});
        return e;
    }
};

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

// Eight codes of (x - zero) / scale; inv15 is the reciprocal of scale, over 15. The product,
// clamped as a number in [0, 1], decides unless it is so near a tie that the IEEE quotient has to
// (they differ by less than 2^-18).
__device__ __forceinline__ uint32_t encode8(const float *x, float zero, float scale, float inv15) {
    constexpr float kMagic = 12582912.f;                 // 1.5 * 2^23: adding it rounds to an integer
    float n[8], off = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float t = __saturatef(__fmul_rn(__fsub_rn(x[i], zero), inv15));
        n[i] = __fsub_rn(__fmaf_rn(t, 15.f, kMagic), kMagic);
        off = fmaxf(off, fabsf(__fmaf_rn(t, 15.f, -n[i])));
    }
    if (off > 0.5f - 6e-6f) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            n[i] = fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(x[i], zero), scale)), 0.f), 15.f);
    }
    // four codes make a whole number below 2^16
    float four[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
        four[h] = __fmaf_rn(__fmaf_rn(n[4 * h + 3], 16.f, n[4 * h + 2]), 256.f, __fmaf_rn(n[4 * h + 1], 16.f, n[4 * h]));
    return __byte_perm(__float_as_uint(__fadd_rn(four[0], 8388608.f)), __float_as_uint(__fadd_rn(four[1], 8388608.f)),
                       0x5410);
}

// Writing: a lane has kCh channels of a row. What is done once a row -- the shuffles, the
// parameters, the slot's address -- is most of a lane's instructions at 8 channels, and the
// kernel is bound by instructions (8192 tokens of 8 kv heads, written and read back: 26.8 us
// at 8, 23.3 at 16, 21.3 at 32; two rows a lane were slower at each. Clamping and packing in
// float arithmetic, off the integer pipe: 20.9; with the wider reading 19.4, 64 channels 21.4;
// CTAs of 128 threads rather than 256: 19.1).
template <typename T, int D, int kCh>
__global__ __launch_bounds__(kThreads) void kv_write_int4_kernel(const T *__restrict__ k, const T *__restrict__ v,
                                                                 const int32_t *__restrict__ slots,
                                                                 uint32_t num_tokens, const Int4Cache c,
                                                                 unsigned int *err) {
    constexpr int kLanes = D / kCh, kWords = kCh / 8;   // lanes per row; 8 channels, a word of codes, each
    constexpr int kPairs = kThreads / kLanes / 2;
    // launched as a dependent of the kernel before; a kernel launched after this one may start
    // its set-up once everything before this one has finished
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int part = threadIdx.x % kLanes;
    const bool is_v = (threadIdx.x / kLanes) & 1;
    const uint32_t th = blockIdx.x * kPairs + threadIdx.x / (2 * kLanes);   // (token, kv head) pair
    const uint32_t t = th / (uint32_t)c.num_kv_heads;
    const int h = (int)(th - t * c.num_kv_heads);
    Run8<T> x[kWords];
#pragma unroll
    for (int w = 0; w < kWords; ++w) x[w].clear();
    int64_t dst = -1;
    if (t < num_tokens) {
        const T *src = (is_v ? v : k) + (int64_t)th * D + part * kCh;
#pragma unroll
        for (int w = 0; w < kWords; ++w) x[w].load(src + 8 * w);
        dst = cache_row(c, slots[t], h, part == 0 && h == 0 && !is_v, err);
    }
    Extrema<T> e = x[0].extrema();
#pragma unroll
    for (int w = 1; w < kWords; ++w) e.merge(x[w].extrema());
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) e.merge(e.of_lane(o));
    const float2 range = e.values();
    const float lo = max_nan(min_nan(range.x, 65504.f), -65504.f);
    const float hi = max_nan(min_nan(range.y, 65504.f), -65504.f);
    const __half zero_h = __float2half_rn(lo);
    const __half scale_h = __float2half_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.f));
    const float zero = __half2float(zero_h), scale = __half2float(scale_h);
    const float inv15 = scale > 0.f ? __fdiv_rn(__frcp_rn(scale), 15.f) : 0.f;
    alignas(16) uint32_t codes[kWords];
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
        float y[8];
        x[w].values(y);
        // The clamp itself, above: it shows where the minimum rounds up to a zero next to 65504, as
        // only float32 can (below, the zero is -65504 and the code 0 either way).
        if constexpr (std::is_same_v<T, float>) {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = fminf(y[i], 65504.f);
        }
        codes[w] = scale > 0.f ? encode8(y, zero, scale, inv15) : 0u;
    }
    const uint32_t mine = (uint32_t)__half_as_ushort(scale_h) | ((uint32_t)__half_as_ushort(zero_h) << 16);
    const uint32_t other = __shfl_xor_sync(0xffffffffu, mine, kLanes);   // the V row's, for the K row's lanes
    if (dst < 0) return;
    uint32_t *out = reinterpret_cast<uint32_t *>(is_v ? c.value : c.key) + dst * (D / 8) + part * kWords;
    if constexpr (kWords == 4) *reinterpret_cast<uint4 *>(out) = *reinterpret_cast<uint4 *>(codes);
    else if constexpr (kWords == 2) *reinterpret_cast<uint2 *>(out) = *reinterpret_cast<uint2 *>(codes);
    else out[0] = codes[0];
    if (part == 0 && !is_v) reinterpret_cast<uint2 *>(c.params)[dst] = make_uint2(mine, other);
}

// Reading: a lane has kCh channels of a row, in words of 8 a row's lanes apart, so that loads and
// stores of a warp are contiguous; again most instructions come once a row (131,071 tokens of 8
// kv heads: 8 channels 206 us, four such rows a lane 109.7, 16 channels of two rows 103.8, 32 of
// one 103.2, 6.6 TB/s).
template <typename T, int D, int kCh>
__global__ __launch_bounds__(kThreads) void kv_read_int4_kernel(T *__restrict__ k, T *__restrict__ v,
                                                                const int32_t *__restrict__ slots,
                                                                uint32_t num_tokens, const Int4Cache c,
                                                                unsigned int *err) {
    constexpr int kLanes = D / kCh, kWords = kCh / 8;
    constexpr int kPairs = kThreads / kLanes / 2;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int part = threadIdx.x % kLanes;
    const bool is_v = (threadIdx.x / kLanes) & 1;
    const uint32_t th = blockIdx.x * kPairs + threadIdx.x / (2 * kLanes);   // (token, kv head) pair
    const uint32_t t = th / (uint32_t)c.num_kv_heads;
    const int h = (int)(th - t * c.num_kv_heads);
    if (t >= num_tokens) return;
    const int64_t src = cache_row(c, slots[t], h, part == 0 && h == 0 && !is_v, err);
    if (src < 0) return;
    const uint32_t *row = reinterpret_cast<const uint32_t *>(is_v ? c.value : c.key) + src * (D / 8) + part;
    uint32_t codes[kWords];
#pragma unroll
    for (int w = 0; w < kWords; ++w) codes[w] = __ldcs(row + w * kLanes);
    const float2 f = __half22float2(reinterpret_cast<const __half2 *>(c.params)[src * 2 + is_v]);
    const float scale = f.x * 16777216.f;
    T *dst = (is_v ? v : k) + (int64_t)th * D + part * 8;
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
        // a code in an f16's low bits is code * 2^-24, so no integer is converted; its product
        // with the scale is exact in float32 (4 + 11 bits), so the fused form rounds once
        float x[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 n = __half22float2(as2<__half2>((codes[w] >> (4 * i)) & 0x000F000Fu));
            x[i] = fmaf(n.x, scale, f.y);
            x[i + 4] = fmaf(n.y, scale, f.y);
        }
        store8(dst + w * kLanes * 8, x);
    }
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

// Channels per lane: more where there are enough rows to fill the SMs all the same.
constexpr int kFewChannels = 8, kManyChannels = 32;
// (8192 pairs written and read back 6.6 us at 8, 6.2 at 32; 2048 3.9 and 4.9.)
constexpr int64_t kManyRows = 4096;              // (token, kv head) pairs

template <int D> unsigned row_grid(const Int4Cache &c, int64_t num_tokens, int channels) {
    const int pairs = kThreads / (D / channels) / 2;     // of a CTA
    return (unsigned)((num_tokens * c.num_kv_heads + pairs - 1) / pairs);
}

template <typename T, int D>
int write_t(const void *k, const void *v, const int32_t *slots, int64_t n, const Int4Cache &c, unsigned int *err,
            cudaStream_t s) {
    const bool many = n * c.num_kv_heads >= kManyRows;
    auto kern = many ? kv_write_int4_kernel<T, D, kManyChannels> : kv_write_int4_kernel<T, D, kFewChannels>;
    return launch_pdl(kern, dim3(row_grid<D>(c, n, many ? kManyChannels : kFewChannels)), dim3(kThreads), 0, s,
                      (const T *)k, (const T *)v, slots, (uint32_t)n, c, err);
}

template <typename T, int D>
int read_t(void *k, void *v, const int32_t *slots, int64_t n, const Int4Cache &c, unsigned int *err,
           cudaStream_t s) {
    const bool many = n * c.num_kv_heads >= kManyRows;
    auto kern = many ? kv_read_int4_kernel<T, D, kManyChannels> : kv_read_int4_kernel<T, D, kFewChannels>;
    return launch_pdl(kern, dim3(row_grid<D>(c, n, many ? kManyChannels : kFewChannels)), dim3(kThreads), 0, s, (T *)k,
                      (T *)v, slots, (uint32_t)n, c, err);
}

template <typename T>
int write_d(const void *k, const void *v, const int32_t *slots, int64_t n, const Int4Cache &c, unsigned int *err,
            cudaStream_t s) {
    return c.head_dim == 128 ? write_t<T, 128>(k, v, slots, n, c, err, s) : write_t<T, 64>(k, v, slots, n, c, err, s);
}
template <typename T>
int read_d(void *k, void *v, const int32_t *slots, int64_t n, const Int4Cache &c, unsigned int *err,
           cudaStream_t s) {
    return c.head_dim == 128 ? read_t<T, 128>(k, v, slots, n, c, err, s) : read_t<T, 64>(k, v, slots, n, c, err, s);
}

}  // namespace

int launch_kv_write_int4(const void *k, const void *v, int src_dtype, const int32_t *slot_mapping,
                         int64_t num_tokens, const Int4Cache &c, unsigned int *err, cudaStream_t stream) {
    switch (src_dtype) {
    case PA_DTYPE_F32: return write_d<float>(k, v, slot_mapping, num_tokens, c, err, stream);
    case PA_DTYPE_F16: return write_d<__half>(k, v, slot_mapping, num_tokens, c, err, stream);
    case PA_DTYPE_BF16: return write_d<__nv_bfloat16>(k, v, slot_mapping, num_tokens, c, err, stream);
    default: return -2;
    }
}

int launch_kv_read_int4(void *k, void *v, int dst_dtype, const int32_t *slot_mapping, int64_t num_tokens,
                        const Int4Cache &c, unsigned int *err, cudaStream_t stream) {
    switch (dst_dtype) {
    case PA_DTYPE_F32: return read_d<float>(k, v, slot_mapping, num_tokens, c, err, stream);
    case PA_DTYPE_F16: return read_d<__half>(k, v, slot_mapping, num_tokens, c, err, stream);
    case PA_DTYPE_BF16: return read_d<__nv_bfloat16>(k, v, slot_mapping, num_tokens, c, err, stream);
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
