// Scatter into an 8-bit paged cache with a scale for each block of tokens and kv head, and
// its read-back.
//
// The slot arithmetic is that of "PagedAttention实现" write_kv and "04 - Paged Attention
// 实现进度" B.2 (slot = block * block_size + offset). The format is not on the pages: E4M3 codes
// [num_blocks, num_kv_heads, block_size, head_dim] and, per block and kv head, a float32 scale
// for K and one for V; a channel stands for code * scale. The scatter makes a scale the
// smallest power of two 2^e, e >= -100, for which the largest finite magnitude in the block is
// at most 448 * 2^e (E4M3 is a floating-point format, so a scale between two powers of two would
// buy no precision, and dividing by a power of two is exact; a foreign scale becomes the next
// power of two). When new tokens make it grow, the
// codes that the block held are re-encoded: exact, but for those that come to lie below E4M3's
// normal numbers. A call that writes a block's first slot starts the block anew: what else it
// held, its scales too, counts no more.
//
// Tokens of one block stand next to each other in slot_mapping, so a block's new tokens are a
// run of it, which starts where the block of the token before is another. A team of warps takes
// a run of one kv head and of K or V: it reads the run's rows into registers, finds their largest
// magnitude, then the scale, re-encodes the block's older codes where the scale grew, and writes
// the new ones. A run of a single token (a decode step's) takes the lanes of one row, several
// side by side in a warp. (Atomic maxima over all tokens, whatever their order, would need the
// old scales kept beside the new ones and two more launches.)
//
// What bounds it (one GB300, 8 kv heads of 128 channels): a decode step's 64 tokens 1.9 us, the latency of
// three dependent loads; 8192 tokens, 50 MB, 10.7 us with the rows in L2 and 14.8 from HBM, instructions and the same chain
// with 16 warps an SM (five CTAs an SM, which spill, 11.1 and 15.2). All CTAs of a few tokens stand next to each other in the grid, so
// that their rows, which lie side by side, are read at the same time (heads far apart: 12.2). Reading back
// 131,071 tokens, 805 MB, takes 121 us, 6.65 TB/s, as fast as a copy; 8192 just written 7.2.
#include "common.cuh"
#include "kernels_fp8_block.h"

#include <algorithm>
#include <type_traits>

namespace pa {
namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;
// Rows of a lane held in registers: 16 a warp (8192 tokens of 64 channels with 16 and 32 rows a warp 7.8
// and 9.0 us, of 128 channels with 8 and 16 15.2 and 10.8).
template <int D> constexpr int kKeep = D / 32;
constexpr int kMinScaleExp = -100;
constexpr int kWriteCtas = 4;                    // of the scatter, on an SM (one less for float32 rows)
constexpr int kColumn = 32;                      // tokens, a lane each, whose runs the scatter's CTAs take together
template <typename T> constexpr int kWriteCtasOf = kWriteCtas - (sizeof(T) == 4);
// Channels per lane in reading: more where there are enough rows to fill the SMs all the same (us
// with 8 and 32 channels, 8 kv heads: 100 tokens 1.4, 1.6; 700 1.9, 1.9; 1000 2.4, 2.1).
constexpr int kFewChannels = 8, kManyChannels = 32;
constexpr int64_t kManyRows = 4096;              // (token, kv head) pairs
constexpr int kFullCtas = 14;                    // of reading, on an SM: there is little room for more
constexpr int kSmemOfSm = 228 * 1024, kSmemOfCta = 1024;   // bytes an SM has, and of them what a CTA takes by itself

template <typename T2> __device__ __forceinline__ T2 as2(uint32_t u) { return *reinterpret_cast<T2 *>(&u); }
template <typename T2> __device__ __forceinline__ uint32_t bits2(T2 v) { return *reinterpret_cast<uint32_t *>(&v); }
// The largest magnitude of some 16-bit (packed maxima) or float32 channels; NaN is passed over.
template <typename T2, int N> __device__ __forceinline__ uint32_t packed_largest(const uint4 (&raw)[N]) {
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (uint32_t w : {raw[i].x, raw[i].y, raw[i].z, raw[i].w})
            a = bits2(__hmax2(as2<T2>(a), __habs2(as2<T2>(w))));
    return bits2(__hmax2(as2<T2>(a), as2<T2>(__byte_perm(a, a, 0x1032))));
}
template <typename T, int N> __device__ __forceinline__ float largest_or_inf(const uint4 (&raw)[N]) {
    if constexpr (sizeof(T) == 2) {
        using T2 = std::conditional_t<std::is_same_v<T, __half>, __half2, __nv_bfloat162>;
        return Elem<T>::to_f(as2<T2>(packed_largest<T2>(raw)).x);
    } else {
        float a = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (uint32_t w : {raw[i].x, raw[i].y, raw[i].z, raw[i].w}) a = fmaxf(a, fabsf(__uint_as_float(w)));
        return a;
    }
}

// 16 channels of a row as loaded.
template <typename T> struct Run16 {
    uint4 raw[sizeof(T)];
    __device__ __forceinline__ void load(const T *src) {
#pragma unroll
        for (int u = 0; u < (int)sizeof(T); ++u) raw[u] = reinterpret_cast<const uint4 *>(src)[u];
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int u = 0; u < (int)sizeof(T); ++u) raw[u] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void values(float *x) const {
#pragma unroll
        for (int u = 0; u < (int)sizeof(T); ++u) Vec16<T>::unpack(raw[u], x + u * Vec16<T>::N);
    }
    // the largest finite magnitude
    __device__ __forceinline__ float largest() const {
        float x[16], a = largest_or_inf<T>(raw);
        if (a == INFINITY) {
            values(x);
            a = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) a = fmaxf(a, fabsf(x[i]) < INFINITY ? fabsf(x[i]) : 0.f);
        }
        return a;
    }
};

// Codes of x[0..15] * f (code i in byte i): nearest, ties to the even code, saturating at +-448,
// NaN to a NaN code.
__device__ __forceinline__ uint4 encode16(const float *x, float f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // products in pairs; of a conversion, the first source operand lands in the upper byte
        asm("{\n\t.reg .b64 a, b, s;\n\t.reg .f32 x0, x1, x2, x3;\n\t.reg .b16 lo, hi;\n\t"
            "mov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\tmov.b64 s, {%5, %5};\n\t"
            "mul.rn.f32x2 a, a, s;\n\tmul.rn.f32x2 b, b, s;\n\tmov.b64 {x0, x1}, a;\n\tmov.b64 {x2, x3}, b;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 lo, x1, x0;\n\tcvt.rn.satfinite.e4m3x2.f32 hi, x3, x2;\n\t"
            "mov.b32 %0, {lo, hi};\n\t}"
            : "=r"(w[i])
            : "f"(x[4 * i]), "f"(x[4 * i + 1]), "f"(x[4 * i + 2]), "f"(x[4 * i + 3]), "f"(f));
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

__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }   // -126..127

// The exponent of the scale of a block whose new tokens have magnitudes up to amax: the smallest
// e >= kMinScaleExp with amax <= 448 * 2^e = 1.75 * 2^(e + 8) and, where what the block holds under
// the scale `old` counts, old <= 2^e. (2^126 has an exact normal reciprocal.)
__device__ __forceinline__ int next_scale(float amax, float old, bool fresh, bool &held) {
    const uint32_t b = __float_as_uint(amax), o = __float_as_uint(old);
    const int e = max(kMinScaleExp, (int)(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0));
    held = !fresh && old > 0.f && old <= 0x1p126f;
    return held ? max(e, (int)(o >> 23) - 127 + ((o & 0x7FFFFFu) != 0 ? 1 : 0)) : e;
}

// The block of a slot, or -1: no token.
__device__ __forceinline__ int block_of(const Fp8BlockCache &c, int32_t slot) {
    return slot < 0 || slot >= c.num_slots ? -1 : slot >> c.log2_block_size;
}

// Re-encodes a block's rows first, first + step, ... of this lane's 16 channels, a few in flight
// at once; codes: of row 0.
template <int kLanes>
__device__ __forceinline__ void reencode(uint4 *codes, int first, int step, int bs, float ratio) {
    constexpr int kBatch = 4;
#pragma unroll 1
    for (int i0 = first; i0 < bs; i0 += kBatch * step) {
        uint4 old[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            if (i0 + u * step < bs) old[u] = codes[(i0 + u * step) * kLanes];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (i0 + u * step >= bs) break;
            float x[16];
            decode16(old[u], x);
            codes[(i0 + u * step) * kLanes] = encode16(x, ratio);
        }
    }
}

// 2^log2_team: warps that share a run (at most kWarps). `split` CTAs in a row take the runs that start in
// kColumn tokens of slot_mapping, so that their rows are read at the same time: the parts of all runs,
// in order, are dealt to their warps in turn, and a warp finds its own without passing by the others.
template <typename T, int D>
__global__ __launch_bounds__(kThreads, kWriteCtasOf<T>) void kv_write_fp8_block_kernel(const T *__restrict__ k, const T *__restrict__ v,
                                                                      int64_t k_stride, int64_t v_stride,
                                                                      const int32_t *__restrict__ slots,
                                                                      int64_t num_tokens, const Fp8BlockCache c,
                                                                      int log2_team, int split, unsigned int *err) {
    constexpr int kLanes = D / 16, kRows = 32 / kLanes;   // lanes of a row; rows of a warp
    __shared__ float maxima[kWarps];
    // launched as a dependent of the kernel before; a kernel launched after this one may start
    // its set-up once everything before this one has finished
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row = lane / kLanes, part = (lane % kLanes) * 16;
    const int Hk = c.num_kv_heads, bs = 1 << c.log2_block_size;
    // the runs that start in this CTA's tokens, from a window of 64: whether a token has a block,
    // continues the run of the token before, is its block's first
    const uint32_t column = blockIdx.x / (uint32_t)split, place = blockIdx.x - column * split;
    const int64_t t0 = (int64_t)column * kColumn;
    int32_t slot[2];
    int block[2];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const int64_t t = t0 + 32 * w + lane;
        slot[w] = t < num_tokens ? slots[t] : -1;
        block[w] = block_of(c, slot[w]);
    }
    const int last = lane == 0 && t0 > 0 ? block_of(c, slots[t0 - 1]) : -1;
    if (block[0] < 0 && slot[0] != -1 && place == 0 && warp == 0) raise_error(err, PA_DEVERR_SLOT);
    uint64_t goes_on = 0, firsts = 0;
    uint32_t starts = 0;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        int before = __shfl_up_sync(0xffffffffu, block[w], 1);
        const int end = __shfl_sync(0xffffffffu, block[0], 31);
        if (lane == 0) before = w == 0 ? last : end;
        goes_on |= (uint64_t)__ballot_sync(0xffffffffu, block[w] >= 0 && block[w] == before) << (32 * w);
        firsts |= (uint64_t)__ballot_sync(0xffffffffu, block[w] >= 0 && (slot[w] & (bs - 1)) == 0) << (32 * w);
        if (w == 0) starts = __ballot_sync(0xffffffffu, block[0] >= 0 && block[0] != before);
    }
    // a slot of the window's token i (each lane asks for its own)
    auto slot_at = [&](int i) {
        const int32_t lo = __shfl_sync(0xffffffffu, slot[0], i & 31), hi = __shfl_sync(0xffffffffu, slot[1], i & 31);
        return i < 32 ? lo : hi;
    };

    const int units = 2 * Hk, quads = (units + kRows - 1) / kRows;   // of a run: (kv head, K or V)
    const int warps = split * kWarps, my_warp = place * kWarps + warp;
    const int team = 1 << log2_team, group = warp >> log2_team, member = warp & (team - 1);
    const int teams = warps >> log2_team, my_team = my_warp >> log2_team;
    auto sync = [&] {
        if (team == 1) __syncwarp();
        else asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(team * 32) : "memory");
    };
    // the place of the r-th bit of a mask
    auto place_of = [&](uint32_t mask, int r) {
        return __ffs(__ballot_sync(0xffffffffu, (mask >> lane & 1) && __popc(mask & ((1u << lane) - 1)) == r)) - 1;
    };
    // Runs of one token: a unit for each row of the warp, every run's warps dealt in turn.
    const uint32_t singles = starts & ~(uint32_t)(goes_on >> 1);
    const int single_tasks = __popc(singles) * quads;
#pragma unroll 1
    for (int task = my_warp; task < single_tasks; task += warps) {
        const int r = task / quads, q = task - r * quads, s = place_of(singles, r);
        const int64_t first = t0 + s;
        const int at = slot_at(s), b = at >> c.log2_block_size, off = at & (bs - 1);
        const bool fresh = firsts >> s & 1;
        const int u = q * kRows + row;
        const bool live = u < units, is_v = u & 1;
        const int kvh = min(u >> 1, Hk - 1);
        float *scale_at = reinterpret_cast<float *>(c.scales + ((int64_t)b * Hk + kvh)) + is_v;
        Run16<T> x;
        x.load((is_v ? v + first * v_stride : k + first * k_stride) + kvh * D + part);
        const float old = *scale_at;
        float amax = x.largest();
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        bool held;
        const int e = next_scale(amax, old, fresh, held);
        const float scale = pow2f(e);
        uint4 *codes = reinterpret_cast<uint4 *>(static_cast<unsigned char *>(is_v ? c.value : c.key) +
                                                 (((int64_t)b * Hk + kvh) << c.log2_block_size) * D + part);
        // the older codes of these units, each by the whole warp
        uint32_t grown = __ballot_sync(0xffffffffu, live && held && scale > old && part == 0);
        for (; grown; grown &= grown - 1) {
            const int from = __ffs(grown) - 1;
            const uint64_t rows = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(codes), from);
            const float ratio = __shfl_sync(0xffffffffu, old * pow2f(-e), from);
            reencode<kLanes>(reinterpret_cast<uint4 *>(rows + part), row, kRows, bs, ratio);
        }
        __syncwarp();                                  // older codes before new ones
        if (live) {
            float y[16];
            x.values(y);
            codes[off * kLanes] = encode16(y, pow2f(-e));
            if (part == 0) *scale_at = scale;
        }
    }
    // Longer ones: a unit for each team, which follow where those ended.
    const uint32_t longer = starts & ~singles;
    const int tasks = __popc(longer) * units, skipped = single_tasks % warps >> log2_team;
#pragma unroll 1
    for (int task = my_team - skipped + (my_team < skipped ? teams : 0); task < tasks; task += teams) {
        const int r = task / units, u = task - r * units, s = place_of(longer, r);
        const int64_t first = t0 + s;
        const int b = slot_at(s) >> c.log2_block_size;
        // tokens of the run that the window shows, and beyond it
        int n = __ffsll((long long)~(goes_on >> (s + 1)));
        bool fresh = (firsts >> s & (~0ull >> (64 - n))) != 0;
        if (s + n == 64) {
            for (int len = 32; len == 32; n += len) {
                const int64_t t = first + n + lane;
                const int32_t next = t < num_tokens ? slots[t] : -1;
                const uint32_t other = ~__ballot_sync(0xffffffffu, block_of(c, next) == b);
                len = other ? __ffs(other) - 1 : 32;
                fresh |= __any_sync(0xffffffffu, lane < len && (next & (bs - 1)) == 0);
            }
        }
        const bool is_v = u & 1;
        const int kvh = u >> 1;
        const T *src = (is_v ? v + first * v_stride : k + first * k_stride) + kvh * D + part;
        const int64_t stride = is_v ? v_stride : k_stride;
        const int row0 = member * kRows + row, step = team * kRows;
        Run16<T> x[kKeep<D>];
        uint32_t offs = 0, lives = 0;                  // a row's place in its block, a byte each; whether there is one
        float *scale_at = reinterpret_cast<float *>(c.scales + ((int64_t)b * Hk + kvh)) + is_v;
        const float old = *scale_at;
#pragma unroll
        for (int j = 0; j < kKeep<D>; ++j) {
            const int i = row0 + j * step;
            x[j].clear();
            if (i < n) x[j].load(src + i * stride);
        }
#pragma unroll
        for (int j = 0; j < kKeep<D>; ++j) {
            const int i = row0 + j * step;
            const int32_t in_window = slot_at(min(s + i, 63));
            if (i < n) {
                offs |= (uint32_t)((s + i < 64 ? in_window : slots[first + i]) & (bs - 1)) << (8 * j);
                lives |= 1u << j;
            }
        }
        float amax = 0.f;
#pragma unroll
        for (int j = 0; j < kKeep<D>; ++j) amax = fmaxf(amax, x[j].largest());
#pragma unroll 1
        for (int i = row0 + kKeep<D> * step; i < n; i += step) {   // a long run of a large block
            Run16<T> more;
            more.load(src + i * stride);
            amax = fmaxf(amax, more.largest());
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if (team > 1) {
            if (lane == 0) maxima[warp] = amax;
            sync();
            for (int w = 0; w < team; ++w) amax = fmaxf(amax, maxima[group * team + w]);
        }
        bool held;
        const int e = next_scale(amax, old, fresh, held);
        const float scale = pow2f(e), inv = pow2f(-e);
        uint4 *codes = reinterpret_cast<uint4 *>(static_cast<unsigned char *>(is_v ? c.value : c.key) +
                                                 (((int64_t)b * Hk + kvh) << c.log2_block_size) * D + part);
        if (held && scale > old) reencode<kLanes>(codes, row0, step, bs, old * inv);
        sync();                                    // older codes before new ones; maxima and the old scale are read
#pragma unroll
        for (int j = 0; j < kKeep<D>; ++j) {
            float y[16];
            x[j].values(y);
            if (lives >> j & 1) codes[(offs >> (8 * j) & 255) * kLanes] = encode16(y, inv);
            asm volatile("" ::: "memory");         // one row after the other, for fewer registers
        }
#pragma unroll 1
        for (int i = row0 + kKeep<D> * step; i < n; i += step) {
            Run16<T> more;
            more.load(src + i * stride);
            float y[16];
            more.values(y);
            codes[(slots[first + i] & (bs - 1)) * kLanes] = encode16(y, inv);
        }
        if (member == 0 && lane == 0) *scale_at = scale;
    }
}

template <typename T> __device__ __forceinline__ void store8(T *dst, const float *x) {
    alignas(16) T v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = Elem<T>::from_f(x[i]);
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4 *>(dst)[i] = reinterpret_cast<const uint4 *>(v)[i];
}

// Reading: a lane has kCh channels of a row, in words of 8 a row's lanes apart, so that loads and
// stores of a warp are contiguous; a K row and its V row are side by side.
template <typename T, int D, int kCh>
__global__ __launch_bounds__(kThreads) void kv_read_fp8_block_kernel(T *__restrict__ k, T *__restrict__ v,
                                                                     const int32_t *__restrict__ slots,
                                                                     uint32_t num_tokens, const Fp8BlockCache c,
                                                                     unsigned int *err) {
    constexpr int kLanes = D / kCh, kWords = kCh / 8, kPairs = kThreads / kLanes / 2;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int part = threadIdx.x % kLanes;
    const bool is_v = (threadIdx.x / kLanes) & 1;
    const uint32_t th = blockIdx.x * kPairs + threadIdx.x / (2 * kLanes);   // (token, kv head) pair
    const uint32_t t = th / (uint32_t)c.num_kv_heads;
    const int h = (int)(th - t * c.num_kv_heads);
    if (t >= num_tokens) return;
    const int32_t slot = slots[t];
    const int64_t block = block_of(c, slot);
    if (block < 0) {
        if (slot != -1 && part == 0 && h == 0 && !is_v) raise_error(err, PA_DEVERR_SLOT);
        return;
    }
    const int64_t run = block * c.num_kv_heads + h;
    const int64_t row = (run << c.log2_block_size) + (slot & ((1 << c.log2_block_size) - 1));
    const uint2 *src = static_cast<const uint2 *>(is_v ? c.value : c.key) + row * (D / 8) + part;
    uint2 codes[kWords];
#pragma unroll
    for (int w = 0; w < kWords; ++w) codes[w] = __ldcs(src + w * kLanes);
    const float scale = reinterpret_cast<const float *>(c.scales + run)[is_v];
    T *dst = (is_v ? v : k) + (int64_t)th * D + part * 8;
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
        float x[8];
        decode4(codes[w].x, x);
        decode4(codes[w].y, x + 4);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= scale;
        store8(dst + w * kLanes * 8, x);
    }
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
            const Fp8BlockCache &c, int sms, unsigned int *err, cudaStream_t s) {
    constexpr int kRows = 32 / (D / 16);               // of a warp
    // as many warps a team as hold a block's rows in registers
    int log2_team = 0;
    while (1 << log2_team < kWarps && kRows * kKeep<D> << log2_team < 1 << c.log2_block_size) ++log2_team;
    // CTAs of a column: a warp for each unit of runs of 8 (8 kv heads, us with half, as many and twice: 16,384 tokens,
    // blocks of 16 23.9, 21.5, 24.2; 8192, of 32 12.6, 10.8, 13.6; of 256, f32 32.4, 30.8, 36.7), or more where columns
    // are few: as many as the device holds (us with three quarters, as many and one and a half times: single tokens of
    // 1024 sequences 3.6, 3.0, 4.1, of 2048 5.0, 4.4, 5.5; 2000 tokens of one 4.8, 3.6, 4.1, 50 of each of 40 5.6, 4.7, 5.8;
    // of f32, which fewer CTAs hold, as many and one and a third times: 3.8, 4.5, 6.1, 7.8, 6.3, 5.9, 7.0, 7.3), up
    // to a warp for each step that single tokens need.
    const int Hk = c.num_kv_heads;
    const int64_t columns = (n + kColumn - 1) / kColumn;
    const int64_t for_runs = ((Hk << log2_team) + 1) / 2;
    const int64_t for_singles = ((2 * Hk + kRows - 1) / kRows * kColumn + kWarps - 1) / kWarps;
    const int64_t ctas = std::max(for_runs, std::min(for_singles, (int64_t)sms * kWriteCtasOf<T> / columns));
    const int split = (int)std::max<int64_t>(1, std::min(ctas, INT32_MAX / columns));
    return launch_pdl(kv_write_fp8_block_kernel<T, D>, dim3((unsigned)(columns * split)), dim3(kThreads), 0, s,
                      (const T *)k, (const T *)v, ks, vs, slots, n, c, log2_team, split, err);
}

template <typename T, int D>
int read_t(void *k, void *v, const int32_t *slots, int64_t n, const Fp8BlockCache &c, int sms, unsigned int *err,
           cudaStream_t s) {
    const bool many = n * c.num_kv_heads >= kManyRows;
    const int pairs = kThreads / (D / (many ? kManyChannels : kFewChannels)) / 2;   // of a CTA
    const int64_t ctas = (n * c.num_kv_heads + pairs - 1) / pairs, each = (ctas + sms - 1) / sms;
    // CTAs of a dependent start where the kernel before leaves room, and small ones crowd the SMs that it leaves
    // first. Where the SMs are not full anyway, they ask for shared memory that no more fit into than spread
    // evenly (read-backs after a scatter, us of both without and so: 2159 tokens of 4 kv heads of 64 channels, f32
    // 13.9, 6.9, bf16 9.5, 5.7; 2000 of 8 10.5, 9.6; 560 4.2, 4.2; not launched as a dependent: 7.2, 5.9, 9.0, 4.0, but 1 to 2 us
    // more each outside a graph). (On another stream beside a decode, whose joining kernel waits in the rest of the SMs, a
    // read-back comes at its end with shared memory or without: after 485 and 474 of 490 us.)
    const int smem = each < kFullCtas ? (int)(kSmemOfSm / each) - kSmemOfCta : 0;
    auto kern = many ? kv_read_fp8_block_kernel<T, D, kManyChannels> : kv_read_fp8_block_kernel<T, D, kFewChannels>;
    static bool attr_set[2][kMaxDevices] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return -1;
    if (!attr_set[many][dev]) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemOfSm - kSmemOfCta) != cudaSuccess)
            return -1;
        attr_set[many][dev] = true;
    }
    return launch_pdl(kern, dim3((unsigned)ctas), dim3(kThreads), smem, s, (T *)k, (T *)v, slots, (uint32_t)n, c, err);
}

template <typename T>
int write_d(const void *k, const void *v, int64_t ks, int64_t vs, const int32_t *slots, int64_t n,
            const Fp8BlockCache &c, int sms, unsigned int *err, cudaStream_t s) {
    return c.head_dim == 128 ? write_t<T, 128>(k, v, ks, vs, slots, n, c, sms, err, s)
                             : write_t<T, 64>(k, v, ks, vs, slots, n, c, sms, err, s);
}
template <typename T>
int read_d(void *k, void *v, const int32_t *slots, int64_t n, const Fp8BlockCache &c, int sms, unsigned int *err,
           cudaStream_t s) {
    return c.head_dim == 128 ? read_t<T, 128>(k, v, slots, n, c, sms, err, s) : read_t<T, 64>(k, v, slots, n, c, sms, err, s);
}

}  // namespace

int launch_kv_write_fp8_block(const void *k, const void *v, int64_t k_stride, int64_t v_stride, int src_dtype,
                              const int32_t *slot_mapping, int64_t num_tokens, const Fp8BlockCache &c,
                              int sms, unsigned int *err, cudaStream_t stream) {
    switch (src_dtype) {
    case PA_DTYPE_F32: return write_d<float>(k, v, k_stride, v_stride, slot_mapping, num_tokens, c, sms, err, stream);
    case PA_DTYPE_F16: return write_d<__half>(k, v, k_stride, v_stride, slot_mapping, num_tokens, c, sms, err, stream);
    case PA_DTYPE_BF16:
        return write_d<__nv_bfloat16>(k, v, k_stride, v_stride, slot_mapping, num_tokens, c, sms, err, stream);
    default: return -2;
    }
}

int launch_kv_read_fp8_block(void *k, void *v, int dst_dtype, const int32_t *slot_mapping, int64_t num_tokens,
                             const Fp8BlockCache &c, int sms, unsigned int *err, cudaStream_t stream) {
    switch (dst_dtype) {
    case PA_DTYPE_F32: return read_d<float>(k, v, slot_mapping, num_tokens, c, sms, err, stream);
    case PA_DTYPE_F16: return read_d<__half>(k, v, slot_mapping, num_tokens, c, sms, err, stream);
    case PA_DTYPE_BF16: return read_d<__nv_bfloat16>(k, v, slot_mapping, num_tokens, c, sms, err, stream);
    default: return -2;
    }
}

int launch_copy_scales_fp8_block(float2 *scales, const int32_t *pairs, int64_t num_pairs, int64_t num_blocks,
                                 int num_kv_heads, unsigned int *err, cudaStream_t stream) {
    copy_scales_kernel<<<(unsigned)num_pairs, kThreads, 0, stream>>>(scales, pairs, num_blocks, num_kv_heads, err);
    return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace pa
