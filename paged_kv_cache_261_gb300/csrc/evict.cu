// Eviction from a paged cache by accumulated attention weight.
//
// Per sequence b and kv head h, with c the context length, n = min(c, keep_lens[b]) and
// r = min(recent, n): the last r tokens stay, and of the c - r before them the n - r of
// the largest mass (equal masses: the lower index first; a NaN counts below every
// number). The staying tokens keep their order; token kept[i] becomes token i.
//
// Selection (evict_select_kernel, one CTA per (sequence, kv head)): masses become
// unsigned keys of the same order, a radix descent over the key's digits finds the
// (n - r)-th largest key and how many of the tokens equal to it stay, and one ordered
// pass writes the indices and the masses. Counts and prefix sums are whole numbers, so
// the result does not depend on timing.
//
// Movement (evict_move_kernel): a CTA moves one slice of one plane's rows of one
// (sequence, kv head), tile after tile in increasing order, each tile read into
// registers by the whole CTA before any of it is written. Since kept[i] >= i and both
// rise, a tile's writes land on rows that no later tile reads, also when the
// out table names the sequence's own blocks (eviction in place).
#include "common.cuh"
#include "kernels_compress.h"

namespace pa {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kDigitBits = 11;
constexpr int kBins = 1 << kDigitBits;

// Masses as keys of the same order: NaN lowest, -0 equal to +0.
__device__ __forceinline__ uint32_t mass_key(float x) {
    if (x != x) return 0u;
    const uint32_t u = __float_as_uint(x + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix of v over the CTA's threads, in thread order; *total: the sum.
__device__ __forceinline__ int block_prefix(int v, int *warp_sums, int *total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
    }
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    int w = lane < kSelThreads / 32 ? warp_sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += u;
    }
    *total = __shfl_sync(0xffffffffu, w, 31);
    const int before = warp == 0 ? 0 : __shfl_sync(0xffffffffu, w, warp - 1);
    __syncthreads();                    // warp_sums may be reused
    return before + inc - v;
}

struct EvictSplit {
    int c, n, r;
};
__device__ __forceinline__ EvictSplit evict_split(const EvictParams &p, int b, bool report) {
    EvictSplit s;
    s.c = p.context_lens[b];
    int keep = p.keep_lens[b];
    bool bad = s.c < 0 || s.c > p.context_limit || keep < 0;
    s.c = max(0, min(s.c, p.context_limit));
    s.n = max(0, min(s.c, keep));
    if (s.n > p.keep_limit) {
        bad = true;
        s.n = p.keep_limit;
    }
    if (bad && report) raise_error(p.err, PA_DEVERR_CONTEXT);
    s.r = min(p.recent, s.n);
    return s;
}

__global__ __launch_bounds__(kSelThreads) void evict_select_kernel(const EvictParams p) {
    __shared__ int hist[kBins];
    __shared__ int warp_sums[32];
    __shared__ uint32_t found[2];       // the digit of the threshold, and how many keys lie above it
    const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
    const EvictSplit s = evict_split(p, b, tid == 0 && h == 0);
    const int64_t row = (int64_t)b * p.num_kv_heads + h;
    const float *mass = p.mass + row * p.mass_len;
    float *mass_out = p.mass_out + row * p.mass_out_len;
    int32_t *kept = p.kept + row * p.kept_len;
    const int cand = s.c - s.r;         // tokens that compete
    int want = s.n - s.r;               // how many of them stay
    // the want-th largest key among the candidates, digit by digit
    uint32_t key = 0, mask = 0;         // the digits found so far
    if (want > 0 && want < cand) {
        for (int shift = 32 - kDigitBits; ; shift = shift > kDigitBits ? shift - kDigitBits : 0) {
            const int bits = mask == 0 ? kDigitBits : min(kDigitBits, 32 - __popc(mask));
            const uint32_t dmask = ((1u << bits) - 1u) << shift;
            for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
            __syncthreads();
            for (int t = tid; t < cand; t += kSelThreads) {
                const uint32_t k = mass_key(mass[t]);
                if ((k & mask) == key) atomicAdd(&hist[(k & dmask) >> shift], 1);
            }
            __syncthreads();
            // thread i takes the bins counted from the top: 2i and 2i + 1
            const int top = (1 << bits) - 1, i0 = top - 2 * tid;
            const int h0 = i0 >= 0 ? hist[i0] : 0, h1 = i0 >= 1 ? hist[i0 - 1] : 0;
            int total;
            const int above = block_prefix(h0 + h1, warp_sums, &total);
            if (above < want && above + h0 >= want) {
                found[0] = (uint32_t)i0;
                found[1] = (uint32_t)above;
            } else if (above + h0 < want && above + h0 + h1 >= want) {
                found[0] = (uint32_t)(i0 - 1);
                found[1] = (uint32_t)(above + h0);
            }
            __syncthreads();
            key |= found[0] << shift;
            mask |= dmask;
            want -= (int)found[1];
            if (shift == 0) break;
            __syncthreads();
        }
    }
    // now: keys above `key` stay, and the first `want` equal to it
    const bool all = s.n - s.r >= cand, none = s.n - s.r <= 0;
    int base = 0, ties = 0;
    if (!none) {
        for (int t0 = 0; t0 < cand; t0 += kSelThreads) {
            const int t = t0 + tid;
            const float x = t < cand ? mass[t] : 0.f;
            const uint32_t k = mass_key(x);
            const int eq = t < cand && !all && k == key;
            int total;
            const int eq_before = block_prefix(eq, warp_sums, &total) + ties;
            ties += total;
            const int stay = t < cand && (all || k > key || (eq && eq_before < want));
            const int at = base + block_prefix(stay, warp_sums, &total);
            base += total;
            if (stay) {
                kept[at] = t;
                mass_out[at] = x;
            }
        }
    }
    for (int i0 = 0; i0 < s.r; i0 += kSelThreads) {      // the recent tokens, read before they are written
        const int i = i0 + tid;
        const float x = i < s.r ? mass[cand + i] : 0.f;
        __syncthreads();
        if (i < s.r) {
            kept[s.n - s.r + i] = cand + i;
            mass_out[s.n - s.r + i] = x;
        }
    }
    __syncthreads();
    for (int64_t i = s.n + tid; i < p.kept_len; i += kSelThreads) kept[i] = -1;
    for (int64_t i = s.n + tid; i < p.mass_out_len; i += kSelThreads) mass_out[i] = 0.f;
}

constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 4;

// VecT: 16 bytes (code and channel rows) or 8 (parameter rows).
template <typename VecT>
__device__ __forceinline__ void move_rows(const EvictParams &p, const EvictPlane &pl, const EvictSplit &s, int b,
                                          int h, const int32_t *kept) {
    const int vecs = pl.row_bytes / (int)sizeof(VecT);           // vectors per row
    const int32_t *src_table = p.block_tables + (int64_t)b * p.max_blocks;
    const int32_t *dst_table = p.out_block_tables + (int64_t)b * p.out_max_blocks;
    const int bs_mask = (1 << p.log2_block_size) - 1;
    char *base = pl.base + h * pl.head_stride;
    const int64_t total = (int64_t)s.n * vecs;
    for (int64_t i0 = 0; i0 < total; i0 += kMoveThreads * kMoveUnroll) {
        VecT v[kMoveUnroll];
        VecT *dst[kMoveUnroll];
#pragma unroll
        for (int u = 0; u < kMoveUnroll; ++u) {
            const int64_t i = i0 + u * kMoveThreads + threadIdx.x;
            dst[u] = nullptr;
            if (i >= total) continue;
            const int to = (int)(i / vecs), c = (int)(i - (int64_t)to * vecs);
            const int from = kept[to];
            const int32_t sb = src_table[from >> p.log2_block_size], db = dst_table[to >> p.log2_block_size];
            if (sb < 0 || sb >= p.num_blocks || db < 0 || db >= p.num_blocks) {
                raise_error(p.err, PA_DEVERR_BLOCK_ID);
                continue;
            }
            const VecT *src = reinterpret_cast<const VecT *>(base + sb * pl.block_stride +
                                                             (from & bs_mask) * pl.token_stride) + c;
            dst[u] = reinterpret_cast<VecT *>(base + db * pl.block_stride + (to & bs_mask) * pl.token_stride) + c;
            if (dst[u] == src) dst[u] = nullptr;                 // stays where it is
            else v[u] = *src;
        }
        __syncthreads();                                         // the whole tile has been read
#pragma unroll
        for (int u = 0; u < kMoveUnroll; ++u)
            if (dst[u]) *dst[u] = v[u];
    }
}

__global__ __launch_bounds__(kMoveThreads) void evict_move_kernel(const EvictParams p) {
    const int h = blockIdx.x, b = blockIdx.y;
    const EvictPlane &pl = p.planes[blockIdx.z];
    const EvictSplit s = evict_split(p, b, false);
    const int32_t *kept = p.kept + ((int64_t)b * p.num_kv_heads + h) * p.kept_len;
    if (pl.row_bytes % 16 == 0) move_rows<uint4>(p, pl, s, b, h, kept);
    else move_rows<uint2>(p, pl, s, b, h, kept);
}

}  // namespace

int launch_evict(const EvictParams &p, cudaStream_t stream) {
    evict_select_kernel<<<dim3((unsigned)p.num_kv_heads, (unsigned)p.num_seqs), kSelThreads, 0, stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return -1;
    evict_move_kernel<<<dim3((unsigned)p.num_kv_heads, (unsigned)p.num_seqs, (unsigned)p.num_planes), kMoveThreads, 0,
                        stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace pa
