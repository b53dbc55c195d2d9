// Eviction from a paged cache by accumulated attention weight.
//
// Per sequence b and kv head h, with c the context length, n = min(c, keep_lens[b]) and
// r = min(recent, n): the last r tokens stay, and of the c - r before them the n - r of
// the largest mass (equal masses: the lower index first; a NaN counts below every
// number). The staying tokens keep their order; token kept[i] becomes token i.
//
// Selection (evict_select_kernel, a CTA or a cluster of them per (sequence, kv head)): the row's
// masses are read once, each CTA keeping a slice in shared memory. As unsigned keys of the
// same order, a radix descent over three digits finds the (n - r)-th largest key and how
// many of the tokens equal to it stay: each CTA counts its slice's digits, and every CTA
// adds the counts of the cluster. Then each warp writes the indices and masses that stay
// of its part of the slice, behind those that the parts before it keep. Counts are whole
// numbers, so the result does not depend on timing, and every mass has been read before
// the first is written, so mass_out may be mass.
//
// A call's tables and masses bound its rows before their lengths are known, so the cluster,
// its shared memory and this choice follow what they hold, not the contexts: where they hold
// more than 393,216 tokens, too many for a cluster's shared memory, every row of the call takes
// evict_select_long_kernel: one CTA, the masses read again for every digit, written in one
// ordered pass (8 kv heads, one context, cut to 4000: 393,216 tokens 54 us in all by clusters,
// 393,232 by this kernel 489, a million 1229).
//
// Movement (evict_move_kernel, a cluster of CTAs per (sequence, kv head, plane)): the rows
// move in waves, each read into registers by the whole cluster before any of it is
// written. Since kept[i] >= i and both rise, a wave's writes land on rows that no later
// wave reads, also when the out table names the sequence's own blocks (eviction in place).
//
// What bounds it (one GB300): 64 sequences of 512 to 4096 tokens, 8 kv heads, cut to 1024 in
// bf16 take 102 us: the movement 84, at 6.4 TB/s of rows read and written, and the selection
// 16.5, its barriers and counts. For 8 sequences of 32k to 128k cut to 8192 the selection takes
// 54 us (two waves of CTAs, with 21 MB of masses beside their counts in shared memory).
#include <cooperative_groups.h>

#include <algorithm>

#include "common.cuh"
#include "kernels_compress.h"

namespace pa {
namespace {

namespace cg = cooperative_groups;

constexpr int kSelThreads = 1024;       // of the kernel for long rows
constexpr int kDigitBits = 11;
constexpr int kBins = 1 << kDigitBits;

// Masses as keys of the same order: NaN lowest, -0 equal to +0.
__device__ __forceinline__ uint32_t mass_key(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    return x == x ? u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u) : 0u;
}

// Exclusive prefix of v over the CTA's threads, in thread order; *total: the sum.
template <int kThreads> __device__ __forceinline__ int block_prefix(int v, int *warp_sums, int *total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
    }
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    int w = lane < kThreads / 32 ? warp_sums[lane] : 0;
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

__global__ __launch_bounds__(kSelThreads) void evict_select_long_kernel(const EvictParams p) {
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
            const int above = block_prefix<kSelThreads>(h0 + h1, warp_sums, &total);
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
            const int eq_before = block_prefix<kSelThreads>(eq, warp_sums, &total) + ties;
            ties += total;
            const int stay = t < cand && (all || k > key || (eq && eq_before < want));
            const int at = base + block_prefix<kSelThreads>(stay, warp_sums, &total);
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

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxSlice = 48 * 1024;    // masses per CTA: 192 KB of shared memory
constexpr int kList = 2048;             // long 4-bit contexts 189 -> 179 us, with their read-back
__global__ __launch_bounds__(kThreads) void evict_select_kernel(const EvictParams p) {
    extern __shared__ __align__(16) float slice[];      // this CTA's masses
    __shared__ __align__(16) int hist[kBins];
    __shared__ __align__(16) int sums[kBins / 2];      // this CTA's part of the cluster's counts
    __shared__ uint32_t seg[kWarps];    // sums of each warp
    __shared__ int found[3];            // the digit of the threshold, how many keys lie above it, and how many
                                        // of this CTA's have it (the counts themselves are cleared soon)
    __shared__ uint32_t list[kList];    // keys of the candidates that share the threshold's first digit,
    __shared__ unsigned char list_warp[kList];   // whose warp's tokens they are,
    __shared__ int listed;                       // how many,
    __shared__ uint32_t extra[kWarps];           // and how many of a warp's stay, ties << 16
    __shared__ uint32_t counts;         // of this CTA's slice: tokens that stay anyway, ties << 16
    cg::cluster_group cluster = cg::this_cluster();
    const int nc = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = blockIdx.x / nc, b = blockIdx.y;
    // (no early trigger: the moving CTAs, resident early, slowed the second wave of long rows)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const EvictSplit s = evict_split(p, b, tid == 0 && blockIdx.x == 0);
    const int64_t row = (int64_t)b * p.num_kv_heads + h;
    const float *mass = p.mass + row * p.mass_len;
    float *mass_out = p.mass_out + row * p.mass_out_len;
    int32_t *kept = p.kept + row * p.kept_len;
    const int cand = s.c - s.r;         // tokens that compete
    int want = s.n - s.r;               // how many of them stay
    const bool all = want >= cand, none = want <= 0;

    // this CTA's tokens [t0, t0 + len), and this warp's part [w0, w1) of them
    const int per = (((s.c + nc - 1) / nc) + 3) & ~3;
    const int t0 = min(s.c, rank * per), len = min(s.c, t0 + per) - t0;
    const int n_cand = max(0, min(len, cand - t0));
    const int wlen = (((len + kWarps - 1) / kWarps) + 127) & ~127;
    const int w0 = min(len, warp * wlen), w1 = min(len, w0 + wlen);
    const bool search = !all && !none;
    auto sync = [&]() {
        if (nc > 1) cluster.sync();
        else __syncthreads();
    };
    static_assert(kBins == 4 * kThreads, "four bins a thread");
    reinterpret_cast<int4 *>(hist)[tid] = make_int4(0, 0, 0, 0);
    if (tid < kWarps) extra[tid] = 0;
    if (tid == 0) listed = 0;
    __syncthreads();
    // the masses come in, and the first digit of their keys is counted
    constexpr int kFirst = 32 - kDigitBits;
    {
        constexpr int kUnroll = 8;
        for (int i0 = 0; i0 < len; i0 += kThreads * kUnroll) {
            float v[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int i = i0 + u * kThreads + tid;
                v[u] = i < len ? mass[t0 + i] : 0.f;
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int i = i0 + u * kThreads + tid;
                if (i < len) slice[i] = v[u];
                if (search && i < n_cand) atomicAdd(&hist[mass_key(v[u]) >> kFirst], 1);
            }
        }
    }
    uint32_t key = 0, mask = 0, sum = 0;   // the digits found; this warp's tokens that stay anyway, ties << 16
    bool short_list = false;
    if (search) {
        for (int shift = kFirst;; shift = shift > kDigitBits ? shift - kDigitBits : 0) {
            const int bits = shift > 0 ? kDigitBits : 32 - 2 * kDigitBits;
            const uint32_t digits = (1u << bits) - 1u;
            if (shift != kFirst) {
                reinterpret_cast<int4 *>(hist)[tid] = make_int4(0, 0, 0, 0);
                __syncthreads();
                const int n = short_list ? listed : n_cand;
                for (int i = tid; i < n; i += kThreads) {
                    const uint32_t k = short_list ? list[i] : mass_key(slice[i]);
                    if ((k & mask) == key) atomicAdd(&hist[(k >> shift) & digits], 1);
                }
            }
            sync();
            if (nc > 1) {
                // CTA r adds up the r-th part of the bins over the cluster (every CTA reading all
                // counts of all others took 21 us of the 70 on long contexts)
                const int part = kBins / nc;
                for (int i = tid; i < part; i += kThreads) {
                    int t = 0;
#pragma unroll
                    for (int c = 0; c < kMaxCluster; ++c)
                        if (c < nc) t += cluster.map_shared_rank(hist, c)[rank * part + i];
                    sums[i] = t;
                }
                cluster.sync();
            }
            // thread i: the bins counted from the top, 4 i to 4 i + 3, of the whole cluster
            const int i0 = (int)digits - 4 * tid;
            int n[4] = {0, 0, 0, 0};
            if (i0 >= 3) {
                const int part = kBins / nc, b0 = i0 - 3;
                const int4 v = *reinterpret_cast<const int4 *>(
                    nc > 1 ? cluster.map_shared_rank(sums, b0 / part) + b0 % part : hist + b0);
                n[0] = v.w;
                n[1] = v.z;
                n[2] = v.y;
                n[3] = v.x;
            }
            const int mine = n[0] + n[1] + n[2] + n[3];
            const int of_warp = __reduce_add_sync(0xffffffffu, mine);
            if (lane == 0) seg[warp] = (uint32_t)of_warp;
            __syncthreads();
            // the warp that holds the threshold looks for it among its bins
            const int v = lane < kWarps ? (int)seg[lane] : 0;
            int up_to = v;
#pragma unroll
            for (int o = 1; o < kWarps; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, up_to, o);
                if (lane >= o) up_to += x;
            }
            const int target = __ffs(__ballot_sync(0xffffffffu, up_to >= want)) - 1;
            if (warp == target) {
                int above = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int x = __shfl_up_sync(0xffffffffu, above, o);
                    if (lane >= o) above += x;
                }
                above += __shfl_sync(0xffffffffu, up_to - v, target) - mine;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (above < want && above + n[j] >= want) {
                        found[0] = i0 - j;
                        found[1] = above;
                        found[2] = hist[i0 - j];
                    }
                    above += n[j];
                }
            }
            sync();                     // every CTA has read the counts
            key |= (uint32_t)found[0] << shift;
            mask |= digits << shift;
            want -= found[1];
            if (shift == 0) break;
            if (shift == kFirst && found[2] <= kList) {
                // few candidates share the threshold's first digit: the other digits, and the
                // verdict on the rest, need no further pass over the slice
                short_list = true;
                for (int i = w0 + 4 * lane; i < w1; i += 128) {
                    const float4 x4 = *reinterpret_cast<const float4 *>(slice + i);
                    const float x[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t k = mass_key(x[j]), d = k >> kFirst;
                        const bool in = i + j < n_cand;
                        sum += i + j < w1 && (!in || d > (key >> kFirst));
                        if (in && i + j < w1 && d == key >> kFirst) {
                            const int at = atomicAdd(&listed, 1);
                            list[at] = k;
                            list_warp[at] = (unsigned char)warp;
                        }
                    }
                }
                __syncthreads();
            }
        }
    }
    __syncthreads();
    // ---- what stays: the recent tokens, keys above `key`, and the first `want` equal to it
    static_assert(kMaxSlice < 65536, "counts of a slice in 16 bits");
    // token i of the slice: 1 = stays anyway, 1 << 16 = equal to the threshold
    auto verdict = [&](float x, int i) -> uint32_t {
        const uint32_t k = mass_key(x);
        const bool sure = t0 + i >= cand || all || (!none && k > key);
        return i >= w1 ? 0u : (sure ? 1u : (!none && k == key ? 0x10000u : 0u));
    };
    if (short_list) {
        for (int i = tid; i < listed; i += kThreads) {
            const uint32_t k = list[i];
            if (k >= key) atomicAdd(&extra[list_warp[i]], k > key ? 1u : 0x10000u);
        }
        __syncthreads();
    } else {
        for (int i = w0 + 4 * lane; i < w1; i += 128) {
            const float4 x = *reinterpret_cast<const float4 *>(slice + i);
            sum += verdict(x.x, i) + verdict(x.y, i + 1) + verdict(x.z, i + 2) + verdict(x.w, i + 3);
        }
    }
    sum = __reduce_add_sync(0xffffffffu, sum) + extra[warp];
    if (lane == 0) seg[warp] = sum;
    __syncthreads();
    uint32_t up_to = lane < kWarps ? seg[lane] : 0u;    // of the warps 0 .. lane
#pragma unroll
    for (int o = 1; o < kWarps; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, up_to, o);
        if (lane >= o) up_to += v;
    }
    const uint32_t whole = __shfl_sync(0xffffffffu, up_to, kWarps - 1);
    const uint32_t ahead = warp == 0 ? 0u : __shfl_sync(0xffffffffu, up_to, warp - 1);
    int sure_before = (int)(ahead & 0xFFFFu), ties_before = (int)(ahead >> 16);   // this warp's tokens
    if (nc > 1) {
        if (tid == 0) counts = whole;
        cluster.sync();                 // every mass of the row has been read, too
        for (int c = 0; c < rank; ++c) {
            const uint32_t o = *cluster.map_shared_rank(&counts, c);
            sure_before += (int)(o & 0xFFFFu);
            ties_before += (int)(o >> 16);
        }
    }
    for (int i0 = w0; i0 < w1; i0 += 128) {
        const int i = i0 + 4 * lane;
        const float4 x4 = i < w1 ? *reinterpret_cast<const float4 *>(slice + i) : make_float4(0.f, 0.f, 0.f, 0.f);
        const float x[4] = {x4.x, x4.y, x4.z, x4.w};
        uint32_t d[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) d[j] = verdict(x[j], i + j);
        const uint32_t mine = d[0] + d[1] + d[2] + d[3];
        uint32_t upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        const uint32_t tile = __shfl_sync(0xffffffffu, upto, 31);
        int sure = sure_before + (int)((upto - mine) & 0xFFFFu), ties = ties_before + (int)((upto - mine) >> 16);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool tie = d[j] >> 16;
            // position: the sure ones before, and the ties before, of which `want` stay
            if (d[j] == 1u || (tie && ties < want)) {
                const int at = sure + min(ties, want);
                kept[at] = t0 + i + j;
                mass_out[at] = x[j];
            }
            sure += (int)(d[j] & 1u);
            ties += tie;
        }
        sure_before += (int)(tile & 0xFFFFu);
        ties_before += (int)(tile >> 16);
    }
    for (int64_t i = s.n + rank * kThreads + tid; i < p.kept_len; i += nc * kThreads) kept[i] = -1;
    for (int64_t i = s.n + rank * kThreads + tid; i < p.mass_out_len; i += nc * kThreads) mass_out[i] = 0.f;
    if (nc > 1) cluster.sync();         // the counts are read by other CTAs until here
}

constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 4;

// kSide: the rows have parameters (4-bit caches). A plane's CTAs move its half of them, a row a
// thread. (CTAs of their own, a third of the launch for a ninth of the bytes, took as long as the
// others: long 4-bit contexts 159.5 us, with their read-back, against 152.)
template <bool kSide>
__device__ __forceinline__ void move_rows(const EvictParams &p, const EvictPlane &pl, const EvictSplit &s, int b,
                                          int h, const int32_t *kept, int rank, int nc, int part, int parts) {
    cg::cluster_group cluster = cg::this_cluster();
    const uint32_t vecs = (uint32_t)pl.row_bytes / 16u / (uint32_t)parts;   // vectors of a row that this CTA moves
    const int32_t *src_table = p.block_tables + (int64_t)b * p.max_blocks;
    const int32_t *dst_table = p.out_block_tables + (int64_t)b * p.out_max_blocks;
    const int bs_mask = (1 << p.log2_block_size) - 1;
    char *base = pl.base + h * pl.head_stride + part * (int)(vecs * 16);
    [[maybe_unused]] char *side = kSide ? pl.side + ((h * pl.head_stride) >> pl.side_shift) : nullptr;
    // A wave: up to 256 whole rows a CTA, kMoveUnroll vectors a thread. While a wave's rows are
    // read, the next one's places are looked up, one row a thread, into shared memory.
    const uint32_t rows_cta = min((uint32_t)kMoveThreads, kMoveThreads * kMoveUnroll / vecs);
    const uint32_t used = rows_cta * vecs;
    const int64_t step = (int64_t)rows_cta * nc;
    __shared__ longlong2 place[2][kMoveThreads];                 // source and destination in bytes, or -1
    auto index = [&](int64_t r0) -> int {                        // this thread's row of the wave: its source token
        const int64_t to = r0 + (int64_t)rank * rows_cta + threadIdx.x;
        return threadIdx.x < rows_cta && to < s.n ? kept[to] : -1;
    };
    auto look_up = [&](int64_t r0, int from, int buf) {
        longlong2 at = make_longlong2(-1, -1);
        if (from >= 0) {
            const int to = (int)(r0 + (int64_t)rank * rows_cta + threadIdx.x);
            const int32_t sb = src_table[from >> p.log2_block_size], db = dst_table[to >> p.log2_block_size];
            if (sb < 0 || sb >= p.num_blocks || db < 0 || db >= p.num_blocks) {
                raise_error(p.err, PA_DEVERR_BLOCK_ID);
            } else {
                at.x = sb * pl.block_stride + (from & bs_mask) * pl.token_stride;
                at.y = db * pl.block_stride + (to & bs_mask) * pl.token_stride;
                if (at.x == at.y) at.y = -1;                     // stays where it is
            }
        }
        place[buf][threadIdx.x] = at;
    };
    int from = index(0);
    look_up(0, from, 0);
    from = index(step);
    __syncthreads();
    int buf = 0;
    for (int64_t r0 = 0; r0 < s.n; r0 += step, buf ^= 1) {
        uint4 v[kMoveUnroll], *dst[kMoveUnroll];
        [[maybe_unused]] uint32_t sv = 0, *sdst = nullptr;       // the parameters of row threadIdx.x
        if (kSide && threadIdx.x < rows_cta) {
            const longlong2 at = place[buf][threadIdx.x];
            if (at.y >= 0) {
                sv = *reinterpret_cast<const uint32_t *>(side + (at.x >> pl.side_shift));
                sdst = reinterpret_cast<uint32_t *>(side + (at.y >> pl.side_shift));
            }
        }
#pragma unroll
        for (int u = 0; u < kMoveUnroll; ++u) {
            const uint32_t i = u * kMoveThreads + threadIdx.x;
            const uint32_t r = i / vecs, c = i - r * vecs;
            dst[u] = nullptr;
            if (i >= used) continue;
            const longlong2 at = place[buf][r];
            if (at.y < 0) continue;
            v[u] = reinterpret_cast<const uint4 *>(base + at.x)[c];
            dst[u] = reinterpret_cast<uint4 *>(base + at.y) + c;
        }
        look_up(r0 + step, from, buf ^ 1);
        from = index(r0 + 2 * step);
        if (nc > 1) cluster.sync();                              // the whole wave has been read
        else __syncthreads();
#pragma unroll
        for (int u = 0; u < kMoveUnroll; ++u)
            if (dst[u]) *dst[u] = v[u];
        if (kSide && sdst) *sdst = sv;
    }
}

template <bool kSide> __global__ __launch_bounds__(kMoveThreads) void evict_move_kernel(const EvictParams p) {
    cg::cluster_group cluster = cg::this_cluster();
    const int nc = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int h = blockIdx.x / nc, b = blockIdx.y;
    const EvictPlane &pl = p.planes[blockIdx.z & 1];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const EvictSplit s = evict_split(p, b, false);
    const int32_t *kept = p.kept + ((int64_t)b * p.num_kv_heads + h) * p.kept_len;
    move_rows<kSide>(p, pl, s, b, h, kept, rank, nc, (int)(blockIdx.z >> 1), (int)(gridDim.z >> 1));
}

template <typename Kern>
int launch_cluster(Kern kern, int heads, int seqs, int z, int cluster, int threads, size_t smem, cudaStream_t stream,
                   const EvictParams &p) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(heads * cluster), (unsigned)seqs, (unsigned)z);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess ? 0 : -1;
}

// CTAs per cluster: enough that the launch fills the SMs twice, at most 8.
int cluster_for(int64_t units, int sms) {
    int c = 1;
    while (c < kMaxCluster && units * c < 2 * (int64_t)sms) c *= 2;
    return c;
}

}  // namespace

int launch_evict(const EvictParams &p, int sms, cudaStream_t stream) {
    static bool attr_set[kMaxDevices] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return -1;
    if (!attr_set[dev]) {
        if (cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSlice * 4) !=
            cudaSuccess)
            return -1;
        attr_set[dev] = true;
    }
    const int64_t rows = (int64_t)p.num_seqs * p.num_kv_heads;
    // The selection's clusters grow with the longest row that there may be, to 16384 masses a CTA:
    // what a cluster's barriers cost is more than its other CTAs save (8 kv heads, whole call, us, against clusters
    // that fill the SMs: one sequence of 300 tokens 8.5 and 14.7, 16 of 2000 14.7 and 33.6, 16 of
    // 16000 23.9 and 37.7, 4 of 40000 25.9 and 27.4; one of 16000 18.6 and 17.2). Short rows in wide
    // tables and masses pay for it: 64 sequences of 512 to 4096, 8 kv heads, evicted in place to 1024
    // again and again, 44 us in all where 4096 tokens fit, 50 at 16384, 85 at 32768, 250 at 131072.
    int c = 1;
    while (c < kMaxCluster && (int64_t)c * 16384 < p.context_limit) c *= 2;
    const int64_t slice = ((p.context_limit + c - 1) / c + 3) & ~int64_t(3);
    int rc = 0;
    if (slice <= kMaxSlice) {
        rc = launch_cluster(evict_select_kernel, p.num_kv_heads, p.num_seqs, 1, c, kThreads, (size_t)slice * 4, stream,
                            p);
    } else {
        evict_select_long_kernel<<<dim3((unsigned)p.num_kv_heads, (unsigned)p.num_seqs), kSelThreads, 0, stream>>>(p);
        rc = cudaGetLastError() == cudaSuccess ? 0 : -1;
    }
    if (rc != 0) return rc;
    // Where few rows' clusters leave SMs idle, a row's vectors, which move independently, are
    // parted among clusters, to no less than 64 bytes (4-bit rows are no longer and stay whole):
    // 8 kv heads, bf16, one context of 100,000 cut to 4000 39.8 -> 30.9 us, two cut to 30,000
    // 176 -> 135.
    int parts = 1;
    const int vecs = p.planes[0].row_bytes / 16;
    while (rows * 2 * parts * kMaxCluster < 2 * (int64_t)sms && vecs % (2 * parts) == 0 && vecs / (2 * parts) >= 4)
        parts *= 2;
    // the movement's clusters fill the SMs, but have no more CTAs than one wave takes (50 tokens of 8
    // kv heads: 8.5 -> 7.9 us in all)
    int m = cluster_for(rows * 2 * parts, sms);
    const int64_t wave = std::min<int64_t>(kMoveThreads, kMoveThreads * kMoveUnroll / (vecs / parts));
    while (m > 1 && (m / 2) * wave >= p.keep_limit) m /= 2;
    return launch_cluster(p.planes[0].side ? evict_move_kernel<true> : evict_move_kernel<false>, p.num_kv_heads,
                          p.num_seqs, 2 * parts, m, kMoveThreads, 0, stream, p);
}

}  // namespace pa
