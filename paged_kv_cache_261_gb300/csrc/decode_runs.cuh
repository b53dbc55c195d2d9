// What the decode kernels over quantised caches share whose work is cut into equal runs of
// stages, one run a warp: the cut, the rows' book-keeping, the kernel that joins the partials of
// rows that several runs share, and the warp-level instructions they are built from.
#pragma once

#include "common.cuh"
#include "f32x2.cuh"
#include "kernels_compress.h"
#include "sm100.cuh"

#include <algorithm>

namespace pa {
namespace {

using namespace sm100;

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            smem_addr(dst)),
        "l"(src), "r"(bytes), "r"(smem_addr(bar))
        : "memory");
}

__device__ __forceinline__ void mma16816(float *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
        "%2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The warp's 8x8 matrix of 16-bit elements, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// Largest value over the lanes of the same lane & 3 (the rows of a fragment's column).
__device__ __forceinline__ float rows_max(float v) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float rows_sum(float v) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }   // -126..127

// The cut of `total` stages into `warps` runs: the first `longer` of them have `len` + 1
// stages, the others `len`; run w starts at stage first(w).
struct Runs {
    uint32_t len, longer;
    __device__ __forceinline__ Runs(uint32_t total, uint32_t warps) : len(total / warps), longer(total - len * warps) {}
    __device__ __forceinline__ uint32_t first(uint32_t w) const { return w * len + min(w, longer); }
    // the run that holds stage s
    __device__ __forceinline__ uint32_t owner(uint32_t s) const {
        const uint32_t head = longer * (len + 1);
        return s < head ? s / (len + 1) : longer + (s - head) / len;
    }
};

// A place in the order of stages: stage s of row (b, kvh), which has ns of them.
struct Cursor {
    int b, kvh, s, ns, ctx;
};

__device__ __forceinline__ int clamped_context(const DecodeParams &p, int b) {
    const int c = p.context_lens[b];
    return c < 0 ? 0 : min(c, p.context_limit);
}

// pre[b]: stages of kTok tokens of one kv head before sequence b, b = 0..num_seqs (after the
// caller's next barrier). warp_sums: kThreads / 32 words. A whole CTA calls it.
template <int kThreads, int kTok>
__device__ __forceinline__ void count_stages(const DecodeParams &p, int *pre, int *warp_sums) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, B = p.num_seqs;
    const int per = (B + kThreads - 1) / kThreads, b0 = min(B, tid * per), b1 = min(B, b0 + per);
    int sum = 0;
    for (int b = b0; b < b1; ++b) {
        const int raw = p.context_lens[b];
        if ((raw < 0 || raw > p.context_limit) && blockIdx.x == 0) raise_error(p.err, PA_DEVERR_CONTEXT);
        sum += (clamped_context(p, b) + kTok - 1) / kTok;
    }
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
    }
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    int at = inc - sum;
    for (int w = 0; w < warp; ++w) at += warp_sums[w];
    for (int b = b0; b < b1; ++b) {
        pre[b] = at;
        at += (clamped_context(p, b) + kTok - 1) / kTok;
    }
    if (b1 == B && (b0 < B || tid == 0)) pre[B] = at;
}

// What the joining kernel needs of every row: its first partial and how many there are
// (0: the row is written by its run). A run's partial of a row is number run + row: both rise
// along the order, so the numbers are distinct and a row's are consecutive.
template <int kThreads>
__device__ __forceinline__ void describe_rows(const DecodeParams &p, int2 *rows, const int *pre, const Runs &runs) {
    const int Hk = p.num_kv_heads;
    for (int r = blockIdx.x * kThreads + threadIdx.x; r < p.num_seqs * Hk; r += gridDim.x * kThreads) {
        const int b = r / Hk, h = r - b * Hk, ns = pre[b + 1] - pre[b];
        int2 info = make_int2(0, 0);
        if (ns > 0) {
            const uint32_t s0 = (uint32_t)pre[b] * Hk + (uint32_t)h * ns;
            const int w0 = (int)runs.owner(s0), w1 = (int)runs.owner(s0 + ns - 1);
            if (w1 > w0) info = make_int2(w0 + r, w1 - w0 + 1);
        }
        rows[r] = info;
    }
}

// Output rows of empty contexts.
template <typename T, int D, int kThreads>
__device__ __forceinline__ void zero_empty_rows(const DecodeParams &p, const int *pre) {
    T *out = reinterpret_cast<T *>(p.out);
    for (int b = blockIdx.x; b < p.num_seqs; b += gridDim.x)
        if (pre[b + 1] == pre[b])
            for (int i = threadIdx.x; i < p.num_heads * D; i += kThreads)
                out[(int64_t)b * p.num_heads * D + i] = Elem<T>::from_f(0.f);
}

// Joins the partials of the rows that several runs share: M = max m_i, L = sum l_i
// 2^(m_i - M), out = sum o_i 2^(m_i - M) / L. Warps per (query head, sequence), WPR: one where a
// row has few partials, 4, 16 or 32 (joined through shared memory) where it has many. A warp reads
// 32 partials' pairs at once, one a lane, and then their outputs, kJoinBatch in flight.
constexpr int kJoinWarps(int wpr) { return wpr < 4 ? 4 : wpr; }      // of a CTA
constexpr int kJoinBatch = 8;

template <typename T, int D, int WPR, int kWarps = kJoinWarps(WPR)>
__global__ __launch_bounds__(kWarps * 32) void decode_join_kernel(const DecodeParams p, const RunWork ws) {
    constexpr int N = D / 32;                          // channels of a lane
    __shared__ float2 ml_s[kWarps];
    __shared__ float o_s[WPR > 1 ? kWarps : 1][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = warp % WPR;
    const int64_t head = (int64_t)blockIdx.x * (kWarps / WPR) + warp / WPR;   // (sequence, query head)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // after the wait: the accumulation of the weights relies on the decode having finished
    asm volatile("griddepcontrol.launch_dependents;");
    if (head >= (int64_t)p.num_seqs * p.num_heads) return;   // with WPR > 1, the whole CTA
    const int G = p.group;
    const int64_t row = head / G;
    const int g = (int)(head - row * G);
    const int2 info = ws.rows[row];
    if (info.y == 0) return;                           // likewise
    const float2 *ml = ws.part_ml + (int64_t)info.x * G + g;
    const float *o = ws.part_o + ((int64_t)info.x * G + g) * D + lane * N;
    float m = -INFINITY, l = 0.f, acc[N];
#pragma unroll
    for (int u = 0; u < N; ++u) acc[u] = 0.f;
    for (int i0 = sub; i0 < info.y; i0 += 32 * WPR) {
        const int n = min(32, (info.y - i0 + WPR - 1) / WPR);   // this warp's partials of the round
        float x[kJoinBatch][N];
        auto load = [&](int k0) {
#pragma unroll
            for (int k = 0; k < kJoinBatch; ++k) {
                if (k0 + k < n) {
                    const float *src = o + (int64_t)(i0 + (k0 + k) * WPR) * G * D;
                    if constexpr (N == 4) *reinterpret_cast<float4 *>(x[k]) = *reinterpret_cast<const float4 *>(src);
                    else *reinterpret_cast<float2 *>(x[k]) = *reinterpret_cast<const float2 *>(src);
                }
            }
        };
        const int i = i0 + lane * WPR;
        const float2 mine = i < info.y ? ml[(int64_t)i * G] : make_float2(-INFINITY, 0.f);
        load(0);                                       // in flight with the pairs
        float mb = mine.x;
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, k));
        mb = fmaxf(mb, m);
        const float a = m == -INFINITY ? 0.f : fast_exp2(m - mb);
        l *= a;
#pragma unroll
        for (int u = 0; u < N; ++u) acc[u] *= a;
        m = mb;
        // a partial whose scores are all NaN has no reference and a NaN sum: keep the NaN
        const float c = mine.x == -INFINITY ? (mine.y == mine.y ? 0.f : mine.y) : fast_exp2(mine.x - mb);
        float lc = mine.y * c;
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) lc += __shfl_xor_sync(0xffffffffu, lc, k);
        l += lc;
        for (int k0 = 0; k0 < n; k0 += kJoinBatch) {
            if (k0 > 0) load(k0);
#pragma unroll
            for (int k = 0; k < kJoinBatch; ++k) {
                if (k0 + k < n) {
                    const float ck = __shfl_sync(0xffffffffu, c, k0 + k);
#pragma unroll
                    for (int u = 0; u < N; ++u) acc[u] = fmaf(x[k][u], ck, acc[u]);
                }
            }
        }
    }
    if constexpr (WPR > 1) {
        if (lane == 0) ml_s[warp] = make_float2(m, l);
#pragma unroll
        for (int u = 0; u < N; ++u) o_s[warp][lane * N + u] = acc[u];
        __syncthreads();
        if (warp != 0) return;
        float M = -INFINITY;
        l = 0.f;
#pragma unroll
        for (int u = 0; u < N; ++u) acc[u] = 0.f;
#pragma unroll
        for (int w = 0; w < WPR; ++w) M = fmaxf(M, ml_s[w].x);
#pragma unroll
        for (int w = 0; w < WPR; ++w) {
            const float2 v = ml_s[w];
            const float f = v.x == -INFINITY ? (v.y == v.y ? 0.f : v.y) : fast_exp2(v.x - M);
            l = fmaf(v.y, f, l);
#pragma unroll
            for (int u = 0; u < N; ++u) acc[u] = fmaf(o_s[w][lane * N + u], f, acc[u]);
        }
    }
    const float inv = 1.f / l;
    alignas(8) T h[N];
#pragma unroll
    for (int u = 0; u < N; ++u) h[u] = Elem<T>::from_f(acc[u] * inv);
    T *dst = reinterpret_cast<T *>(p.out) + head * D + lane * N;
    if constexpr (N == 4) *reinterpret_cast<uint2 *>(dst) = *reinterpret_cast<uint2 *>(h);
    else *reinterpret_cast<uint32_t *>(dst) = *reinterpret_cast<uint32_t *>(h);
}

// The join after a kernel of `warps` warps and stages of `tok` tokens; kMost: warps of a row that has many partials.
template <typename T, int D, int kMost = 16>
int launch_join(const DecodeParams &p, const RunWork &ws, int64_t max_ctx, int tok, int64_t warps, cudaStream_t stream) {
    // Partials a row: about runs / rows, for contexts of the limit's length. (8 kv heads, us with up to
    // 4 warps a row and with 16: one context of 16,000 tokens 21.2 and 13.2, of 131,072 44.9 and 35.9,
    // three of 40,000 to 120,000 60.0 and 55.4; with 11 partials a row, 16 warps are 0.15 slower.)
    // The limit is that of the call's arguments alone, before mass cuts p.context_limit: the warps
    // decide the order of the sums, and out does not depend on whether weights are accumulated.
    const int64_t heads = (int64_t)p.num_seqs * p.num_heads, rows = (int64_t)p.num_seqs * p.num_kv_heads;
    const int64_t limit = std::min(max_ctx, (int64_t)p.max_blocks_per_seq * p.block_size);
    const int64_t stages = (limit + tok - 1) / tok;
    const int64_t runs = std::min<int64_t>(warps, rows * stages);
    const int wpr = runs <= 8 * rows ? 1 : (runs <= 32 * rows ? 4 : kMost), cta = kJoinWarps(wpr);
    auto join = wpr == 1   ? decode_join_kernel<T, D, 1>
                : wpr == 4 ? decode_join_kernel<T, D, 4>
                           : decode_join_kernel<T, D, kMost>;
    return launch_pdl(join, dim3((unsigned)((heads * wpr + cta - 1) / cta)), dim3(cta * 32), 0, stream, p, ws);
}

}  // namespace
}  // namespace pa
