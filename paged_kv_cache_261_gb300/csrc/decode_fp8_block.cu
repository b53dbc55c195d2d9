// Decode attention over an 8-bit paged cache that has a scale for each block of tokens and kv
// head (format: kv_fp8_block.cu).
//
// What is computed is the decode attention of "CS349E lecture 7: 01_paged_attention.py",
// demo 2, paper eq. 4 (block-wise scores through the block table, one softmax over the whole
// context, block-wise V accumulation) over the cache's values, K = code * k_scale and
// V = code * v_scale with the scales of the token's block:
//   q . K_t          = k_scale_t (q . n_t)
//   sum_t p_t V_t[c] = sum_t (p_t v_scale_t) n_t[c]
//
// E4M3 codes are exact in f16, so a pair of codes becomes a pair of matrix operands by one
// conversion. Per 16 tokens a warp multiplies, with mma.m16n8k16 (f16 operands, f32 sums),
//   S^T[16 tok x 8 heads] = n_K[16 x D] . Q^T        A = codes, row = token
//   O^T[D x 8 heads]     += n_V^T[D x 16 tok] . W^T   A = codes, row = channel
// The order of the channels inside a contraction, and of the output's rows over the
// instructions, is free; it is chosen so that every lane's codes are consecutive bytes
// of a row (D / 4 for K, D / 8 for V). S^T's fragments turn into W^T's with one 8x8
// transpose in registers. (An instruction of E4M3 operands would want query and weights as
// sums of three E4M3 terms to keep the 11 bits that f16 has.)
//
// W = p v_scale enters the product as two f16, its rounding and what that left (22 bits; the row sums
// take p unrounded): as one (11 bits) the weights' rounding reached the outputs, 4 to 9 % of the bf16 ones
// rounded to a neighbour of what float32 weights give (us with one and two, bf16: 8B-shaped batch 53.8, 54.2, long contexts
// 202.6, 202.8, one sequence of 700 tokens 5.1, 5.35, 16 query heads to a kv head 63.9, 70.4). Its reference is a
// maximum of the scores (raised only when a score exceeds it by 2^7: no reduction over the lanes before) and a
// power of two above every v_scale seen, so the terms are normal f16 numbers down to 2^-22 of the reference times that
// power and within 2^-33 of it below. The query enters as f16 times a power of two per head: exact for
// bf16 and f16 at every channel within 2^-22 of the row's largest.
//
// Work: the stages (kTok tokens of one sequence and kv head) of the whole call, in order, are
// cut into equal runs, one for each warp of the persistent grid (decode_runs.cuh). Warps share
// nothing. Few rows of short contexts are too little work to cut so: there one to sixteen CTAs, a
// cluster, take each row, its stages dealt to their warps in equal parts, and join the parts
// through each other's shared memory, without a second kernel (row_cluster). Each warp fetches its own
// stages, one ahead and across rows, into its own ring: a block of one kv head is one contiguous run for K and V each, so a stage is a few untiled bulk
// copies, and its blocks' scales one 8-byte copy each, all on one mbarrier. (Boxes that TMA
// swizzles, so that the lanes of a fragment do not meet on few banks, changed nothing: 52.9 and
// 201.7 us on the two cases below.)
//
// What bounds it (one GB300): HBM. Long contexts, 1.34 GB, take 202 us, 6.65 TB/s, as fast as a copy;
// the 8B-shaped batch, 303 MB, 54.2 us, 3 of them the join and about 3 the start. 8 warps with two
// stages of 8 KB each keep 131 KB an SM on their way; more of them is slower, as is less work a
// stage (us with weights as one f16, batch / long, of which 53.3 / 201.5 with two stages of 8 warps: 10 warps 53.0 / 214, 12 54.9 / 216, 8 with three stages 55.0 / 217, 12 with
// three of 4 KB 53.2 / 205, 8 with three of 4 KB 61.7 / 241). 16 query heads to a kv head: 70.4 us on the batch, instructions.
//
// Every wait is bounded; on a timeout the kernel sets PA_DEVERR_WAIT, waits (bounded)
// for its copies in flight and returns.
#include "decode_runs.cuh"
#include "kernels_fp8_block.h"

#include <atomic>
#include <mutex>
#include <type_traits>

namespace pa {
namespace {

constexpr int kStages = 2;
constexpr int kMaxSeqs = 1536;                    // sequences per launch (the host splits larger batches)

// The softmax reference of a head is not raised before a score exceeds it by this many
// powers of two: the weights (f16, up to 2^kWeightExp times 2^kSlack) have the room.
constexpr float kSlack = 7.f;
constexpr int kWeightExp = 8;
constexpr int kMinScaleExp = -100, kMaxScaleExp = 121;   // of the V scales' reference

__host__ __device__ constexpr int stage_tokens(int D) { return 4096 / D; }
constexpr int kWarps = 8;                         // of a CTA, one CTA an SM
constexpr int kClusterSizes = 5;                  // 1, 2, ..., 16 CTAs of a row, where CTAs take rows
constexpr int kRowStages = 7;                     // of a warp, then, at most

template <int D> struct Cfg {
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kTok = stage_tokens(D);              // tokens per stage
    static constexpr int kRow = D;                            // bytes of a token's codes
    static constexpr int kPieces = kTok / 8;                  // blocks per stage, at most
    static constexpr int kOffV = kTok * kRow;
    static constexpr int kOffScale = 2 * kTok * kRow;
    static constexpr int kSlot = kOffScale + kPieces * 8;
    static constexpr int kRing = kWarps * kStages * kSlot;
    // after the ring
    static constexpr int kOffBar = kRing;                             // [kWarps][kStages]
    static constexpr int kOffMisc = kOffBar + kWarps * kStages * 8;   // abort flag; warp sums of the prefix
    static constexpr int kOffPre = kOffMisc + 16 + kWarps * 4;        // int [kMaxSeqs + 1]
    static constexpr int kSmem = kOffPre + (kMaxSeqs + 1) * 4;
    // where CTAs take rows, then: partials float [kWarps + 1][GT][D], the last of them the CTA's, and their
    // float2 (reference, sum) [kWarps + 1][GT]
    static constexpr int kOffPart = (kSmem + 15) / 16 * 16;
    static constexpr int part_bytes(int GT) { return (kWarps + 1) * GT * (D * 4 + 8); }
    static_assert(kOffPart + part_bytes(16) <= 232448, "shared memory budget");
    static_assert(kSlot % 16 == 0 && kOffV % 16 == 0 && kOffScale % 16 == 0, "bulk copies start on 16 bytes");
    static_assert(kPieces <= 8, "a lane per piece");
};

// Two codes, in 16 bits, as two f16.
__device__ __forceinline__ uint32_t widen(uint32_t two) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(two));
    return r;
}
__device__ __forceinline__ uint32_t widen_high(uint32_t two) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(r) : "r"(two));
    return r;
}
// 8 bytes copied asynchronously.
__device__ __forceinline__ void copy8_async(void *dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
// An arrival once this thread's asynchronous copies have landed (one of the phase's count).
__device__ __forceinline__ void arrive_after_copies(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t n;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
    return n;
}
__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Where CTA `rank` of the cluster has what this CTA has at p, and what is there.
__device__ __forceinline__ uint32_t peer_addr(const void *p, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ float2 load_peer2(uint32_t a) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float4 load_peer4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}
// Adds a partial (its reference and sum, its outputs) to a joined one whose reference is M.
__device__ __forceinline__ void join_partial(float M, float2 ml, float4 o, float &L, float4 &acc) {
    // a partial whose scores are all NaN has no reference and a NaN sum: keep the NaN
    const float c = ml.x == -INFINITY ? (ml.y == ml.y ? 0.f : ml.y) : fast_exp2(ml.x - M);
    L = fmaf(ml.y, c, L);
    acc.x = fmaf(o.x, c, acc.x);
    acc.y = fmaf(o.y, c, acc.y);
    acc.z = fmaf(o.z, c, acc.z);
    acc.w = fmaf(o.w, c, acc.w);
}

// GT: query heads padded to 8 or 16. kRowCta: a cluster of CTAs takes a row, its warps equal parts of it.
template <typename T, int D, int GT, bool kRowCta>
__global__ __launch_bounds__(Cfg<D>::kThreads, 1) void decode_fp8_block_kernel(const DecodeParams p,
                                                                                     const RunWork ws) {
    using C = Cfg<D>;
    constexpr int kThreads = C::kThreads;
    constexpr int NT = GT / 8;                         // tiles of 8 heads
    constexpr int kSteps = D / 16;                     // instructions per 16 tokens, S and O alike
    constexpr int kSub = C::kTok / 16;
    extern __shared__ __align__(128) unsigned char smem[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kOffBar);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::kOffMisc);
    int *warp_sums = reinterpret_cast<int *>(smem + C::kOffMisc + 16);
    int *pre = reinterpret_cast<int *>(smem + C::kOffPre);   // stages of a kv head before sequence b
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int li = lane >> 2, lj = lane & 3;           // fragment row and column group
    const int G = p.group, B = p.num_seqs, Hk = p.num_kv_heads;

    if (tid == 0) {
        // a phase: the bytes of the bulk copies, and the lanes that copy scales
        for (int i = 0; i < kWarps * kStages; ++i) mbar_init(&bars[i], 1 + C::kPieces);
        *abort_flag = 0;
        mbar_fence_init();
    }
    // as the other decode kernels: the set-up and the cut of the work (which reads only the
    // call's lengths) overlap the preceding kernel
    asm volatile("griddepcontrol.launch_dependents;");
    auto context = [&](int b) { return clamped_context(p, b); };
    float *parts = reinterpret_cast<float *>(smem + C::kOffPart);                  // [kWarps + 1][G][D]
    float2 *part_ml = reinterpret_cast<float2 *>(parts + (kWarps + 1) * GT * D);   // [kWarps + 1][G]
    int todo = 0;
    Cursor at = {};
    [[maybe_unused]] uint32_t run = 0, total = 0, num_runs = 1;
    if constexpr (kRowCta) {
        const int row = blockIdx.x / cluster_size(), warps = cluster_size() * kWarps;
        at.b = row / Hk;
        at.kvh = row - at.b * Hk;
        at.ctx = context(at.b);
        at.ns = (at.ctx + C::kTok - 1) / C::kTok;
        const int per = (at.ns + warps - 1) / warps;
        at.s = min(at.ns, (int)(cluster_rank() * kWarps + warp) * per);
        todo = min(at.ns, at.s + per) - at.s;
        if (tid == 0 && at.kvh == 0 && cluster_rank() == 0 && at.ctx != p.context_lens[at.b])
            raise_error(p.err, PA_DEVERR_CONTEXT);
        // a warp without stages leaves a partial of nothing
        for (int i = lane; i < G * D && todo == 0; i += 32) parts[warp * G * D + i] = 0.f;
        for (int g = lane; g < G; g += 32) part_ml[warp * G + g] = make_float2(-INFINITY, 0.f);
        __syncthreads();                               // the barriers stand
    } else {
        count_stages<kThreads, C::kTok>(p, pre, warp_sums);
        __syncthreads();
        total = (uint32_t)pre[B] * Hk;                 // below 2^31: the host sees to it
        num_runs = max(1u, min(gridDim.x * kWarps, total));
    }
    const Runs runs(total, num_runs);
    // runs go to the SMs in turn, so few of them still use all
    if constexpr (!kRowCta) run = warp * gridDim.x + blockIdx.x;
    if (!kRowCta && run < num_runs && total > 0) {
        const uint32_t run0 = runs.first(run);
        todo = (int)(runs.len + (run < runs.longer ? 1 : 0));
        int lo = 0, hi = B - 1;                        // the first b whose stages end after run0
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if ((uint32_t)pre[mid + 1] * Hk > run0) hi = mid; else lo = mid + 1;
        }
        at.b = lo;
        at.ns = pre[lo + 1] - pre[lo];
        const uint32_t rest = run0 - (uint32_t)pre[lo] * Hk;
        at.kvh = (int)(rest / (uint32_t)at.ns);
        at.s = (int)(rest - (uint32_t)at.kvh * at.ns);
        at.ctx = context(lo);
    }
    // the next row that has stages (there is one)
    auto next_row = [&](Cursor &c) {
        if constexpr (kRowCta) return;                 // there is none
        c.s = 0;
        if (++c.kvh < Hk) return;
        c.kvh = 0;
        do ++c.b; while (pre[c.b + 1] == pre[c.b]);
        c.ns = pre[c.b + 1] - pre[c.b];
        c.ctx = context(c.b);
    };

    // ---- fetching: lanes 0-7 the K runs, 8-15 the V runs, 16-23 the scales of a stage's
    // blocks (at most 8: block_size >= 8)
    unsigned char *ring = smem + warp * kStages * C::kSlot;
    uint64_t *full = bars + warp * kStages;
    const int kind = lane >> 3;
    const int piece_tok = min(p.block_size, C::kTok), log2_piece = 31 - __clz(piece_tok);
    const int piece_off = (lane & 7) * piece_tok;      // the piece's first token of the stage
    const bool fetches = kind < 3 && piece_off < C::kTok;
    const unsigned char *src_base = static_cast<const unsigned char *>(
        kind == 2 ? p.kv_params : (kind == 1 ? p.value_cache : p.key_cache));
    const uint32_t dst_off = kind == 2 ? C::kOffScale + (lane & 7) * 8 : (kind == 1 ? C::kOffV : 0) + piece_off * C::kRow;
    const uint32_t piece_bytes = kind == 2 ? 8 : piece_tok * C::kRow;
    const uint32_t run_bytes = (uint32_t)C::kRow << p.log2_block_size;     // a block's rows of one kv head
    const uint32_t block_bytes = run_bytes * (uint32_t)Hk;                 // at most 2^16 * 2^8 * 128, less 2^15

    // whether this lane has a piece of the stage to fetch, and its table entry
    auto has_piece = [&](const Cursor &c) { return fetches && c.s * C::kTok + piece_off < c.ctx; };
    auto look_up = [&](const Cursor &c) {
        const int t = c.s * C::kTok + piece_off;
        return has_piece(c) ? p.block_tables[(int64_t)c.b * p.max_blocks_per_seq + (t >> p.log2_block_size)] : -1;
    };
    auto step = [&](Cursor &c) {
        if (++c.s == c.ns) next_row(c);
    };
    // fetch a stage into a slot of the ring (which no lane reads any more)
    auto fetch = [&](const Cursor &nx, int entry, int sl) {
        unsigned char *dst = ring + sl * C::kSlot + dst_off;
        uint64_t *bar = &full[sl];
        const bool live = has_piece(nx), good = live && entry >= 0 && entry < p.num_blocks;
        const uint32_t blocks = __popc(__ballot_sync(0xffffffffu, good) & 0xFFu);
        if (lane == 0) mbar_arrive_expect_tx(bar, blocks * piece_tok * (2 * C::kRow));
        __syncwarp();
        if (good) {
            if (kind == 2) {
                copy8_async(dst, src_base + ((int64_t)entry * Hk + nx.kvh) * 8);
            } else {
                const uint32_t off = (uint32_t)nx.kvh * run_bytes +
                                     (uint32_t)((nx.s * C::kTok + piece_off) & (p.block_size - 1)) * C::kRow;
                bulk_load(dst, src_base + ((uint64_t)(uint32_t)entry * block_bytes + off), piece_bytes, bar);
            }
        } else if (live) {
            // a bad block id: zeros, so its tokens have score and value 0
            if (kind == 0) raise_error(p.err, PA_DEVERR_BLOCK_ID);
            for (uint32_t i = 0; i < piece_bytes; i += 8) *reinterpret_cast<uint2 *>(dst + i) = make_uint2(0, 0);
            fence_proxy_async_smem();
        }
        if (kind == 2 && (lane & 7) < C::kPieces) arrive_after_copies(bar);
        __syncwarp();
    };
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // the first stages, their look-ups in flight together; then one look-up ahead
    Cursor nx = at;
    int entry = -1;
    if (todo > 0) {
        Cursor c[kStages];
        int e[kStages];
#pragma unroll
        for (int i = 0; i < kStages; ++i)
            if (i < todo) {
                c[i] = nx;
                e[i] = look_up(nx);
                if (i + 1 < todo) step(nx);
            }
#pragma unroll
        for (int i = 0; i < kStages; ++i)
            if (i < todo) fetch(c[i], e[i], i);
        entry = look_up(nx);
    }
    if constexpr (!kRowCta) {
        describe_rows<kThreads>(p, ws.rows, pre, runs);
        zero_empty_rows<T, D, kThreads>(p, pre);
        if (todo == 0) return;
    }
    int left = todo;                                   // stages to consume
    int unfetched = todo - min(todo, kStages);         // and to fetch
    int sl = 0;                                        // the slot of the next stage
    uint32_t phase = 0;                                // and its barrier's phase
    bool ok = true;

    T *out = reinterpret_cast<T *>(p.out);
    const T *q = reinterpret_cast<const T *>(p.q);
    while (left > 0) {
        // ---- the part of row (b, kvh) that lies in this run
        const int I_b = at.b, I_kvh = at.kvh;
        const int s_end = min(at.ns, at.s + left);
        const bool whole = !kRowCta && at.s == 0 && s_end == at.ns;
        const int64_t head0 = (int64_t)I_b * p.num_heads + (int64_t)I_kvh * G;

        // the group's query as B fragments, and the factors of x = S * (k_scale * sa) of the
        // heads of S^T's columns
        uint32_t qb[NT][kSteps][2];
        float2 sa[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            constexpr int N = D / 4;                   // channels of a lane
            const int g = nt * 8 + li;
            float x[N];
            const T *src = q + (head0 + min(g, G - 1)) * D + lj * N;
#pragma unroll
            for (int u = 0; u < N / 8; ++u) Vec16<T>::unpack(__ldg(reinterpret_cast<const uint4 *>(src) + u), x + 8 * u);
            float amax = 0.f;
#pragma unroll
            for (int u = 0; u < N; ++u) {
                if (g >= G) x[u] = 0.f;
                amax = fmaxf(amax, fabsf(x[u]));
            }
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            // amax = 1.f * 2^(E - 127), scaled into [2^12, 2^13)
            const int E = (int)((__float_as_uint(amax) >> 23) & 0xFF);
            const int e2 = E == 0 ? 100 : max(-116, min(100, 139 - E));
            const float up = pow2f(e2);
#pragma unroll
            for (int u = 0; u < kSteps; ++u) {
                qb[nt][u][0] = pack_half2(x[4 * u] * up, x[4 * u + 1] * up);
                qb[nt][u][1] = pack_half2(x[4 * u + 2] * up, x[4 * u + 3] * up);
            }
            const float a = p.scale_log2 * pow2f(-e2);
            sa[nt] = make_float2(__shfl_sync(0xffffffffu, a, 8 * lj), __shfl_sync(0xffffffffu, a, 8 * lj + 4));
        }
        float O[NT][kSteps][4];
        float2 nm[NT], l[NT];                          // nm: the negated references
        int r_exp = kMinScaleExp;                      // 2^r_exp = r_top > every v_scale seen
        float r_top = 0.f, cr = 0.f;                   // v_scale * cr < 2^kWeightExp
        bool first = true;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int u = 0; u < kSteps; ++u)
#pragma unroll
                for (int c = 0; c < 4; ++c) O[nt][u][c] = 0.f;
            nm[nt] = make_float2(INFINITY, INFINITY);
            l[nt] = make_float2(0.f, 0.f);
        }
        // one stage; kTail: only its first n tokens belong to the row
        auto stage = [&](auto tail, const unsigned char *slot, int n) {
            constexpr bool kTail = decltype(tail)::value;
            // ---- scores, S^T: rows li and li + 8 of each 16 tokens
            float S[kSub][NT][4];
            float vs[kSub][2];
            float rmax = 0.f;
#pragma unroll
            for (int sub = 0; sub < kSub; ++sub) {
                float S2[NT][4];                       // a second chain of sums
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 4; ++c) S[sub][nt][c] = S2[nt][c] = 0.f;
                uint32_t ka[D / 16], kb[D / 16];       // this lane's words of the two rows
                const unsigned char *kr = slot + (sub * 16 + li) * C::kRow + lj * (D / 4);
#pragma unroll
                for (int w = 0; w < D / 64; ++w) {
                    reinterpret_cast<uint4 *>(ka)[w] = reinterpret_cast<const uint4 *>(kr)[w];
                    reinterpret_cast<uint4 *>(kb)[w] = reinterpret_cast<const uint4 *>(kr + 8 * C::kRow)[w];
                }
#pragma unroll
                for (int u = 0; u < kSteps; ++u) {
                    const uint32_t a0 = widen(ka[u]), a1 = widen(kb[u]), a2 = widen_high(ka[u]), a3 = widen_high(kb[u]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma16816(u & 1 ? S2[nt] : S[sub][nt], a0, a1, a2, a3, qb[nt][u][0], qb[nt][u][1]);
                }
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int t = sub * 16 + li + 8 * r;
                    const float2 sc = *reinterpret_cast<const float2 *>(slot + C::kOffScale + (t >> log2_piece) * 8);
                    const bool valid = !kTail || t < n;
                    vs[sub][r] = valid ? sc.y : 0.f;
                    rmax = fmaxf(rmax, fabsf(vs[sub][r]));
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const float2 dot = add2(make_float2(S[sub][nt][2 * r], S[sub][nt][2 * r + 1]),
                                                make_float2(S2[nt][2 * r], S2[nt][2 * r + 1]));
                        const float2 x = mul2(dot, make_float2(sc.x * sa[nt].x, sc.x * sa[nt].y));
                        S[sub][nt][2 * r] = valid ? x.x : -INFINITY;
                        S[sub][nt][2 * r + 1] = valid ? x.y : -INFINITY;
                    }
                }
            }
            // ---- this lane's V words of every 16 tokens (2 lj, 2 lj + 1, 2 lj + 8, 2 lj + 9), read
            // before the references are looked at
            uint32_t vw[kSub][4][D / 32];
#pragma unroll
            for (int sub = 0; sub < kSub; ++sub) {
                const unsigned char *vr = slot + C::kOffV + (sub * 16 + 2 * lj) * C::kRow + li * (D / 8);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int t = (k & 1) + (k & 2) * 4;
                    const unsigned char *src = vr + t * C::kRow;
                    if constexpr (D == 128) *reinterpret_cast<uint4 *>(vw[sub][k]) = *reinterpret_cast<const uint4 *>(src);
                    else *reinterpret_cast<uint2 *>(vw[sub][k]) = *reinterpret_cast<const uint2 *>(src);
                    // past the row's end anything may lie, NaN codes too
                    if (kTail && sub * 16 + 2 * lj + t >= n) {
#pragma unroll
                        for (int w = 0; w < D / 32; ++w) vw[sub][k][w] = 0;
                    }
                }
            }
            // ---- the references, raised where a score or a V scale outgrew them
            float over = -INFINITY;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float v = S[0][nt][c];
#pragma unroll
                    for (int sub = 0; sub < kSub; ++sub) v = fmaxf(v, fmaxf(S[sub][nt][c], S[sub][nt][2 + c]));
                    over = fmaxf(over, v + (c ? nm[nt].y : nm[nt].x));
                }
            if (__any_sync(0xffffffffu, first || over > kSlack || rmax >= r_top)) {
                const int r_new = max(r_exp, min(kMaxScaleExp, (int)((__float_as_uint(rows_max(rmax)) >> 23) & 0xFF) - 126));
                const float rs = r_exp - r_new < -126 ? 0.f : pow2f(r_exp - r_new);
                r_exp = r_new;
                r_top = pow2f(r_new);
                cr = pow2f(kWeightExp - r_new);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float a[2];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float &neg = c ? nm[nt].y : nm[nt].x;
                        float v = -neg;
#pragma unroll
                        for (int sub = 0; sub < kSub; ++sub) v = fmaxf(v, fmaxf(S[sub][nt][c], S[sub][nt][2 + c]));
                        v = rows_max(v);
                        a[c] = first ? 0.f : fast_exp2(-neg - v);
                        neg = -v;
                    }
                    if (!first) {
                        l[nt] = mul2(l[nt], make_float2(a[0], a[1]));
#pragma unroll
                        for (int u = 0; u < kSteps; ++u)
#pragma unroll
                            for (int c = 0; c < 4; ++c) O[nt][u][c] *= a[c & 1] * rs;
                    }
                }
                first = false;
            }
            // ---- weights and O^T
#pragma unroll
            for (int sub = 0; sub < kSub; ++sub) {
                uint32_t wb[NT][2], we[NT][2];         // W as f16, and what that rounding left
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const float2 d = add2(make_float2(S[sub][nt][2 * r], S[sub][nt][2 * r + 1]), nm[nt]);
                        const float2 w = make_float2(fast_exp2(d.x), fast_exp2(d.y));
                        l[nt] = add2(l[nt], w);
                        const float v = vs[sub][r] * cr;
                        const float2 wv = mul2(w, make_float2(v, v));
                        const uint32_t wh = pack_half2(wv.x, wv.y);
                        wb[nt][r] = transpose8x8(wh);
                        const float2 hi = __half22float2(*reinterpret_cast<const __half2 *>(&wh));
                        const float2 lo = add2(wv, make_float2(-hi.x, -hi.y));
                        we[nt][r] = transpose8x8(pack_half2(lo.x, lo.y));
                    }
                // two tokens' bytes of two channels side by side
#pragma unroll
                for (int u = 0; u < kSteps; ++u) {
                    const uint32_t sel = u & 1 ? 0x7362u : 0x5140u;
                    const uint32_t x = __byte_perm(vw[sub][0][u / 2], vw[sub][1][u / 2], sel);
                    const uint32_t y = __byte_perm(vw[sub][2][u / 2], vw[sub][3][u / 2], sel);
                    const uint32_t a0 = widen(x), a1 = widen_high(x), a2 = widen(y), a3 = widen_high(y);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma16816(O[nt][u], a0, a1, a2, a3, wb[nt][0], wb[nt][1]);
                        mma16816(O[nt][u], a0, a1, a2, a3, we[nt][0], we[nt][1]);
                    }
                }
            }
        };
        for (; at.s < s_end; ++at.s) {
            const unsigned char *slot = ring + sl * C::kSlot;
            if (!__all_sync(0xffffffffu, mbar_try_wait(&full[sl], phase)) &&
                (__any_sync(0xffffffffu, *abort_flag != 0) || !warp_wait(&full[sl], phase))) {
                ok = false;
                break;
            }
            const int n = at.ctx - at.s * C::kTok;     // valid tokens, at least 1
            if (n >= C::kTok) stage(std::false_type{}, slot, n);
            else stage(std::true_type{}, slot, n);
            __syncwarp();                              // every lane has read the slot
            --left;
            if (unfetched > 0) {
                fetch(nx, entry, sl);
                if (--unfetched > 0) {
                    step(nx);
                    entry = look_up(nx);               // on its way until the next fetch
                }
            }
            if (++sl == kStages) {
                sl = 0;
                phase ^= 1;
            }
        }
        if (!ok) break;

        // ---- the row, or this run's partial of it (unnormalised, with its reference and sum).
        // A lane has channels li D / 8 + 2 u + r of heads 2 lj and 2 lj + 1.
        const int r = I_b * Hk + I_kvh;
        const float unit = pow2f(r_exp - kWeightExp);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float ls = rows_sum(c ? l[nt].y : l[nt].x);
                const int g = nt * 8 + 2 * lj + c;
                if (g >= G) continue;
                const float inv = whole ? 1.f / ls : 1.f;
                const int d0 = li * (D / 8);
#pragma unroll
                for (int u0 = 0; u0 < kSteps; u0 += 4) {
                    float v[8];
#pragma unroll
                    for (int u = 0; u < 4; ++u)
#pragma unroll
                        for (int rr = 0; rr < 2; ++rr) v[2 * u + rr] = O[nt][u0 + u][2 * rr + c] * inv * unit;
                    if (whole) {
                        alignas(16) T h[8];
#pragma unroll
                        for (int u = 0; u < 8; ++u) h[u] = Elem<T>::from_f(v[u]);
                        *reinterpret_cast<uint4 *>(out + (head0 + g) * D + d0 + 2 * u0) = *reinterpret_cast<uint4 *>(h);
                    } else {
                        float *dst = (kRowCta ? parts + (warp * G + g) * D
                                              : ws.part_o + ((int64_t)(run + r) * G + g) * D) + d0 + 2 * u0;
                        *reinterpret_cast<float4 *>(dst) = make_float4(v[0], v[1], v[2], v[3]);
                        *reinterpret_cast<float4 *>(dst + 4) = make_float4(v[4], v[5], v[6], v[7]);
                    }
                }
                if (li == 0 && !whole)
                    (kRowCta ? part_ml[warp * G + g] : ws.part_ml[(int64_t)(run + r) * G + g]) =
                        make_float2(-(c ? nm[nt].y : nm[nt].x), ls);
            }
        if (left > 0) next_row(at);
    }
    if (!ok) {
        *abort_flag = 1;
        raise_error(p.err, PA_DEVERR_WAIT);
        // copies still in flight land before the CTA's shared memory goes away
        for (; left > unfetched; --left) {
            mbar_wait(&full[sl], phase);
            if (++sl == kStages) {
                sl = 0;
                phase ^= 1;
            }
        }
    }
    if constexpr (kRowCta) {
        // The warps' partials joined into the CTA's, and the CTAs' into the row, each CTA taking a part of it.
        __syncthreads();
        const int C4 = D / 4;
        for (int i = tid; i < G * C4; i += kThreads) {
            const int g = i / C4, d = (i - g * C4) * 4;
            float M = -INFINITY, L = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, part_ml[w * G + g].x);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                join_partial(M, part_ml[w * G + g], *reinterpret_cast<const float4 *>(parts + (w * G + g) * D + d), L, acc);
            *reinterpret_cast<float4 *>(parts + (kWarps * G + g) * D + d) = acc;
            if (d == 0) part_ml[kWarps * G + g] = make_float2(M, L);
        }
        cluster_sync();
        const int n = (int)cluster_size();
        const int64_t head0 = (int64_t)at.b * p.num_heads + (int64_t)at.kvh * G;
        for (int i = (int)cluster_rank() * kThreads + tid; i < G * C4; i += n * kThreads) {
            const int g = i / C4, d = (i - g * C4) * 4;
            float M = -INFINITY, L = 0.f;
            for (int r = 0; r < n; ++r) M = fmaxf(M, load_peer2(peer_addr(part_ml + kWarps * G + g, r)).x);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int r = 0; r < n; ++r)
                join_partial(M, load_peer2(peer_addr(part_ml + kWarps * G + g, r)),
                             load_peer4(peer_addr(parts + (kWarps * G + g) * D + d, r)), L, acc);
            const float inv = at.ctx > 0 ? 1.f / L : 0.f;          // an empty context: zeros
            alignas(8) T h[4] = {Elem<T>::from_f(acc.x * inv), Elem<T>::from_f(acc.y * inv), Elem<T>::from_f(acc.z * inv),
                                 Elem<T>::from_f(acc.w * inv)};
            *reinterpret_cast<uint2 *>(out + (head0 + g) * D + d) = *reinterpret_cast<uint2 *>(h);
        }
        cluster_sync();                                // no CTA leaves while another reads its memory
    }
}

// One CTA per SM, and no more than there can be stages.
int launch_grid(int64_t rows, int64_t stages, int sms) {
    return (int)std::max<int64_t>(1, std::min<int64_t>(sms, rows * stages));
}

template <typename T, int D, int GT>
int launch_runs(const DecodeParams &p, const RunWork &ws, int64_t max_ctx, int grid, cudaStream_t stream) {
    using C = Cfg<D>;
    auto kern = decode_fp8_block_kernel<T, D, GT, false>;
    static bool attr_set[kMaxDevices] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return -1;
    if (!attr_set[dev]) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess) return -1;
        attr_set[dev] = true;
    }
    const int rc = launch_pdl(kern, dim3((unsigned)grid), dim3(C::kThreads), C::kSmem, stream, p, ws);
    // (32 warps a row of many partials rather than 16, us: one context of 32,000 tokens of one kv head 15.3 and 11.8, of
    // two 14.0 and 11.7, 131,000 of one 21.5 and 16.9, 16,000 of eight 12.1 and 11.9)
    return rc != 0 ? rc : launch_join<T, D, 32>(p, ws, max_ctx, C::kTok, (int64_t)grid * kWarps, stream);
}

// CTAs that take rows, `cluster` to a row.
template <typename T, int D, int GT> struct RowCtas {
    static constexpr int kSmem = Cfg<D>::kOffPart + Cfg<D>::part_bytes(GT);
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = {};
    RowCtas(int64_t rows, int cluster, cudaStream_t stream) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = (unsigned)cluster;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.gridDim = dim3((unsigned)(rows * cluster));
        cfg.blockDim = dim3(Cfg<D>::kThreads);
        cfg.dynamicSmemBytes = kSmem;
        cfg.stream = stream;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
    }
    RowCtas(const RowCtas &) = delete;

    // How many clusters of 2^i CTAs the device holds at once (asked for once); null on an error.
    static const int *room(int dev) {
        static std::atomic<bool> known[kMaxDevices];
        static std::mutex asking;
        static int n[kMaxDevices][kClusterSizes];
        if (known[dev].load(std::memory_order_acquire)) return n[dev];
        const std::lock_guard<std::mutex> lock(asking);
        if (known[dev].load(std::memory_order_relaxed)) return n[dev];
        auto kern = decode_fp8_block_kernel<T, D, GT, true>;
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess ||
            cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
            return nullptr;
        for (int i = 0; i < kClusterSizes; ++i) {
            RowCtas l(1, 1 << i, nullptr);
            if (cudaOccupancyMaxActiveClusters(&n[dev][i], kern, &l.cfg) != cudaSuccess) return nullptr;
        }
        known[dev].store(true, std::memory_order_release);
        return n[dev];
    }
};

// CTAs of a row where CTAs take rows and join what their warps have themselves, or 0: runs and a joining kernel,
// which costs about as much as a warp's stage, 1.6 us. So rows where no warp has more than one stage beyond what
// runs would give it (and few at all: runs even out lengths below the bound). A cluster doubles while its CTAs
// have stages and all clusters have room at once: 16 of eight CTAs, of which 14 have, are slower than runs.
// us, runs and rows, of G 4 and D 128, by rows and the stages of each: 8 and 2 5.7, 4.0; 8 and 10 5.8, 5.2;
// 8 and 22 5.9, 5.3; 8 and 63 7.5, 5.9; 8 and 125 8.1, 7.1; 14 and 125 10.1, 7.6; 32 and 32 6.8, 5.9; 64 and 32 9.2, 7.2;
// 64 and 63 12.5, 10.7; 96 and 32 11.1, 9.8; 128 and 4 6.4, 4.8; 128 and 32 11.9, 10.7; 144 and 54 17.6, 15.8; not taken, with
// weights as one f16 and up to that many stages: 128 and 63 13.4, 13.9, 16 and 125 8.4, 12.1 (eight CTAs). Of sixteen CTAs, 7
// have room: 1 and 250 7.7, 7.4; 4 and 250 8.5, 7.7; 7 and 250 9.8, 8.3. 32 rows of 32 stages of G 16: 10.4, 8.3.
int row_cluster(int64_t rows, int64_t stages, int sms, const int *room) {
    if (rows > room[0]) return 0;
    int i = 0;
    while (i + 1 < kClusterSizes && kWarps << i < stages && rows <= room[i + 1]) ++i;
    const int64_t mine = (stages + (kWarps << i) - 1) / (kWarps << i);
    const int64_t runs = (rows * stages + (int64_t)sms * kWarps - 1) / ((int64_t)sms * kWarps);
    return mine <= std::min<int64_t>(runs + 1, kRowStages) ? 1 << i : 0;
}

template <typename T, int D, int GT>
int launch_t(const DecodeParams &p, const RunWork &ws, int64_t max_ctx, int64_t stages, int sms, cudaStream_t stream) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return -1;
    const int64_t rows = (int64_t)p.num_seqs * p.num_kv_heads;
    const int *room = RowCtas<T, D, GT>::room(dev);
    if (room == nullptr) return -1;
    const int cluster = row_cluster(rows, stages, sms, room);
    if (cluster == 0) return launch_runs<T, D, GT>(p, ws, max_ctx, launch_grid(rows, stages, sms), stream);
    RowCtas<T, D, GT> l(rows, cluster, stream);
    return cudaLaunchKernelEx(&l.cfg, decode_fp8_block_kernel<T, D, GT, true>, p, ws) == cudaSuccess ? 0 : -1;
}

template <typename T>
int launch_d(const DecodeParams &p, const RunWork &ws, int64_t max_ctx, int64_t stages, int sms, cudaStream_t stream) {
    if (p.head_dim == 128)
        return p.group <= 8 ? launch_t<T, 128, 8>(p, ws, max_ctx, stages, sms, stream)
                            : launch_t<T, 128, 16>(p, ws, max_ctx, stages, sms, stream);
    return p.group <= 8 ? launch_t<T, 64, 8>(p, ws, max_ctx, stages, sms, stream)
                        : launch_t<T, 64, 16>(p, ws, max_ctx, stages, sms, stream);
}

int64_t row_stages(int64_t max_ctx, int64_t head_dim) {
    const int tok = stage_tokens((int)head_dim);
    return (max_ctx + tok - 1) / tok;
}

// Sequences per launch: what the kernel's prefix holds, and a launch's stages in 31 bits.
int64_t seqs_per_launch(int64_t stages, int64_t kv_heads) {
    return std::max<int64_t>(1, std::min<int64_t>(kMaxSeqs, INT32_MAX / std::max<int64_t>(stages * kv_heads, 1)));
}

}  // namespace

bool decode_fp8_block_supported(const DecodeParams &p, int dtype) {
    return (dtype == PA_DTYPE_BF16 || dtype == PA_DTYPE_F16) && (p.head_dim == 64 || p.head_dim == 128) &&
           p.group >= 1 && p.group <= 16 && p.block_size >= 8 && p.block_size <= 256 && p.num_blocks < INT32_MAX &&
           (int64_t)p.num_seqs * p.num_heads < INT32_MAX;
}

// At most one partial per run and one more per row: runs + rows of a launch.
RunWorkSizes decode_fp8_block_work_sizes(int64_t num_seqs, int64_t num_heads, int64_t num_kv_heads, int64_t head_dim,
                                         int64_t max_ctx, int sms) {
    const int64_t group = num_heads / num_kv_heads, stages = row_stages(max_ctx, head_dim);
    const int64_t rows = std::min(num_seqs, seqs_per_launch(stages, num_kv_heads)) * num_kv_heads;
    const int64_t parts = (int64_t)launch_grid(rows, stages, sms) * kWarps + rows;
    RunWorkSizes s;
    s.rows = (size_t)(rows * 8);
    s.part_ml = (size_t)(parts * group * 8);
    s.part_o = (size_t)(parts * group * head_dim * 4);
    return s;
}

int launch_decode_fp8_block(const DecodeParams &p, const RunWork &ws, int64_t max_ctx, int sms, int dtype,
                            cudaStream_t stream) {
    const int64_t stages = row_stages(max_ctx, p.head_dim);
    if (!decode_fp8_block_supported(p, dtype) || stages * p.num_kv_heads > INT32_MAX) return -2;
    const int chunk = (int)std::min<int64_t>(p.num_seqs, seqs_per_launch(stages, p.num_kv_heads));
    for (int b0 = 0; b0 < p.num_seqs; b0 += chunk) {
        DecodeParams c = p;
        const int64_t first = (int64_t)b0 * p.num_heads * p.head_dim * 2;
        c.num_seqs = std::min(chunk, p.num_seqs - b0);
        c.q = static_cast<const char *>(p.q) + first;
        c.out = static_cast<char *>(p.out) + first;
        c.block_tables = p.block_tables + (int64_t)b0 * p.max_blocks_per_seq;
        c.context_lens = p.context_lens + b0;
        const int rc = dtype == PA_DTYPE_BF16 ? launch_d<__nv_bfloat16>(c, ws, max_ctx, stages, sms, stream)
                                              : launch_d<__half>(c, ws, max_ctx, stages, sms, stream);
        if (rc != 0) return rc;
    }
    return 0;
}

}  // namespace pa
