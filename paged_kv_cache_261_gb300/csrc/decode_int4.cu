// Decode attention over a 4-bit paged cache (format: kv_int4.cu).
//
// What is computed is the decode attention of "CS349E lecture 7:
// 01_paged_attention.py", demo 2, paper eq. 4 (block-wise scores through the block
// table, one softmax over the whole context, block-wise V accumulation) over the
// dequantised cache: K = code * k_scale + k_zero per token and kv head, V alike. With
// n the codes, the scale and the zero leave both contractions:
//   q . K_t          = k_scale_t (q . n_t) + k_zero_t sum(q)
//   sum_t p_t V_t[c] = sum_t (p_t v_scale_t) n_t[c] + sum_t p_t v_zero_t
//
// The codes become matrix operands by a mask alone: 0x000n and 0x00n0 are the f16
// subnormals n 2^-24 and 16 n 2^-24, so one AND turns a word's nibbles (0, 4) into a
// pair of f16 and another its nibbles (1, 5); shifted by 8, the other four. The powers
// of two leave through the query (its odd channels divided by 16) and the output.
// Per 16 tokens a warp multiplies, with mma.m16n8k16 (f16 operands, f32 sums),
//   S^T[16 tok x 8 heads] = n_K[16 x D] . Q^T        A = codes, row = token
//   O^T[D x 8 heads]     += n_V^T[D x 16 tok] . W^T   A = codes, row = channel
// The order of the channels inside a contraction, and of the output's rows over the
// instructions, is free; it is chosen so that every lane's codes are consecutive bytes
// of a row (D / 8 for K, D / 16 for V). S^T's fragments turn into W^T's with one 8x8
// transpose in registers.
//
// W = p v_scale enters the product as f16 (11 bits; the row sums take p unrounded). Its
// reference is a maximum of the scores (raised only when a score exceeds it by 2^7: no
// reduction over the lanes before) and a power of two above every v_scale seen, so
// weights are normal f16 numbers down to 2^-22 of the reference times that power and within
// 2^-33 of it below: a V row far larger than the others costs them bits. The query enters
// as f16 times a power of two per head: exact for bf16 and f16 at every channel within
// 2^-22 of the row's largest.
//
// The codes enter about their middle, 7.5, or the rounding of W would come out multiplied by
// codes that are all of one sign, and the sums over a long context, which cancel against
// those of the zeros, would drown it. Odd tokens have their codes complemented (by the mask's
// instruction) and their W negated, so the products sum up around zero; with
// v_mid = v_zero + 7.5 v_scale and s = +-1,
//   sum_t p_t V_t[c] = sum_t (s_t W_t) n'_t[c] - 7.5 sum_t (s_t W_t) + sum_t p_t v_mid_t,
// n' = n or 15 - n, and every W the rounded one. Error of f16 outputs over contexts of 60,000
// flat weights: 2.9e-4, 2.0e-4 of it their own rounding (6.1e-4 with plain codes, at 3 % less
// time; codes made signed by an f16 addition cost 7 %).
//
// Work: the stages (64 tokens of one sequence and kv head) of the whole call, in order,
// are cut into equal runs, one for each warp of the persistent grid; a run that covers a
// row (sequence, kv head) writes its result, the others leave partials that a second
// kernel joins. Warps share nothing, so nothing synchronises them. (Items of a CTA whose
// warps joined their states through shared memory took 65 us on the 8B-shaped batch, with
// 27.7 instructions a token against 18 in this form.) Each warp fetches its own stages, one
// ahead and across rows, into its own ring: a block of one kv head is one contiguous run for
// K, V and the parameters each, so a stage is a few untiled bulk copies on one mbarrier.
//
// What bounds it (one GB300): the 8B-shaped batch, 162 MB, takes 38.0 us, of which about 8
// are the two kernels' start and the join; long contexts, 711 MB, take 126.8 us, 5.6 TB/s.
// The copies alone take 33.7 and 115 us.
// Stages of 32 tokens and 16 warps per SM: 39.9 and 135 us (a stage's fixed work, about 60
// instructions, comes twice as often, and 128 registers leave less in flight).
//
// Every wait is bounded; on a timeout the kernel sets PA_DEVERR_WAIT, waits (bounded)
// for its copies in flight and returns.
#include "common.cuh"
#include "kernels_compress.h"
#include "sm100.cuh"

#include <algorithm>
#include <type_traits>

namespace pa {
namespace {

using namespace sm100;

// Two stages a warp: 209 KB per SM. (With stages of 32 tokens, where a third fitted, it
// measured slower: 41.7 against 39.9 us on the 8B-shaped batch, 137.8 against 135.4 us on
// long contexts.)
constexpr int kStages = 2;
constexpr int kMaxSeqs = 1536;                    // sequences per launch (the host splits larger batches)

// The softmax reference of a head is not raised before a score exceeds it by this many
// powers of two: the weights (f16, up to 2^kWeightExp times 2^kSlack) have the room.
constexpr float kSlack = 7.f;
constexpr int kWeightExp = 8;

// GT: query heads padded to 8 or 16.
template <int D, int GT> struct Cfg {
    static constexpr int kWarps = kInt4Warps(GT);
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kTok = kInt4StageTokens;             // tokens per stage
    static constexpr int kRow = D / 2;                        // bytes of a token's codes
    static constexpr int kOffV = kTok * kRow;
    static constexpr int kOffPar = 2 * kTok * kRow;
    static constexpr int kSlot = kTok * (2 * kRow + 8);
    static constexpr int kRing = kWarps * kStages * kSlot;
    // after the ring
    static constexpr int kOffBar = kRing;                             // [kWarps][kStages]
    static constexpr int kOffMisc = kOffBar + kWarps * kStages * 8;   // abort flag; warp sums of the prefix
    static constexpr int kOffPre = kOffMisc + 16 + kWarps * 4;        // int [kMaxSeqs + 1]
    static constexpr int kSmem = kOffPre + (kMaxSeqs + 1) * 4;
    static_assert(kSmem <= 232448, "shared memory budget");
    static_assert(kSlot % 16 == 0 && kOffV % 16 == 0 && kOffPar % 16 == 0, "bulk copies start on 16 bytes");
};

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
__device__ __forceinline__ float2 unpack_half2(uint32_t u) { return __half22float2(*reinterpret_cast<__half2 *>(&u)); }
// Two fp32 lanes in one instruction: a * b + c, a * b, a + b.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};"
        "\n\tfma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};"
        "\n\tmul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};"
        "\n\tadd.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
// a += the two halves of b, in f32.
__device__ __forceinline__ void add_halves(float2 &a, uint32_t b) {
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tadd.rn.f32.f16 %0, lo, %0;\n\tadd.rn.f32.f16 %1, hi, %1;\n\t}"
        : "+f"(a.x), "+f"(a.y)
        : "r"(b));
}
// (x ^ flip) & mask in one instruction.
__device__ __forceinline__ uint32_t codes(uint32_t x, uint32_t mask, uint32_t flip) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0x48;" : "=r"(r) : "r"(x), "r"(mask), "r"(flip));
    return r;
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

template <typename T, int D, int GT, bool kScore>
__global__ __launch_bounds__((Cfg<D, GT>::kThreads), 1) void decode_int4_kernel(const DecodeParams p, const Int4Work ws) {
    using C = Cfg<D, GT>;
    constexpr int kWarps = C::kWarps, kThreads = C::kThreads;
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
        for (int i = 0; i < kWarps * kStages; ++i) mbar_init(&bars[i], 1);
        *abort_flag = 0;
        mbar_fence_init();
    }
    // as the other decode kernels: the set-up and the cut of the work (which reads only the
    // call's lengths) overlap the preceding kernel
    asm volatile("griddepcontrol.launch_dependents;");
    auto context = [&](int b) {
        const int c = p.context_lens[b];
        return c < 0 ? 0 : min(c, p.context_limit);
    };
    {
        const int per = (B + kThreads - 1) / kThreads, b0 = min(B, tid * per), b1 = min(B, b0 + per);
        int sum = 0;
        for (int b = b0; b < b1; ++b) {
            const int raw = p.context_lens[b];
            if ((raw < 0 || raw > p.context_limit) && blockIdx.x == 0) raise_error(p.err, PA_DEVERR_CONTEXT);
            sum += (context(b) + C::kTok - 1) / C::kTok;
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
            at += (context(b) + C::kTok - 1) / C::kTok;
        }
        if (b1 == B && (b0 < B || tid == 0)) pre[B] = at;
    }
    __syncthreads();
    const uint32_t total = (uint32_t)pre[B] * Hk;      // below 2^31: the host sees to it
    const uint32_t num_runs = max(1u, min(gridDim.x * kWarps, total));
    const Runs runs(total, num_runs);
    // runs go to the SMs in turn, so few of them still use all
    const uint32_t run = warp * gridDim.x + blockIdx.x;
    int todo = 0;
    Cursor at = {};
    if (run < num_runs && total > 0) {
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
        c.s = 0;
        if (++c.kvh < Hk) return;
        c.kvh = 0;
        do ++c.b; while (pre[c.b + 1] == pre[c.b]);
        c.ns = pre[c.b + 1] - pre[c.b];
        c.ctx = context(c.b);
    };

    // ---- fetching: lanes 0-7 the K runs, 8-15 the V runs, 16-23 the parameters of a
    // stage's blocks (at most 8: block_size >= 8)
    unsigned char *ring = smem + warp * kStages * C::kSlot;
    uint64_t *full = bars + warp * kStages;
    const int kind = lane >> 3;
    const int piece_tok = min(p.block_size, C::kTok);
    const int piece_off = (lane & 7) * piece_tok;      // the piece's first token of the stage
    const int piece_row = kind == 2 ? 8 : C::kRow;     // bytes per token of this lane's array
    const bool fetches = kind < 3 && piece_off < C::kTok;
    const unsigned char *src_base = static_cast<const unsigned char *>(
        kind == 2 ? p.kv_params : (kind == 1 ? p.value_cache : p.key_cache));
    const uint32_t dst_off = (kind == 2 ? C::kOffPar : (kind == 1 ? C::kOffV : 0)) + piece_off * piece_row;
    const uint32_t piece_bytes = piece_tok * piece_row;
    const uint32_t run_bytes = (uint32_t)piece_row << p.log2_block_size;   // a block's rows of one kv head
    const uint32_t block_bytes = run_bytes * (uint32_t)Hk;                 // at most 2^16 * 2^8 * 64

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
        if (lane == 0) mbar_arrive_expect_tx(bar, blocks * piece_tok * (2 * C::kRow + 8));
        __syncwarp();
        if (good) {
            const uint32_t off = (uint32_t)nx.kvh * run_bytes +
                                 (uint32_t)((nx.s * C::kTok + piece_off) & (p.block_size - 1)) * piece_row;
            bulk_load(dst, src_base + ((uint64_t)(uint32_t)entry * block_bytes + off), piece_bytes, bar);
        } else if (live) {
            // a bad block id: zeros, so its tokens have score and value 0
            if (kind == 0) raise_error(p.err, PA_DEVERR_BLOCK_ID);
            for (uint32_t i = 0; i < piece_bytes; i += 8) *reinterpret_cast<uint2 *>(dst + i) = make_uint2(0, 0);
            fence_proxy_async_smem();
        }
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
    // what the joining kernel needs of every row: its first partial and how many there are
    // (0: the row is written here). A run's partial of a row is number run + row: both rise
    // along the order, so the numbers are distinct and a row's are consecutive.
    for (int r = blockIdx.x * kThreads + tid; r < B * Hk; r += gridDim.x * kThreads) {
        const int b = r / Hk, h = r - b * Hk, ns = pre[b + 1] - pre[b];
        int2 info = make_int2(0, 0);
        if (ns > 0) {
            const uint32_t s0 = (uint32_t)pre[b] * Hk + (uint32_t)h * ns;
            const int w0 = (int)runs.owner(s0), w1 = (int)runs.owner(s0 + ns - 1);
            if (w1 > w0) info = make_int2(w0 + r, w1 - w0 + 1);
        }
        ws.rows[r] = info;
    }
    T *out = reinterpret_cast<T *>(p.out);
    for (int b = blockIdx.x; b < B; b += gridDim.x)    // rows of empty contexts
        if (pre[b + 1] == pre[b])
            for (int i = tid; i < p.num_heads * D; i += kThreads)
                out[(int64_t)b * p.num_heads * D + i] = Elem<T>::from_f(0.f);

    if (todo == 0) return;
    int left = todo;                                   // stages to consume
    int unfetched = todo - min(todo, kStages);         // and to fetch
    int sl = 0;                                        // the slot of the next stage
    uint32_t phase = 0;                                // and its barrier's phase
    bool ok = true;

    uint32_t flip;                                     // odd tokens' codes, complemented; a register, so that
    asm volatile("mov.b32 %0, 0xFFFF0000;" : "=r"(flip));   // complement and mask are one instruction
    [[maybe_unused]] const uint64_t keep = kScore ? l2_keep() : 0;
    const T *q = reinterpret_cast<const T *>(p.q);
    while (left > 0) {
        // ---- the part of row (b, kvh) that lies in this run
        const int I_b = at.b, I_kvh = at.kvh;
        const int s_end = min(at.ns, at.s + left);
        const bool whole = at.s == 0 && s_end == at.ns;
        const int64_t head0 = (int64_t)I_b * p.num_heads + (int64_t)I_kvh * G;

        // the group's query as B fragments, and the factors of x = S * (k_scale * sa) + k_zero * sb
        // of the heads of S^T's columns
        uint32_t qb[NT][kSteps][2];
        float2 sa[NT], sb[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            constexpr int N = D / 4;                   // channels of a lane
            const int g = nt * 8 + li;
            float x[N];
            const T *src = q + (head0 + min(g, G - 1)) * D + lj * N;
#pragma unroll
            for (int u = 0; u < N / 8; ++u) Vec16<T>::unpack(__ldg(reinterpret_cast<const uint4 *>(src) + u), x + 8 * u);
            float amax = 0.f, sum = 0.f;
#pragma unroll
            for (int u = 0; u < N; ++u) {
                if (g >= G) x[u] = 0.f;
                amax = fmaxf(amax, fabsf(x[u]));
                sum += x[u];
            }
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                sum += __shfl_xor_sync(0xffffffffu, sum, o);
            }
            // amax = 1.f * 2^(E - 127), scaled into [2^12, 2^13)
            const int E = (int)((__float_as_uint(amax) >> 23) & 0xFF);
            const int e2 = E == 0 ? 100 : max(-116, min(100, 139 - E));
            const float up = pow2f(e2), up16 = pow2f(e2 - 4);
#pragma unroll
            for (int w = 0; w < N / 8; ++w) {
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    const float *y = x + 8 * w + 2 * hh;
                    qb[nt][2 * w + hh][0] = pack_half2(y[0] * up, y[4] * up);
                    qb[nt][2 * w + hh][1] = pack_half2(y[1] * up16, y[5] * up16);
                }
            }
            const float a = p.scale_log2 * pow2f(-e2) * 16777216.f, c = p.scale_log2 * sum;
            sa[nt] = make_float2(__shfl_sync(0xffffffffu, a, 8 * lj), __shfl_sync(0xffffffffu, a, 8 * lj + 4));
            sb[nt] = make_float2(__shfl_sync(0xffffffffu, c, 8 * lj), __shfl_sync(0xffffffffu, c, 8 * lj + 4));
        }
        float O[NT][kSteps][4];
        float2 nm[NT], l[NT], z[NT], sw[NT];           // nm: the negated references; sw: sums of W
        int r_exp = -40;                               // 2^r_exp = r_top > every v_scale seen
        float r_top = 0.f, cr = 0.f;                   // |v_scale * cr| < 2^kWeightExp, negative in odd rows
        bool first = true;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int u = 0; u < kSteps; ++u)
#pragma unroll
                for (int c = 0; c < 4; ++c) O[nt][u][c] = 0.f;
            nm[nt] = make_float2(INFINITY, INFINITY);
            l[nt] = z[nt] = sw[nt] = make_float2(0.f, 0.f);
        }
        // one stage; kTail: only its first n tokens belong to the row
        auto stage = [&](auto tail, const unsigned char *slot, int ts, int n) {
            constexpr bool kTail = decltype(tail)::value;
            // ---- scores, S^T: rows li and li + 8 of each 16 tokens
            float S[kSub][NT][4];
            float vs[kSub][2], vz[kSub][2];
            float rmax = 0.f;
#pragma unroll
            for (int sub = 0; sub < kSub; ++sub) {
                float S2[NT][4];                       // a second chain of sums
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 4; ++c) S[sub][nt][c] = S2[nt][c] = 0.f;
                uint32_t ka[D / 32], kb[D / 32];   // this lane's words of the two rows
                const unsigned char *kr = slot + (sub * 16 + li) * C::kRow + lj * (D / 8);
                if constexpr (D == 128) {
                    *reinterpret_cast<uint4 *>(ka) = *reinterpret_cast<const uint4 *>(kr);
                    *reinterpret_cast<uint4 *>(kb) = *reinterpret_cast<const uint4 *>(kr + 8 * C::kRow);
                } else {
                    *reinterpret_cast<uint2 *>(ka) = *reinterpret_cast<const uint2 *>(kr);
                    *reinterpret_cast<uint2 *>(kb) = *reinterpret_cast<const uint2 *>(kr + 8 * C::kRow);
                }
#pragma unroll
                for (int w = 0; w < D / 32; ++w) {
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        const uint32_t a = ka[w] >> (8 * hh), b = kb[w] >> (8 * hh);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma16816(hh ? S2[nt] : S[sub][nt], a & 0x000F000Fu, b & 0x000F000Fu, a & 0x00F000F0u,
                                     b & 0x00F000F0u, qb[nt][2 * w + hh][0], qb[nt][2 * w + hh][1]);
                    }
                }
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int t = sub * 16 + li + 8 * r;
                    const uint2 par = *reinterpret_cast<const uint2 *>(slot + C::kOffPar + t * 8);
                    const float2 kp = unpack_half2(par.x), vp = unpack_half2(par.y);
                    const bool valid = !kTail || t < n;
                    vs[sub][r] = valid ? vp.x : 0.f;
                    vz[sub][r] = valid ? fmaf(7.5f, vp.x, vp.y) : 0.f;    // the value of code 7.5
                    rmax = fmaxf(rmax, fabsf(vs[sub][r]));
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const float2 dot = add2(make_float2(S[sub][nt][2 * r], S[sub][nt][2 * r + 1]),
                                                make_float2(S2[nt][2 * r], S2[nt][2 * r + 1]));
                        const float2 x = fma2(dot, make_float2(kp.x * sa[nt].x, kp.x * sa[nt].y),
                                              make_float2(kp.y * sb[nt].x, kp.y * sb[nt].y));
                        S[sub][nt][2 * r] = valid ? x.x : -INFINITY;
                        S[sub][nt][2 * r + 1] = valid ? x.y : -INFINITY;
                        if constexpr (kScore) {
                            const int pl = nt * 4 + lj;    // planes of two heads
                            if (valid && 2 * pl < G)
                                store_keep(p.ws_logits + ((int64_t)I_b * Hk + I_kvh) * p.logits_row +
                                               ((int64_t)pl * p.logits_len + ts + t) * 2,
                                           make_float2(S[sub][nt][2 * r], S[sub][nt][2 * r + 1]), keep);
                        }
                    }
                }
            }
            // ---- this lane's V words of every 16 tokens (2 lj, 2 lj + 1, 2 lj + 8, 2 lj + 9), read
            // before the references are looked at (long contexts 127.9 -> 122.7 us)
            uint32_t vw[kSub][4][D / 64];
#pragma unroll
            for (int sub = 0; sub < kSub; ++sub) {
                const unsigned char *vr = slot + C::kOffV + (sub * 16 + 2 * lj) * C::kRow + li * (D / 16);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const unsigned char *src = vr + ((k & 1) + (k & 2) * 4) * C::kRow;
                    if constexpr (D == 128) *reinterpret_cast<uint2 *>(vw[sub][k]) = *reinterpret_cast<const uint2 *>(src);
                    else vw[sub][k][0] = *reinterpret_cast<const uint32_t *>(src);
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
                const int r_new = max(r_exp, min(17, (int)((__float_as_uint(rows_max(rmax)) >> 23) & 0xFF) - 126));
                const float rs = pow2f(r_exp - r_new);
                r_exp = r_new;
                r_top = pow2f(r_new);
                cr = pow2f(kWeightExp - r_new) * (li & 1 ? -1.f : 1.f);
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
                        const float2 a2 = make_float2(a[0], a[1]);
                        l[nt] = mul2(l[nt], a2);
                        z[nt] = mul2(z[nt], a2);
                        sw[nt] = mul2(sw[nt], make_float2(a[0] * rs, a[1] * rs));
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
                uint32_t wb[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const float2 d = add2(make_float2(S[sub][nt][2 * r], S[sub][nt][2 * r + 1]), nm[nt]);
                        const float2 w = make_float2(fast_exp2(d.x), fast_exp2(d.y));
                        l[nt] = add2(l[nt], w);
                        z[nt].x = fmaf(w.x, vz[sub][r], z[nt].x);
                        z[nt].y = fmaf(w.y, vz[sub][r], z[nt].y);
                        const float v = vs[sub][r] * cr;
                        const uint32_t wh = pack_half2(w.x * v, w.y * v);
                        add_halves(sw[nt], wh);
                        wb[nt][r] = transpose8x8(wh);
                    }
                // 16 bits (4 channels) of two tokens' bytes side by side: byte b of both in
                // the low bytes of the halves, for the pairs of nibbles that byte holds
                constexpr int H = D / 32;              // 16-bit pieces of a lane's bytes
#pragma unroll
                for (int h = 0; h < H / 2; ++h)
#pragma unroll
                    for (int eb = 0; eb < 2; ++eb) {
                        // byte eb of piece h (rows li) and of piece h + H / 2 (rows li + 8)
                        const int h2 = h + H / 2;
                        const uint32_t sel = (h & 1 ? 0x6622u : 0x4400u) + (eb ? 0x1111u : 0u);
                        const uint32_t sel2 = (h2 & 1 ? 0x6622u : 0x4400u) + (eb ? 0x1111u : 0u);
                        const uint32_t x0 = __byte_perm(vw[sub][0][h / 2], vw[sub][1][h / 2], sel);
                        const uint32_t x1 = __byte_perm(vw[sub][0][h2 / 2], vw[sub][1][h2 / 2], sel2);
                        const uint32_t x2 = __byte_perm(vw[sub][2][h / 2], vw[sub][3][h / 2], sel);
                        const uint32_t x3 = __byte_perm(vw[sub][2][h2 / 2], vw[sub][3][h2 / 2], sel2);
#pragma unroll
                        for (int en = 0; en < 2; ++en) {
                            const uint32_t mask = en ? 0x00F000F0u : 0x000F000Fu;
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma16816(O[nt][4 * h + 2 * eb + en], codes(x0, mask, flip), codes(x1, mask, flip),
                                         codes(x2, mask, flip), codes(x3, mask, flip), wb[nt][0], wb[nt][1]);
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
            const int ts = at.s * C::kTok, n = at.ctx - ts;   // valid tokens, at least 1
            if (n >= C::kTok) stage(std::false_type{}, slot, ts, n);
            else stage(std::true_type{}, slot, ts, n);
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
        // A lane has channels li D / 8 + r D / 16 + u of heads 2 lj and 2 lj + 1.
        const int r = I_b * Hk + I_kvh;
        const float unit = pow2f(r_exp - kWeightExp), even = pow2f(r_exp + 24 - kWeightExp),
                    odd = pow2f(r_exp + 20 - kWeightExp);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float ls = rows_sum(c ? l[nt].y : l[nt].x);
                const float zs = rows_sum(fmaf(c ? sw[nt].y : sw[nt].x, -7.5f * unit, c ? z[nt].y : z[nt].x));
                const int g = nt * 8 + 2 * lj + c;
                if (g >= G) continue;
                const float inv = whole ? 1.f / ls : 1.f;
#pragma unroll
                for (int rr = 0; rr < 2; ++rr) {
                    float v[kSteps];
#pragma unroll
                    for (int u = 0; u < kSteps; ++u)
                        v[u] = fmaf(O[nt][u][2 * rr + c], u & 1 ? odd : even, zs) * inv;
                    const int d0 = li * (D / 8) + rr * (D / 16);
                    if (whole) {
                        alignas(16) T h[kSteps];
#pragma unroll
                        for (int u = 0; u < kSteps; ++u) h[u] = Elem<T>::from_f(v[u]);
                        T *dst = out + (head0 + g) * D + d0;
                        if constexpr (kSteps == 8) *reinterpret_cast<uint4 *>(dst) = *reinterpret_cast<uint4 *>(h);
                        else *reinterpret_cast<uint2 *>(dst) = *reinterpret_cast<uint2 *>(h);
                    } else {
                        float *dst = ws.part_o + ((int64_t)(run + r) * G + g) * D + d0;
#pragma unroll
                        for (int u = 0; u < kSteps; u += 4)
                            *reinterpret_cast<float4 *>(dst + u) = make_float4(v[u], v[u + 1], v[u + 2], v[u + 3]);
                    }
                }
                if (li == 0) {
                    if (!whole) ws.part_ml[(int64_t)(run + r) * G + g] = make_float2(-(c ? nm[nt].y : nm[nt].x), ls);
                    else if (kScore) reinterpret_cast<float2 *>(p.ws_score_ml)[head0 + g] = make_float2(-(c ? nm[nt].y : nm[nt].x), ls);
                }
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
}

// Joins the partials of the rows that several runs share: M = max m_i, L = sum l_i
// 2^(m_i - M), out = sum o_i 2^(m_i - M) / L. Warps per (query head, sequence), WPR: one where a
// row has few partials, 4 or 16 (joined through shared memory) where it has many. A warp reads
// 32 partials' pairs at once, one a lane, and then their outputs, kJoinBatch in flight.
constexpr int kJoinWarps(int wpr) { return wpr < 4 ? 4 : wpr; }      // of a CTA
constexpr int kJoinBatch = 8;

template <typename T, int D, int WPR, int kWarps = kJoinWarps(WPR)>
__global__ __launch_bounds__(kWarps * 32) void decode_int4_join_kernel(const DecodeParams p, const Int4Work ws) {
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

template <typename T, int D, int GT, bool kScore>
int launch_t(const DecodeParams &p, const Int4Work &ws, int64_t max_ctx, int grid, cudaStream_t stream) {
    using C = Cfg<D, GT>;
    auto kern = decode_int4_kernel<T, D, GT, kScore>;
    static bool attr_set[kMaxDevices] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return -1;
    if (!attr_set[dev]) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess) return -1;
        attr_set[dev] = true;
    }
    const int rc = launch_pdl(kern, dim3((unsigned)grid), dim3(C::kThreads), C::kSmem, stream, p, ws);
    if (rc != 0) return rc;
    // Partials a row: about runs / rows, for contexts of the limit's length. (8 kv heads, us with up to
    // 4 warps a row and with 16: one context of 16,000 tokens 21.2 and 13.2, of 131,072 44.9 and 35.9,
    // three of 40,000 to 120,000 60.0 and 55.4; with 11 partials a row, 16 warps are 0.15 slower.)
    // The limit is that of the call's arguments alone, before mass cuts p.context_limit: the warps
    // decide the order of the sums, and out does not depend on whether weights are accumulated.
    const int64_t heads = (int64_t)p.num_seqs * p.num_heads, rows = (int64_t)p.num_seqs * p.num_kv_heads;
    const int64_t limit = std::min(max_ctx, (int64_t)p.max_blocks_per_seq * p.block_size);
    const int64_t stages = (limit + C::kTok - 1) / C::kTok;
    const int64_t runs = std::min<int64_t>((int64_t)grid * C::kWarps, rows * stages);
    const int wpr = runs <= 8 * rows ? 1 : (runs <= 32 * rows ? 4 : 16), cta = kJoinWarps(wpr);
    auto join = wpr == 1   ? decode_int4_join_kernel<T, D, 1>
                : wpr == 4 ? decode_int4_join_kernel<T, D, 4>
                           : decode_int4_join_kernel<T, D, 16>;
    return launch_pdl(join, dim3((unsigned)((heads * wpr + cta - 1) / cta)), dim3(cta * 32), 0, stream, p, ws);
}

template <typename T, int D>
int launch_g(const DecodeParams &p, const Int4Work &ws, int64_t max_ctx, int grid, cudaStream_t stream) {
    if (p.ws_logits)
        return p.group <= 8 ? launch_t<T, D, 8, true>(p, ws, max_ctx, grid, stream)
                            : launch_t<T, D, 16, true>(p, ws, max_ctx, grid, stream);
    return p.group <= 8 ? launch_t<T, D, 8, false>(p, ws, max_ctx, grid, stream)
                        : launch_t<T, D, 16, false>(p, ws, max_ctx, grid, stream);
}

template <typename T>
int launch_d(const DecodeParams &p, const Int4Work &ws, int64_t max_ctx, int grid, cudaStream_t stream) {
    return p.head_dim == 128 ? launch_g<T, 128>(p, ws, max_ctx, grid, stream)
                             : launch_g<T, 64>(p, ws, max_ctx, grid, stream);
}

int64_t row_stages(int64_t max_ctx) { return (max_ctx + kInt4StageTokens - 1) / kInt4StageTokens; }

// Sequences per launch: what the kernel's prefix holds, and a launch's stages in 31 bits.
int64_t seqs_per_launch(int64_t max_ctx, int64_t kv_heads) {
    const int64_t ns = row_stages(max_ctx) * kv_heads;
    return std::max<int64_t>(1, std::min<int64_t>(kMaxSeqs, INT32_MAX / std::max<int64_t>(ns, 1)));
}

// One CTA per SM, and no more than there can be stages.
int launch_grid(int64_t seqs, int64_t kv_heads, int64_t max_ctx, int sms) {
    return (int)std::max<int64_t>(1, std::min<int64_t>(sms, seqs * kv_heads * row_stages(max_ctx)));
}

}  // namespace

bool decode_int4_supported(const DecodeParams &p, int dtype) {
    return (dtype == PA_DTYPE_BF16 || dtype == PA_DTYPE_F16) && (p.head_dim == 64 || p.head_dim == 128) &&
           p.group >= 1 && p.group <= 16 && p.block_size >= 8 && p.block_size <= 256 && p.num_blocks < INT32_MAX &&
           (int64_t)p.num_seqs * p.num_heads < INT32_MAX;
}

// At most one partial per run and one more per row: runs + rows of a launch.
Int4WorkSizes decode_int4_work_sizes(int64_t num_seqs, int64_t num_heads, int64_t num_kv_heads, int64_t head_dim,
                                     int64_t max_ctx, int sms) {
    const int group = (int)(num_heads / num_kv_heads);
    const int64_t seqs = std::min(num_seqs, seqs_per_launch(max_ctx, num_kv_heads));
    const int64_t rows = seqs * num_kv_heads;
    const int64_t parts = (int64_t)launch_grid(seqs, num_kv_heads, max_ctx, sms) * kInt4Warps(group <= 8 ? 8 : 16) + rows;
    Int4WorkSizes s;
    s.rows = (size_t)(rows * 8);
    s.part_ml = (size_t)(parts * group * 8);
    s.part_o = (size_t)(parts * group * head_dim * 4);
    return s;
}

int launch_decode_int4(const DecodeParams &p, const Int4Work &ws, int64_t max_ctx, int sms, float *mass,
                       int64_t mass_len, int dtype, cudaStream_t stream) {
    if (!decode_int4_supported(p, dtype) || row_stages(max_ctx) * p.num_kv_heads > INT32_MAX) return -2;
    const int chunk = (int)std::min<int64_t>(p.num_seqs, seqs_per_launch(max_ctx, p.num_kv_heads));
    for (int b0 = 0; b0 < p.num_seqs; b0 += chunk) {
        DecodeParams c = p;
        const int64_t rows = (int64_t)b0 * p.num_heads;
        c.num_seqs = std::min(chunk, p.num_seqs - b0);
        c.q = static_cast<const char *>(p.q) + rows * p.head_dim * 2;
        c.out = static_cast<char *>(p.out) + rows * p.head_dim * 2;
        c.block_tables = p.block_tables + (int64_t)b0 * p.max_blocks_per_seq;
        c.context_lens = p.context_lens + b0;
        if (p.ws_logits) {
            c.ws_logits = p.ws_logits + (int64_t)b0 * p.num_kv_heads * p.logits_row;
            c.ws_score_ml = p.ws_score_ml + rows * 2;
        }
        const int grid = launch_grid(c.num_seqs, c.num_kv_heads, max_ctx, sms);
        int rc = dtype == PA_DTYPE_BF16 ? launch_d<__nv_bfloat16>(c, ws, max_ctx, grid, stream)
                                        : launch_d<__half>(c, ws, max_ctx, grid, stream);
        if (rc == 0 && mass)
            rc = launch_decode_mass(c, 2, mass + (int64_t)b0 * p.num_kv_heads * mass_len, mass_len, &ws, stream);
        if (rc != 0) return rc;
    }
    return 0;
}

}  // namespace pa
