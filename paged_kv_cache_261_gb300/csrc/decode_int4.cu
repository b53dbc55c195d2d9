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
// reference is the running maximum of the scores times a power of two above every
// v_scale seen (and 2^-14), so weights are normal f16 numbers down to 2^-28 of the
// largest, whatever the scale of V. The query enters as f16 times a power of two per
// head: exact for bf16 and f16 at every channel within 2^-22 of the row's largest.
//
// Work: one item of decode_order.cuh (sequence, kv head, partition) per CTA at a time,
// persistent CTAs of 8 warps. The warps share an item's stages (32 or 64 tokens) in
// turn and keep separate softmax states, joined through shared memory at the item's end;
// nothing else synchronises them. Each warp fetches its own stages, two ahead and across
// items, into its own ring: a block of one kv head is one contiguous run for K, V and
// the parameters each, so a stage is a few untiled bulk copies on one mbarrier.
//
// Every wait is bounded; on a timeout the kernel sets PA_DEVERR_WAIT, waits (bounded)
// for its copies in flight and returns.
#include "common.cuh"
#include "decode_order.cuh"
#include "kernels_compress.h"
#include "sm100.cuh"

namespace pa {
namespace {

using namespace sm100;
using decode_order::Item;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 3;
constexpr int kMaxSeqs = 512;                     // sequences per launch (the host splits larger batches)

// GT: query heads padded to 8 or 16.
template <int D, int GT> struct Cfg {
    static constexpr int kTok = GT == 8 ? 32 : 64;            // tokens per stage
    static constexpr int kRow = D / 2;                        // bytes of a token's codes
    static constexpr int kOffV = kTok * kRow;
    static constexpr int kOffPar = 2 * kTok * kRow;
    static constexpr int kSlot = kTok * (2 * kRow + 8);
    static constexpr int kRing = kWarps * kStages * kSlot;
    // after the ring
    static constexpr int kOffMl = kRing;                              // float2 [kWarps][GT]
    static constexpr int kOffHeld = kOffMl + kWarps * GT * 8;         // int [kWarps]
    static constexpr int kOffBar = kOffHeld + kWarps * 4;             // [kWarps][kStages]
    static constexpr int kOffMisc = kOffBar + kWarps * kStages * 8;   // abort flag, item counts
    static constexpr int kOffPrefix = (kOffMisc + 16 + 15) & ~15;     // int [kMaxSeqs + 1]; later the item table
    static constexpr int kOffOrder = kOffPrefix + (kMaxSeqs + 1) * 4;
    static constexpr int kOffCtx = kOffOrder + kMaxSeqs * 4;
    static constexpr int kOffPs = kOffCtx + kMaxSeqs * 4;
    static constexpr int kSmem = kOffPs + kMaxSeqs * 4;
    static constexpr int kCtas = GT == 8 ? 2 : 1;             // per SM: registers and shared memory
    static constexpr int kPad = D + 4;                        // floats per head row of a warp's output
    static_assert(kSmem - kOffPrefix >= decode_order::kTableItems * 16, "item table fits the ordering arrays");
    static_assert(kSmem <= (GT == 8 ? 115712 : 232448), "shared memory budget");
    static_assert(GT * kPad * 4 <= kSlot, "a warp's output fits the stage it read last");
    static_assert(kWarps * GT * 8 >= kMaxSeqs, "the (max, sum) pairs serve as the ordering scratch");
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

// A warp's place in its sequence of stages: item `k` of the CTA, stage `s` of the item
// (every kWarps-th is this warp's; the first one moves on with the stages of the items
// before, so the warps' totals stay within one stage of each other).
struct Cursor {
    Item I;
    int k, s, ns, rot;
};

template <typename T, int D, int GT, bool kScore>
__global__ __launch_bounds__(kThreads, (Cfg<D, GT>::kCtas)) void decode_int4_kernel(const DecodeParams p) {
    using C = Cfg<D, GT>;
    constexpr int NT = GT / 8;                         // tiles of 8 heads
    constexpr int kSteps = D / 16;                     // instructions per 16 tokens, S and O alike
    constexpr int kSub = C::kTok / 16;
    extern __shared__ __align__(128) unsigned char smem[];
    float2 *ml_s = reinterpret_cast<float2 *>(smem + C::kOffMl);
    int *held_s = reinterpret_cast<int *>(smem + C::kOffHeld);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kOffBar);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::kOffMisc);
    int *counts = reinterpret_cast<int *>(smem + C::kOffMisc + 4);
    int *prefix = reinterpret_cast<int *>(smem + C::kOffPrefix);
    int *order = reinterpret_cast<int *>(smem + C::kOffOrder);
    const decode_order::SeqCache cache{reinterpret_cast<int *>(smem + C::kOffCtx),
                                       reinterpret_cast<int *>(smem + C::kOffPs)};
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int li = lane >> 2, lj = lane & 3;           // fragment row and column group
    const int G = p.group;

    if (tid == 0) {
        for (int i = 0; i < kWarps * kStages; ++i) mbar_init(&bars[i], 1);
        *abort_flag = 0;
        mbar_fence_init();
    }
    // as the other decode kernels: the set-up and the item order (which reads only the
    // call's lengths) overlap the preceding kernel
    asm volatile("griddepcontrol.launch_dependents;");
    decode_order::build(p, prefix, order, counts, reinterpret_cast<unsigned char *>(ml_s), cache);
    __syncthreads();
    const int n4 = counts[0];
    const int total_items = (counts[0] + counts[1]) * p.num_kv_heads;
    int4 *items = reinterpret_cast<int4 *>(smem + C::kOffPrefix);
    decode_order::build_item_table<(decode_order::kTableItems + kThreads - 1) / kThreads>(p, prefix, order, n4, cache,
                                                                                         total_items, items);
    const int nmy = decode_order::cta_items(total_items);
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");

    unsigned char *ring = smem + warp * kStages * C::kSlot;
    uint64_t *full = bars + warp * kStages;

    // ---- fetching: lanes 0-7 the K runs, 8-15 the V runs, 16-23 the parameters of a
    // stage's blocks (at most 8: block_size >= 8)
    const int piece = lane & 7, kind = lane >> 3;
    const int piece_tok = min(p.block_size, C::kTok);
    const int piece_row = kind == 2 ? 8 : C::kRow;     // bytes per token of this lane's array
    const unsigned char *src_base = static_cast<const unsigned char *>(
        kind == 2 ? p.kv_params : (kind == 1 ? p.value_cache : p.key_cache));
    const int dst_off = (kind == 2 ? C::kOffPar : (kind == 1 ? C::kOffV : 0)) + piece * piece_tok * piece_row;

    auto item_stages = [&](const Item &I) { return I.t1 > I.t0 ? (I.t1 - I.t0 + C::kTok - 1) / C::kTok : 0; };
    // moves to the next stage of this warp at or after the cursor's; false: none is left
    auto settle = [&](Cursor &c) -> bool {
        while (c.s >= c.ns) {
            if (c.k + 1 >= nmy) return false;
            c.rot = (c.rot + c.ns) & (kWarps - 1);
            ++c.k;
            c.I = decode_order::unpack_item(items[c.k]);
            c.ns = item_stages(c.I);
            c.s = (warp - c.rot) & (kWarps - 1);
        }
        return true;
    };
    auto start = [&](Cursor &c) -> bool {
        c.k = -1;
        c.rot = 0;
        c.ns = c.s = 0;
        return settle(c);
    };
    // this lane's table entry of the cursor's stage: -1 = nothing to fetch, else the block id
    // (checked when used)
    auto entry = [&](const Cursor &c) -> int {
        const int ts = c.I.t0 + c.s * C::kTok;
        const int t = ts + piece * piece_tok;
        if (kind > 2 || piece * piece_tok >= C::kTok || t >= c.I.t1) return -2;
        return p.block_tables[(int64_t)c.I.b * p.max_blocks_per_seq + (t >> p.log2_block_size)];
    };
    uint32_t issued = 0;
    // fetch the cursor's stage into the next slot of the ring (which no lane reads any more)
    auto issue = [&](const Cursor &c, int e) {
        unsigned char *slot = ring + (issued % kStages) * C::kSlot;
        uint64_t *bar = &full[issued % kStages];
        const int ts = c.I.t0 + c.s * C::kTok;
        const bool live = e != -2, good = e >= 0 && e < p.num_blocks;
        const uint32_t bytes = (uint32_t)(piece_tok * piece_row);
        const uint32_t blocks = __popc(__ballot_sync(0xffffffffu, good) & 0xFFu);
        if (lane == 0) mbar_arrive_expect_tx(bar, blocks * piece_tok * (2 * C::kRow + 8));
        __syncwarp();
        if (good) {
            const int64_t row = (((int64_t)e * p.num_kv_heads + c.I.kvh) << p.log2_block_size) +
                                ((ts + piece * piece_tok) & (p.block_size - 1));
            bulk_load(slot + dst_off, src_base + row * piece_row, bytes, bar);
        } else if (live) {
            // a bad block id: zeros, so its tokens have score and value 0
            if (kind == 0) raise_error(p.err, PA_DEVERR_BLOCK_ID);
            for (uint32_t i = 0; i < bytes; i += 8) *reinterpret_cast<uint2 *>(slot + dst_off + i) = make_uint2(0, 0);
            fence_proxy_async_smem();
        }
        __syncwarp();
        ++issued;
    };

    Cursor fetch;
    bool more = start(fetch);
    int e_next = more ? entry(fetch) : -2;
    auto fetch_one = [&]() {
        if (!more) return;
        issue(fetch, e_next);
        fetch.s += kWarps;
        more = settle(fetch);
        e_next = more ? entry(fetch) : -2;             // in flight until the next fetch
    };
    for (int i = 0; i < kStages; ++i) fetch_one();

    T *out = reinterpret_cast<T *>(p.out);
    const T *q = reinterpret_cast<const T *>(p.q);
    uint32_t used = 0;                                 // stages consumed
    int rot = 0;
    bool ok = true;
    for (int k = 0; k < nmy; ++k) {
        const Item I = decode_order::unpack_item(items[k]);
        const int64_t head0 = (int64_t)I.b * p.num_heads + (int64_t)I.kvh * G;
        const int ns = item_stages(I);
        if (ns == 0) {
            for (int i = tid; i < G * D; i += kThreads) out[head0 * D + i] = Elem<T>::from_f(0.f);
            continue;
        }
        const int s0 = (warp - rot) & (kWarps - 1);
        rot = (rot + ns) & (kWarps - 1);

        float O[NT][kSteps][4];
        float m[NT][2], l[NT][2], z[NT][2];
        int r_exp = -40;                               // 2^r_exp > every v_scale seen
        uint32_t held = 0;
        if (s0 < ns) {
            // ---- the group's query as B fragments, and per head (in S^T's columns)
            // x = S * (k_scale * sa) + k_zero * sb
            uint32_t qb[NT][kSteps][2];
            float sa[NT][2], sb[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                constexpr int N = D / 4;               // channels of a lane
                const int g = nt * 8 + li;
                float x[N];
                const T *src = q + (head0 + (g < G ? g : 0)) * D + lj * N;
#pragma unroll
                for (int u = 0; u < N / 8; ++u)
                    Vec16<T>::unpack(__ldg(reinterpret_cast<const uint4 *>(src) + u), x + 8 * u);
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
                const float a = p.scale_log2 * pow2f(-e2), b = p.scale_log2 * sum;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    sa[nt][c] = __shfl_sync(0xffffffffu, a, 8 * lj + 4 * c) * 16777216.f;
                    sb[nt][c] = __shfl_sync(0xffffffffu, b, 8 * lj + 4 * c);
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int u = 0; u < kSteps; ++u)
#pragma unroll
                    for (int c = 0; c < 4; ++c) O[nt][u][c] = 0.f;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    m[nt][c] = -INFINITY;
                    l[nt][c] = z[nt][c] = 0.f;
                }
            }
            for (int s = s0; s < ns; s += kWarps, ++used) {
                const unsigned char *slot = ring + (used % kStages) * C::kSlot;
                if (!ok || __any_sync(0xffffffffu, *abort_flag != 0) ||
                    !warp_wait(&full[used % kStages], (used / kStages) & 1)) {
                    ok = false;
                    break;
                }
                const int ts = I.t0 + s * C::kTok;
                const int n = I.t1 - ts;               // valid tokens, at least 1
                // ---- scores, S^T: rows li and li + 8 of each 16 tokens
                float S[kSub][NT][4];
                float vs[kSub][2], vz[kSub][2];
                float rmax = 0.f;
#pragma unroll
                for (int sub = 0; sub < kSub; ++sub) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 4; ++c) S[sub][nt][c] = 0.f;
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
                                mma16816(S[sub][nt], a & 0x000F000Fu, b & 0x000F000Fu, a & 0x00F000F0u,
                                         b & 0x00F000F0u, qb[nt][2 * w + hh][0], qb[nt][2 * w + hh][1]);
                        }
                    }
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int t = sub * 16 + li + 8 * r;
                        const uint2 par = *reinterpret_cast<const uint2 *>(slot + C::kOffPar + t * 8);
                        const float2 kp = unpack_half2(par.x), vp = unpack_half2(par.y);
                        const bool valid = t < n;
                        vs[sub][r] = valid ? vp.x : 0.f;
                        vz[sub][r] = valid ? vp.y : 0.f;
                        rmax = fmaxf(rmax, fabsf(vs[sub][r]));
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                float &x = S[sub][nt][2 * r + c];
                                x = valid ? fmaf(x, kp.x * sa[nt][c], kp.y * sb[nt][c]) : -INFINITY;
                            }
                            if constexpr (kScore) {
                                const int g = nt * 8 + 2 * lj;
                                float *lg = p.ws_logits +
                                            (((int64_t)I.b * p.num_kv_heads + I.kvh) * p.logits_len + ts + t) * G + g;
                                if (valid && g < G) lg[0] = S[sub][nt][2 * r];
                                if (valid && g + 1 < G) lg[1] = S[sub][nt][2 * r + 1];
                            }
                        }
                    }
                }
                // ---- running references; the rows so far are rescaled where one grew
                rmax = rows_max(rmax);
                const int r_new = max(r_exp, min(17, (int)((__float_as_uint(rmax) >> 23) & 0xFF) - 126));
                bool grew = r_new != r_exp;
                float mx[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float v = S[0][nt][c];
#pragma unroll
                        for (int sub = 0; sub < kSub; ++sub) v = fmaxf(v, fmaxf(S[sub][nt][c], S[sub][nt][2 + c]));
                        mx[nt][c] = fmaxf(m[nt][c], rows_max(v));
                        grew |= mx[nt][c] != m[nt][c];
                    }
                if (__any_sync(0xffffffffu, grew)) {
                    const float rs = pow2f(r_exp - r_new);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const float a = fast_exp2(m[nt][c] - mx[nt][c]);
                            l[nt][c] *= a;
                            z[nt][c] *= a;
#pragma unroll
                            for (int u = 0; u < kSteps; ++u) {
                                O[nt][u][c] *= a * rs;
                                O[nt][u][2 + c] *= a * rs;
                            }
                            m[nt][c] = mx[nt][c];
                        }
                    r_exp = r_new;
                }
                const float cr = pow2f(14 - r_exp);
                // ---- weights and O^T
#pragma unroll
                for (int sub = 0; sub < kSub; ++sub) {
                    uint32_t wb[NT][2];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const float p0 = fast_exp2(S[sub][nt][2 * r] - m[nt][0]);
                            const float p1 = fast_exp2(S[sub][nt][2 * r + 1] - m[nt][1]);
                            l[nt][0] += p0;
                            l[nt][1] += p1;
                            z[nt][0] = fmaf(p0, vz[sub][r], z[nt][0]);
                            z[nt][1] = fmaf(p1, vz[sub][r], z[nt][1]);
                            const float v = vs[sub][r] * cr;
                            wb[nt][r] = transpose8x8(pack_half2(p0 * v, p1 * v));
                        }
                    // this lane's bytes of tokens 2 lj, 2 lj + 1, 2 lj + 8, 2 lj + 9
                    const unsigned char *vr = slot + C::kOffV + (sub * 16 + 2 * lj) * C::kRow + li * (D / 16);
                    uint32_t v0[D / 64], v1[D / 64], v2[D / 64], v3[D / 64];
                    if constexpr (D == 128) {
                        *reinterpret_cast<uint2 *>(v0) = *reinterpret_cast<const uint2 *>(vr);
                        *reinterpret_cast<uint2 *>(v1) = *reinterpret_cast<const uint2 *>(vr + C::kRow);
                        *reinterpret_cast<uint2 *>(v2) = *reinterpret_cast<const uint2 *>(vr + 8 * C::kRow);
                        *reinterpret_cast<uint2 *>(v3) = *reinterpret_cast<const uint2 *>(vr + 9 * C::kRow);
                    } else {
                        v0[0] = *reinterpret_cast<const uint32_t *>(vr);
                        v1[0] = *reinterpret_cast<const uint32_t *>(vr + C::kRow);
                        v2[0] = *reinterpret_cast<const uint32_t *>(vr + 8 * C::kRow);
                        v3[0] = *reinterpret_cast<const uint32_t *>(vr + 9 * C::kRow);
                    }
                    // piece h: the h-th 16 bits (4 channels) of the lane's bytes, of two tokens
                    constexpr int H = D / 32;
                    uint32_t x01[H], x23[H];
#pragma unroll
                    for (int h = 0; h < H; ++h) {
                        const uint32_t sel = h & 1 ? 0x7632u : 0x5410u;
                        x01[h] = __byte_perm(v0[h / 2], v1[h / 2], sel);
                        x23[h] = __byte_perm(v2[h / 2], v3[h / 2], sel);
                    }
#pragma unroll
                    for (int h = 0; h < H / 2; ++h)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t mask = e & 1 ? 0x00F000F0u : 0x000F000Fu;
                            const int sh = e >= 2 ? 8 : 0;
                            const uint32_t a0 = (x01[h] >> sh) & mask, a1 = (x01[h + H / 2] >> sh) & mask;
                            const uint32_t a2 = (x23[h] >> sh) & mask, a3 = (x23[h + H / 2] >> sh) & mask;
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) mma16816(O[nt][4 * h + e], a0, a1, a2, a3, wb[nt][0], wb[nt][1]);
                        }
                }
                __syncwarp();                          // every lane has read the slot
                held = used % kStages;
                if (s + kWarps < ns) fetch_one();
            }
        }
        // ---- join the warps: each leaves its (max, sum) pairs and its output, in the units
        // of the result, in the slot that it read last
        if (s0 < ns && ok) {
            float *buf = reinterpret_cast<float *>(ring + held * C::kSlot);
            const float even = pow2f(r_exp + 10), odd = pow2f(r_exp + 6);   // 2^(r_exp - 14) 2^24, / 16
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float ls = rows_sum(l[nt][c]), zs = rows_sum(z[nt][c]);
                    const int g = nt * 8 + 2 * lj + c;
                    if (li == 0) ml_s[warp * GT + g] = make_float2(m[nt][c], ls);
                    // channels of rows li: li * D / 8 + u, of rows li + 8: D / 16 further
                    float *dst = buf + g * C::kPad + li * (D / 8);
#pragma unroll
                    for (int r = 0; r < 2; ++r)
#pragma unroll
                        for (int u = 0; u < kSteps; u += 4) {
                            float4 v;
                            v.x = fmaf(O[nt][u][2 * r + c], even, zs);
                            v.y = fmaf(O[nt][u + 1][2 * r + c], odd, zs);
                            v.z = fmaf(O[nt][u + 2][2 * r + c], even, zs);
                            v.w = fmaf(O[nt][u + 3][2 * r + c], odd, zs);
                            *reinterpret_cast<float4 *>(dst + r * (D / 16) + u) = v;
                        }
                }
            fence_proxy_async_smem();                  // the slot is fetched into again below
        }
        if (lane == 0) held_s[warp] = s0 < ns && ok ? (int)held : -1;
        __syncthreads();
        for (int i = tid; i < G * D; i += kThreads) {
            const int g = i / D, d = i % D;
            float M = -INFINITY, L = 0.f, A = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                if (held_s[w] >= 0) M = fmaxf(M, ml_s[w * GT + g].x);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const int h = held_s[w];
                if (h < 0) continue;
                const float2 v = ml_s[w * GT + g];
                const float f = v.x == -INFINITY ? (v.y == v.y ? 0.f : v.y) : fast_exp2(v.x - M);
                L = fmaf(v.y, f, L);
                A = fmaf(reinterpret_cast<const float *>(smem + (w * kStages + h) * C::kSlot)[g * C::kPad + d], f, A);
            }
            const int64_t r = (head0 + g) * p.max_partitions + I.slot;
            if (I.direct) out[(head0 + g) * D + d] = Elem<T>::from_f(A / L);
            else p.ws_o[r * D + d] = A;
            if (d == 0) {
                if (!I.direct) reinterpret_cast<float2 *>(p.ws_ml)[r] = make_float2(M, L);
                if constexpr (kScore) reinterpret_cast<float2 *>(p.ws_score_ml)[r] = make_float2(M, L);
            }
        }
        __syncthreads();
        if (s0 < ns && ok) fetch_one();
    }
    if (!ok) {
        *abort_flag = 1;
        raise_error(p.err, PA_DEVERR_WAIT);
        // copies still in flight land before the CTA's shared memory goes away
        for (uint32_t j = used; j != issued; ++j) mbar_wait(&full[j % kStages], (j / kStages) & 1);
    }
}

template <typename T, int D, int GT, bool kScore>
int launch_t(const DecodeParams &p, cudaStream_t stream) {
    using C = Cfg<D, GT>;
    auto kern = decode_int4_kernel<T, D, GT, kScore>;
    static bool attr_set[kMaxDevices] = {};
    static int num_sms[kMaxDevices] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return -1;
    if (!attr_set[dev]) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess) return -1;
        if (cudaDeviceGetAttribute(&num_sms[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return -1;
        attr_set[dev] = true;
    }
    const int64_t max_items = (int64_t)p.num_seqs * p.num_kv_heads * p.max_partitions;
    const int64_t slots = (int64_t)C::kCtas * num_sms[dev];
    return launch_pdl(kern, dim3((unsigned)(max_items < slots ? max_items : slots)), dim3(kThreads), C::kSmem, stream,
                      p);
}

template <typename T, int D> int launch_g(const DecodeParams &p, cudaStream_t stream) {
    if (p.ws_logits) return p.group <= 8 ? launch_t<T, D, 8, true>(p, stream) : launch_t<T, D, 16, true>(p, stream);
    return p.group <= 8 ? launch_t<T, D, 8, false>(p, stream) : launch_t<T, D, 16, false>(p, stream);
}

template <typename T> int launch_d(const DecodeParams &p, cudaStream_t stream) {
    return p.head_dim == 128 ? launch_g<T, 128>(p, stream) : launch_g<T, 64>(p, stream);
}

}  // namespace

bool decode_int4_supported(const DecodeParams &p, int dtype) {
    return (dtype == PA_DTYPE_BF16 || dtype == PA_DTYPE_F16) && (p.head_dim == 64 || p.head_dim == 128) &&
           p.group >= 1 && p.group <= 16 && p.block_size >= 8 && p.block_size <= 256 &&
           p.partition_size % decode_order::kTile == 0 && p.num_blocks < INT32_MAX &&
           (int64_t)p.num_seqs * p.num_heads < INT32_MAX;
}

// Batches above kMaxSeqs sequences run as independent launches of up to kMaxSeqs.
int launch_decode_int4(const DecodeParams &p, int dtype, cudaStream_t stream) {
    if (!decode_int4_supported(p, dtype)) return -2;
    // sequences per launch: at most kMaxSeqs, and few enough that no CTA gets more
    // than the item table holds (items <= num_seqs * kv heads * partitions)
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return -1;
    const int64_t per_seq = (int64_t)p.num_kv_heads * p.max_partitions;
    const int64_t by_items = (int64_t)decode_order::kTableItems * (p.group <= 8 ? 2 : 1) * sms / per_seq;
    const int chunk = (int)(by_items < 1 ? 1 : (by_items < kMaxSeqs ? by_items : kMaxSeqs));
    for (int b0 = 0; b0 < p.num_seqs; b0 += chunk) {
        DecodeParams c = p;
        const int64_t rows = (int64_t)b0 * p.num_heads;
        c.num_seqs = min(chunk, p.num_seqs - b0);
        c.q = static_cast<const char *>(p.q) + rows * p.head_dim * 2;
        c.out = static_cast<char *>(p.out) + rows * p.head_dim * 2;
        c.block_tables = p.block_tables + (int64_t)b0 * p.max_blocks_per_seq;
        c.context_lens = p.context_lens + b0;
        if (p.ws_ml) {
            c.ws_ml = p.ws_ml + rows * p.max_partitions * 2;
            c.ws_o = p.ws_o + rows * p.max_partitions * p.head_dim;
        }
        if (p.ws_logits) {
            c.ws_logits = p.ws_logits + rows * p.logits_len;
            c.ws_score_ml = p.ws_score_ml + rows * p.max_partitions * 2;
        }
        const int rc = dtype == PA_DTYPE_BF16 ? launch_d<__nv_bfloat16>(c, stream) : launch_d<__half>(c, stream);
        if (rc != 0) return rc;
    }
    return 0;
}

}  // namespace pa
