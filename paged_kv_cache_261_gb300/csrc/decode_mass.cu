// Accumulated attention weights of a decode step.
//
// With x_t the log2-unit scores of query head h and (M, L) the maximum and sum of its
// softmax over the whole context (the partitions' pairs joined: M = max m_p,
// L = sum l_p 2^(m_p - M)), the head's weight of token t is 2^(x_t - M) / L, and
//   mass[b, kvh, t] += sum over the heads of kv head kvh of that weight,
// added in head order, so the result does not depend on timing.
//
// The decode kernels leave the scores (planes of V heads, see kernels.h) and the pairs of
// every partition in the workspace; this kernel reads each score once (4 G bytes per token
// and kv head, next to the 8 of mass itself) and is bound by that traffic.
#include "common.cuh"
#include "kernels_compress.h"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxG = 16;

// Tokens per thread, kThreads apart: their scores (kTok * V * NP floats), and the weights they
// are added to, are read before the heads' (M, L) are joined, which takes two round trips
// itself. (A loop of one token a thread after the join took 22 us on the 8B-shaped batch,
// against 6.)
constexpr int tokens_per_thread(int heads) { return heads <= 2 ? 8 : (heads <= 4 ? 4 : (heads <= 8 ? 2 : 1)); }

// V floats as one load. (All loads here are of L2: beside the joining kernel, nothing has
// made this SM's L1 forget what earlier kernels read.)
template <int V> __device__ __forceinline__ void load_vec(const float *src, float *v) {
    if constexpr (V == 1) {
        v[0] = __ldcg(src);
    } else if constexpr (V == 2) {
        const float2 f = __ldcg(reinterpret_cast<const float2 *>(src));
        v[0] = f.x;
        v[1] = f.y;
    } else {
#pragma unroll
        for (int u = 0; u < V; u += 4) {
            const float4 f = __ldcg(reinterpret_cast<const float4 *>(src + u));
            v[u] = f.x;
            v[u + 1] = f.y;
            v[u + 2] = f.z;
            v[u + 3] = f.w;
        }
    }
}

// NP planes of V heads, of which the first `group` exist.
template <int V, int NP>
__global__ __launch_bounds__(kThreads) void decode_mass_kernel(const DecodeParams p, float *__restrict__ mass,
                                                               int64_t mass_len, int rounds, const RunWork ws) {
    constexpr int kHeads = V * NP, kTok = tokens_per_thread(kHeads);
    constexpr int kChunk = kThreads * kTok;
    __shared__ float M_s[kMaxG], inv_s[kMaxG];
    const int kvh = blockIdx.y, b = blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = p.group;
    // Over a 4-bit cache the kernel before is the one that joins the partials. Nothing here needs
    // its results, and it starts dependents only once the decode has finished, so the two run side
    // by side; this one waits for it at its end, so that whatever follows comes after both.
    const bool beside = ws.rows != nullptr;
    if (!beside) asm volatile("griddepcontrol.wait;" ::: "memory");
    // Over planes of several heads the decode, and so most likely the next call's, is a persistent
    // kernel of one CTA per SM, whose early start pays (8B-shaped batch 114.0 -> 112.2 us, of the
    // 4-bit cache 48.7 -> 47.3). The SIMT decode's CTAs would be packed onto whatever SMs are free
    // first (32 sequences of 8 heads, 1 kv head, head_dim 64: 152.6 us a call against 69.3), and an
    // eviction's are, a little (4-bit decode and eviction 71.3 -> 77.6).
    if constexpr (V > 1) asm volatile("griddepcontrol.launch_dependents;");
    int ctx = p.context_lens[b];
    ctx = ctx < 0 ? 0 : min(ctx, p.context_limit);
    const int64_t c0 = (int64_t)blockIdx.x * rounds * kChunk;
    if (c0 >= ctx) {
        if (beside) asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }
    const float *x = p.ws_logits + ((int64_t)b * p.num_kv_heads + kvh) * p.logits_row;
    float *dst = mass + ((int64_t)b * p.num_kv_heads + kvh) * mass_len;
    int t0 = (int)c0 + threadIdx.x;
    const int end = (int)min((int64_t)ctx, c0 + (int64_t)rounds * kChunk);
    float v[kTok][kHeads], old[kTok];
    auto load = [&]() {
#pragma unroll
        for (int i = 0; i < kTok; ++i) {
            const int t = t0 + i * kThreads;
            if (t >= end) continue;
            old[i] = __ldcg(dst + t);
#pragma unroll
            for (int pl = 0; pl < NP; ++pl)
                if (pl * V < G) load_vec<V>(x + ((int64_t)pl * p.logits_len + t) * V, v[i] + pl * V);
        }
    };
    load();
    // the pairs of a head: of its partitions, or (4-bit) of the runs that share the row, or the
    // one of a row that a run covers
    const int64_t row = (int64_t)b * p.num_kv_heads + kvh;
    const int2 info = beside ? __ldcg(ws.rows + row) : make_int2(0, 0);
    const int nparts = beside ? max(1, info.y) : (ctx - 1) / p.partition_size + 1;
    for (int g = warp; g < G; g += kThreads / 32) {
        const float2 *ml = info.y > 0 ? ws.part_ml + (int64_t)info.x * G + g
                                      : reinterpret_cast<const float2 *>(p.ws_score_ml) + (row * G + g) * p.max_partitions;
        const int64_t step = info.y > 0 ? G : 1;
        float M = -INFINITY, L = 0.f;
        for (int i = lane; i < nparts; i += 32) {       // the lane's own pairs, one pass
            const float2 a = __ldcg(ml + i * step);
            const float m = fmaxf(M, a.x);
            L = L * (M == -INFINITY ? 0.f : fast_exp2(M - m));
            L = fmaf(a.y, a.x == -INFINITY ? (a.y == a.y ? 0.f : a.y) : fast_exp2(a.x - m), L);
            M = m;
        }
        float top = M;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        L *= M == -INFINITY ? 1.f : fast_exp2(M - top);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
        if (lane == 0) {
            M_s[g] = top;
            inv_s[g] = 1.f / L;
        }
    }
    __syncthreads();
    for (;;) {
#pragma unroll
        for (int i = 0; i < kTok; ++i) {
            const int t = t0 + i * kThreads;
            if (t >= end) continue;
            float w = 0.f;
#pragma unroll
            for (int g = 0; g < kHeads; ++g)
                if (g < G) w = fmaf(fast_exp2(v[i][g] - M_s[g]), inv_s[g], w);
            dst[t] = old[i] + w;
        }
        t0 += kChunk;
        if (t0 >= end) break;
        load();
    }
    if (beside) asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <int V, int NP>
int launch_t(const DecodeParams &p, float *mass, int64_t mass_len, const RunWork &ws, cudaStream_t stream) {
    constexpr int chunk = kThreads * tokens_per_thread(V * NP);
    const int64_t chunks = (p.context_limit + chunk - 1) / chunk;
    // a CTA takes several chunks where there are many of them, so that the joining of its heads'
    // pairs is paid less often
    const int64_t all = chunks * p.num_kv_heads * p.num_seqs;
    const int rounds = (int)(all < 2048 ? 1 : (all / 1024 < 8 ? all / 1024 : 8));
    const dim3 grid((unsigned)((chunks + rounds - 1) / rounds), (unsigned)p.num_kv_heads, (unsigned)p.num_seqs);
    return launch_pdl(decode_mass_kernel<V, NP>, grid, dim3(kThreads), 0, stream, p, mass, mass_len, rounds, ws);
}

}  // namespace

int launch_decode_mass(const DecodeParams &p, int heads_per_plane, float *mass, int64_t mass_len, const RunWork *work,
                       cudaStream_t stream) {
    const RunWork ws = work ? *work : RunWork{};
    if (p.context_limit <= 0) return 0;
    const int planes = (p.group + heads_per_plane - 1) / heads_per_plane;
    switch (heads_per_plane) {
    case 1:
        if (planes <= 1) return launch_t<1, 1>(p, mass, mass_len, ws, stream);
        if (planes <= 2) return launch_t<1, 2>(p, mass, mass_len, ws, stream);
        if (planes <= 4) return launch_t<1, 4>(p, mass, mass_len, ws, stream);
        if (planes <= 8) return launch_t<1, 8>(p, mass, mass_len, ws, stream);
        return launch_t<1, 16>(p, mass, mass_len, ws, stream);
    case 2:
        if (planes <= 1) return launch_t<2, 1>(p, mass, mass_len, ws, stream);
        if (planes <= 2) return launch_t<2, 2>(p, mass, mass_len, ws, stream);
        if (planes <= 4) return launch_t<2, 4>(p, mass, mass_len, ws, stream);
        return launch_t<2, 8>(p, mass, mass_len, ws, stream);
    case 4: return launch_t<4, 2>(p, mass, mass_len, ws, stream);
    case 8: return launch_t<8, 2>(p, mass, mass_len, ws, stream);
    default: return -2;
    }
}

}  // namespace pa
