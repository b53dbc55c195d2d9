// Accumulated attention weights of a decode step.
//
// With x_t the log2-unit scores of query head h and (M, L) the maximum and sum of its
// softmax over the whole context (the partitions' pairs joined: M = max m_p,
// L = sum l_p 2^(m_p - M)), the head's weight of token t is 2^(x_t - M) / L, and
//   mass[b, kvh, t] += sum over the heads of kv head kvh of that weight,
// added in head order, so the result does not depend on timing.
//
// The decode kernels leave the scores as [sequence, kv head, token, head] and the pairs
// of every partition in the workspace; this kernel reads each score once (4 G bytes per
// token and kv head, next to the 8 of mass itself) and is bound by that traffic.
#include "common.cuh"
#include "kernels_compress.h"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxG = 16;

// Tokens per thread, kThreads apart: their scores (kTok * G floats), and the weights they are
// added to, are read before the heads' (M, L) are joined, which takes two round trips itself.
// (A loop of one token a thread after the join took 22 us on the 8B-shaped batch, against XX.)
template <int G> struct MassCfg {
    static constexpr int kTok = G <= 4 ? 8 : (G <= 8 ? 4 : 2);
};

// G: heads of the group, or 0: any number, read one score at a time.
template <int G>
__global__ __launch_bounds__(kThreads) void decode_mass_kernel(const DecodeParams p, float *__restrict__ mass,
                                                               int64_t mass_len) {
    constexpr int kTok = MassCfg<G>::kTok;
    constexpr int kChunk = kThreads * kTok;
    __shared__ float M_s[kMaxG], inv_s[kMaxG];
    const int kvh = blockIdx.y, b = blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g_n = G ? G : p.group;
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int ctx = p.context_lens[b];
    ctx = ctx < 0 ? 0 : min(ctx, p.context_limit);
    const int64_t c0 = (int64_t)blockIdx.x * kChunk;
    if (c0 >= ctx) return;
    const float *x = p.ws_logits + ((int64_t)b * p.num_kv_heads + kvh) * p.logits_len * g_n;
    float *dst = mass + ((int64_t)b * p.num_kv_heads + kvh) * mass_len;
    const int t0 = (int)c0 + threadIdx.x;
    float v[kTok][G ? G : 1], old[kTok];
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
        const int t = t0 + i * kThreads;
        if (t >= ctx) continue;
        old[i] = dst[t];
        if constexpr (G % 4 == 0 && G > 0) {
#pragma unroll
            for (int g = 0; g < G; g += 4) {
                const float4 f = __ldcs(reinterpret_cast<const float4 *>(x + (int64_t)t * G + g));
                v[i][g] = f.x;
                v[i][g + 1] = f.y;
                v[i][g + 2] = f.z;
                v[i][g + 3] = f.w;
            }
        } else if constexpr (G > 0) {
#pragma unroll
            for (int g = 0; g < G; ++g) v[i][g] = __ldcs(x + (int64_t)t * G + g);
        }
    }
    const int nparts = (ctx - 1) / p.partition_size + 1;
    for (int g = warp; g < g_n; g += kThreads / 32) {
        const float2 *ml = reinterpret_cast<const float2 *>(p.ws_score_ml) +
                           ((int64_t)b * p.num_heads + (int64_t)kvh * g_n + g) * p.max_partitions;
        float M = -INFINITY, L = 0.f;
        for (int i = lane; i < nparts; i += 32) {       // the lane's own pairs, one pass
            const float2 a = ml[i];
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
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
        const int t = t0 + i * kThreads;
        if (t >= ctx) continue;
        float w = 0.f;
        if constexpr (G > 0) {
#pragma unroll
            for (int g = 0; g < G; ++g) w = fmaf(fast_exp2(v[i][g] - M_s[g]), inv_s[g], w);
        } else {
            for (int g = 0; g < g_n; ++g) w = fmaf(fast_exp2(__ldcs(x + (int64_t)t * g_n + g) - M_s[g]), inv_s[g], w);
        }
        dst[t] = old[i] + w;
    }
}

template <int G> int launch_g(const DecodeParams &p, float *mass, int64_t mass_len, cudaStream_t stream) {
    constexpr int chunk = kThreads * MassCfg<G>::kTok;
    const dim3 grid((unsigned)((p.context_limit + chunk - 1) / chunk), (unsigned)p.num_kv_heads, (unsigned)p.num_seqs);
    return launch_pdl(decode_mass_kernel<G>, grid, dim3(kThreads), 0, stream, p, mass, mass_len);
}

}  // namespace

int launch_decode_mass(const DecodeParams &p, float *mass, int64_t mass_len, cudaStream_t stream) {
    if (p.context_limit <= 0) return 0;
    switch (p.group) {
    case 1: return launch_g<1>(p, mass, mass_len, stream);
    case 2: return launch_g<2>(p, mass, mass_len, stream);
    case 4: return launch_g<4>(p, mass, mass_len, stream);
    case 8: return launch_g<8>(p, mass, mass_len, stream);
    case 16: return launch_g<16>(p, mass, mass_len, stream);
    default: return launch_g<0>(p, mass, mass_len, stream);
    }
}

}  // namespace pa
