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
constexpr int kChunk = 4096;            // tokens per CTA: the joining of the pairs is amortised over them
constexpr int kMaxG = 16;

template <int VEC>
__global__ __launch_bounds__(kThreads) void decode_mass_kernel(const DecodeParams p, float *__restrict__ mass,
                                                               int64_t mass_len) {
    __shared__ float M_s[kMaxG], inv_s[kMaxG];
    const int kvh = blockIdx.y, b = blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = p.group;
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int ctx = p.context_lens[b];
    ctx = ctx < 0 ? 0 : min(ctx, p.context_limit);
    const int64_t c0 = (int64_t)blockIdx.x * kChunk;
    if (c0 >= ctx) return;
    const int nparts = (ctx - 1) / p.partition_size + 1;
    for (int g = warp; g < G; g += kThreads / 32) {
        const float2 *ml = reinterpret_cast<const float2 *>(p.ws_score_ml) +
                           ((int64_t)b * p.num_heads + (int64_t)kvh * G + g) * p.max_partitions;
        float M = -INFINITY;
        for (int i = lane; i < nparts; i += 32) M = fmaxf(M, ml[i].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        float L = 0.f;
        for (int i = lane; i < nparts; i += 32) {
            const float2 v = ml[i];
            L = fmaf(v.y, v.x == -INFINITY ? 0.f : fast_exp2(v.x - M), L);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
        if (lane == 0) {
            M_s[g] = M;
            inv_s[g] = 1.f / L;
        }
    }
    __syncthreads();
    const float *x = p.ws_logits + ((int64_t)b * p.num_kv_heads + kvh) * p.logits_len * G;
    float *dst = mass + ((int64_t)b * p.num_kv_heads + kvh) * mass_len;
    const int t1 = (int)min((int64_t)ctx, c0 + kChunk);
    for (int t = (int)c0 + threadIdx.x; t < t1; t += kThreads) {
        float w = 0.f;
        for (int g = 0; g < G; g += VEC) {
            float v[VEC];
            if constexpr (VEC == 4) {
                const float4 f = __ldcs(reinterpret_cast<const float4 *>(x + (int64_t)t * G + g));
                v[0] = f.x;
                v[1] = f.y;
                v[2] = f.z;
                v[3] = f.w;
            } else {
                v[0] = __ldcs(x + (int64_t)t * G + g);
            }
#pragma unroll
            for (int u = 0; u < VEC; ++u) w = fmaf(fast_exp2(v[u] - M_s[g + u]), inv_s[g + u], w);
        }
        dst[t] += w;
    }
}

}  // namespace

int launch_decode_mass(const DecodeParams &p, float *mass, int64_t mass_len, cudaStream_t stream) {
    if (p.context_limit <= 0) return 0;
    const dim3 grid((unsigned)((p.context_limit + kChunk - 1) / kChunk), (unsigned)p.num_kv_heads,
                    (unsigned)p.num_seqs);
    if (p.group % 4 == 0)
        return launch_pdl(decode_mass_kernel<4>, grid, dim3(kThreads), 0, stream, p, mass, mass_len);
    return launch_pdl(decode_mass_kernel<1>, grid, dim3(kThreads), 0, stream, p, mass, mass_len);
}

}  // namespace pa
