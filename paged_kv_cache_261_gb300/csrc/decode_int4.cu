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
// One CTA per (partition, kv head, sequence); its warps take tokens in turn, a lane
// holding head_dim / 32 channels of every query head.
#include "common.cuh"
#include "kernels_compress.h"

namespace pa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;

template <typename T, int D, int GT>
__global__ __launch_bounds__(kThreads) void decode_int4_kernel(const DecodeParams p) {
    constexpr int N = D / 32;                            // channels per lane
    __shared__ float m_s[kWarps][GT], l_s[kWarps][GT], o_s[kWarps][GT][D];
    const int part = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = p.group;
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int ctx = p.context_lens[b];
    if (ctx < 0 || ctx > p.context_limit) {
        if (threadIdx.x == 0 && part == 0 && kvh == 0) raise_error(p.err, PA_DEVERR_CONTEXT);
        ctx = ctx < 0 ? 0 : p.context_limit;
    }
    const int nparts = ctx == 0 ? 1 : (ctx + p.partition_size - 1) / p.partition_size;
    if (part >= nparts) return;
    T *out = reinterpret_cast<T *>(p.out);
    const int64_t head0 = (int64_t)b * p.num_heads + (int64_t)kvh * G;
    if (ctx == 0) {
        for (int i = threadIdx.x; i < G * D; i += kThreads) out[head0 * D + i] = Elem<T>::from_f(0.f);
        return;
    }
    const int t0 = part * p.partition_size, t1 = min(ctx, t0 + p.partition_size);
    const T *q = reinterpret_cast<const T *>(p.q);
    float qv[GT][N], qsum[GT], m[GT], l[GT], o[GT][N];
#pragma unroll
    for (int g = 0; g < GT; ++g) {
        qsum[g] = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            qv[g][i] = g < G ? Elem<T>::to_f(q[(head0 + g) * D + lane * N + i]) * p.scale_log2 : 0.f;
            qsum[g] += qv[g][i];
            o[g][i] = 0.f;
        }
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) qsum[g] += __shfl_xor_sync(0xffffffffu, qsum[g], s);
        m[g] = -INFINITY;
        l[g] = 0.f;
    }
    const int32_t *table = p.block_tables + (int64_t)b * p.max_blocks_per_seq;
    const unsigned char *kc = static_cast<const unsigned char *>(p.key_cache);
    const unsigned char *vc = static_cast<const unsigned char *>(p.value_cache);
    const __half2 *par = static_cast<const __half2 *>(p.kv_params);
    for (int t = t0 + warp; t < t1; t += kWarps) {
        const int32_t phys = table[t >> p.log2_block_size];
        uint32_t kw = 0, vw = 0;
        float2 ks = make_float2(0.f, 0.f), vs = ks;      // a bad block id reads as zeros
        if (phys >= 0 && phys < p.num_blocks) {
            const int64_t row = (((int64_t)phys * p.num_kv_heads + kvh) << p.log2_block_size) +
                                (t & (p.block_size - 1));
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                kw |= (uint32_t)kc[row * (D / 2) + lane * (N / 2) + i] << (8 * i);
                vw |= (uint32_t)vc[row * (D / 2) + lane * (N / 2) + i] << (8 * i);
            }
            ks = __half22float2(par[2 * row]);
            vs = __half22float2(par[2 * row + 1]);
        } else if (lane == 0) {
            raise_error(p.err, PA_DEVERR_BLOCK_ID);
        }
#pragma unroll
        for (int g = 0; g < GT; ++g) {
            float x = 0.f;
#pragma unroll
            for (int i = 0; i < N; ++i) x = fmaf(qv[g][i], (float)((kw >> (4 * i)) & 15u), x);
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
            x = fmaf(ks.x, x, ks.y * qsum[g]);
            if (p.ws_logits && lane == 0 && g < G)
                p.ws_logits[(((int64_t)b * p.num_kv_heads + kvh) * p.logits_len + t) * G + g] = x;
            const float m_new = fmaxf(m[g], x);
            const float a = fast_exp2(m[g] - m_new), w = fast_exp2(x - m_new);
            l[g] = fmaf(l[g], a, w);
            m[g] = m_new;
#pragma unroll
            for (int i = 0; i < N; ++i)
                o[g][i] = fmaf(o[g][i], a, w * fmaf((float)((vw >> (4 * i)) & 15u), vs.x, vs.y));
        }
    }
#pragma unroll
    for (int g = 0; g < GT; ++g) {
        if (lane == 0) {
            m_s[warp][g] = m[g];
            l_s[warp][g] = l[g];
        }
#pragma unroll
        for (int i = 0; i < N; ++i) o_s[warp][g][lane * N + i] = o[g][i];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < G * D; i += kThreads) {
        const int g = i / D, d = i % D;
        float M = -INFINITY, L = 0.f, O = 0.f;
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, m_s[w][g]);
        for (int w = 0; w < kWarps; ++w) {
            const float f = m_s[w][g] == -INFINITY ? 0.f : fast_exp2(m_s[w][g] - M);
            L = fmaf(l_s[w][g], f, L);
            O = fmaf(o_s[w][g][d], f, O);
        }
        const int64_t r = (head0 + g) * p.max_partitions + part;
        if (nparts == 1) out[(head0 + g) * D + d] = Elem<T>::from_f(O / L);
        else p.ws_o[r * D + d] = O;
        if (d == 0 && nparts > 1) {
            p.ws_ml[2 * r] = M;
            p.ws_ml[2 * r + 1] = L;
        }
        if (d == 0 && p.ws_logits) {
            p.ws_score_ml[2 * r] = M;
            p.ws_score_ml[2 * r + 1] = L;
        }
    }
}

template <typename T, int D>
int launch_g(const DecodeParams &p, cudaStream_t stream) {
    const dim3 grid((unsigned)p.max_partitions, (unsigned)p.num_kv_heads, (unsigned)p.num_seqs);
    if (p.group <= 1) return launch_pdl(decode_int4_kernel<T, D, 1>, grid, dim3(kThreads), 0, stream, p);
    if (p.group <= 4) return launch_pdl(decode_int4_kernel<T, D, 4>, grid, dim3(kThreads), 0, stream, p);
    if (p.group <= 8) return launch_pdl(decode_int4_kernel<T, D, 8>, grid, dim3(kThreads), 0, stream, p);
    return launch_pdl(decode_int4_kernel<T, D, 16>, grid, dim3(kThreads), 0, stream, p);
}

template <typename T> int launch_d(const DecodeParams &p, cudaStream_t stream) {
    return p.head_dim == 128 ? launch_g<T, 128>(p, stream) : launch_g<T, 64>(p, stream);
}

}  // namespace

bool decode_int4_supported(const DecodeParams &p, int dtype) {
    return (dtype == PA_DTYPE_BF16 || dtype == PA_DTYPE_F16) && (p.head_dim == 64 || p.head_dim == 128) &&
           p.group >= 1 && p.group <= 16 && p.block_size >= 8 && p.block_size <= 256;
}

int launch_decode_int4(const DecodeParams &p, int dtype, cudaStream_t stream) {
    if (!decode_int4_supported(p, dtype)) return -2;
    return dtype == PA_DTYPE_BF16 ? launch_d<__nv_bfloat16>(p, stream) : launch_d<__half>(p, stream);
}

}  // namespace pa
