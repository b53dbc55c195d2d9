// Internal launch interface of the 8-bit cache with a scale for each block of tokens and kv
// head, between the C-ABI layer (capi.cu) and its kernel translation units. Not part of the
// public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kernels_compress.h"

namespace pa {

// E4M3 codes [num_blocks, num_kv_heads, block_size, head_dim] for K and V, and scales
// float32 [num_blocks, num_kv_heads, 2] = (K scale, V scale).
struct Fp8BlockCache {
    void *key;
    void *value;
    float2 *scales;
    int64_t num_slots;         // num_blocks * block_size
    int num_kv_heads;
    int head_dim;              // 64 or 128
    int log2_block_size;
};

// k, v: rows of token t at k + t * k_stride elements. sms: the device's multiprocessors.
int launch_kv_write_fp8_block(const void *k, const void *v, int64_t k_stride, int64_t v_stride, int src_dtype,
                              const int32_t *slot_mapping, int64_t num_tokens, const Fp8BlockCache &c,
                              int sms, unsigned int *err, cudaStream_t stream);
int launch_kv_read_fp8_block(void *k, void *v, int dst_dtype, const int32_t *slot_mapping, int64_t num_tokens,
                             const Fp8BlockCache &c, int sms, unsigned int *err, cudaStream_t stream);
int launch_copy_scales_fp8_block(float2 *scales, const int32_t *pairs, int64_t num_pairs, int64_t num_blocks,
                                 int num_kv_heads, unsigned int *err, cudaStream_t stream);

// Decode attention over such a cache (p.key_cache, p.value_cache, p.kv_params: the scales) of
// contexts up to max_ctx tokens, on `sms` multiprocessors; p's split-K fields are not used.
bool decode_fp8_block_supported(const DecodeParams &p, int dtype);
RunWorkSizes decode_fp8_block_work_sizes(int64_t num_seqs, int64_t num_heads, int64_t num_kv_heads, int64_t head_dim,
                                         int64_t max_ctx, int sms);
int launch_decode_fp8_block(const DecodeParams &p, const RunWork &ws, int64_t max_ctx, int sms, int dtype,
                            cudaStream_t stream);

}  // namespace pa
