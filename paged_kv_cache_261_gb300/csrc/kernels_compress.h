// Internal launch interface of the cache-compression operators (4-bit cache,
// accumulated attention weights, eviction), between the C-ABI layer (capi.cu) and
// their kernel translation units. Not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kernels.h"

namespace pa {

// A 4-bit paged cache: codes [num_blocks, num_kv_heads, block_size, head_dim / 2]
// for K and V, and params float16 [num_blocks, num_kv_heads, block_size, 4].
struct Int4Cache {
    void *key;
    void *value;
    void *params;
    int64_t num_slots;         // num_blocks * block_size
    int num_kv_heads;
    int head_dim;              // 64 or 128
    int log2_block_size;
};

int launch_kv_write_int4(const void *k, const void *v, int src_dtype, const int32_t *slot_mapping,
                         int64_t num_tokens, const Int4Cache &c, unsigned int *err, cudaStream_t stream);
int launch_kv_read_int4(void *k, void *v, int dst_dtype, const int32_t *slot_mapping, int64_t num_tokens,
                        const Int4Cache &c, unsigned int *err, cudaStream_t stream);
int launch_copy_params_int4(void *params, const int32_t *pairs, int64_t num_pairs, int64_t num_blocks,
                            int64_t block_bytes, unsigned int *err, cudaStream_t stream);

// Tokens per stage of the 4-bit decode, and warps of its CTAs (one per SM) by the padded
// group, 8 or 16: as many as the registers allow.
constexpr int kInt4StageTokens = 64;
__host__ __device__ constexpr int kInt4Warps(int gt) { return gt == 8 ? 12 : 8; }

// Workspace of the partials of a decode whose work is cut into equal runs (decode_runs.cuh).
struct RunWork {
    int2 *rows;                // [sequence][kv head] of a launch: first partial, how many
    float2 *part_ml;           // [partial][head of the group]: reference (log2 units), sum
    float *part_o;             // [partial][head of the group][head_dim]
};
struct RunWorkSizes {
    size_t rows, part_ml, part_o;
};
RunWorkSizes decode_int4_work_sizes(int64_t num_seqs, int64_t num_heads, int64_t num_kv_heads, int64_t head_dim,
                                     int64_t max_ctx, int sms);

// Decode attention over a 4-bit cache (p.key_cache, p.value_cache, p.kv_params) of contexts
// up to max_ctx tokens, on `sms` multiprocessors; p's split-K fields are not used. With mass
// set, p.ws_logits and p.ws_score_ml hold the scores and the pairs of rows that one run
// covers, and the weights are added to mass as by launch_decode_mass.
bool decode_int4_supported(const DecodeParams &p, int dtype);
int launch_decode_int4(const DecodeParams &p, const RunWork &ws, int64_t max_ctx, int sms, float *mass,
                       int64_t mass_len, int dtype, cudaStream_t stream);

// Adds each token's softmax weights, summed over the query heads of its kv head, to
// mass [num_seqs, num_kv_heads, mass_len], from the scores (planes of heads_per_plane) and
// (max, sum) pairs that a decode with p.ws_logits left in the workspace. ws: of a 4-bit decode,
// whose joining kernel is the one before on the stream.
int launch_decode_mass(const DecodeParams &p, int heads_per_plane, float *mass, int64_t mass_len, const RunWork *ws,
                       cudaStream_t stream);
// Heads per plane of the kernels: SIMT 1, 4-bit 2, and half the padded group here.
inline int score_plane_tc(int group) { return group <= 4 ? 2 : (group <= 8 ? 4 : 8); }

// One array of rows that an eviction moves: row of (block, offset, kv head) at
// base + block * block_stride + offset * token_stride + head * head_stride.
struct EvictPlane {
    char *base;
    int64_t block_stride, token_stride, head_stride;
    int row_bytes;             // a multiple of 16
    // 4-bit caches: where this array's halves (scale and zero, 4 of 8 bytes) of the parameters
    // are, which lie as the rows do, 1 / 2^side_shift as far apart
    char *side;
    int side_shift;
};

struct EvictParams {
    int32_t *kept;             // [num_seqs, num_kv_heads, kept_len]
    const float *mass;         // [num_seqs, num_kv_heads, mass_len]
    float *mass_out;           // [num_seqs, num_kv_heads, mass_out_len]
    const int32_t *block_tables;
    const int32_t *out_block_tables;
    const int32_t *context_lens;
    const int32_t *keep_lens;
    unsigned int *err;
    int64_t kept_len, mass_len, mass_out_len, num_blocks;
    int max_blocks, out_max_blocks;
    int context_limit;         // tokens the table and mass hold
    int keep_limit;            // tokens the out table, mass_out and kept hold
    int num_seqs, num_kv_heads;
    int log2_block_size;
    int recent;
    EvictPlane planes[2];      // K and V
};
int launch_evict(const EvictParams &p, int sms, cudaStream_t stream);

}  // namespace pa
