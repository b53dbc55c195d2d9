// Internal launch interface of a serving step's preparation (block tables and slot maps from
// the requests' lengths, rotary positions), between the C-ABI layer (capi.cu) and its kernel
// translation units. Not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace pa {

// Requests of a step that the layout kernels hold in shared memory.
constexpr int kMaxLayoutSeqs = 16384;

struct BlocksAppendParams {
    int32_t *block_tables;           // [num_seqs, max_blocks]
    const int32_t *context_lens;
    int32_t *new_context_lens;       // may be context_lens
    const int32_t *query_lens;
    const int32_t *free_blocks;      // [free_cap]
    const int32_t *num_free;
    int32_t *new_num_free;           // may be num_free
    int32_t *query_start_loc;        // [num_seqs + 1]
    int32_t *slot_mapping;           // [num_tokens]
    int32_t *positions;              // [num_tokens]
    unsigned int *err;
    int64_t num_blocks, table_tokens;   // table_tokens: max_blocks * block_size
    int num_seqs, max_blocks, free_cap, num_tokens, log2_block_size;
};
int launch_blocks_append(const BlocksAppendParams &p, int sms, cudaStream_t stream);

struct BlocksReleaseParams {
    const int32_t *block_tables;
    const int32_t *context_lens;
    int32_t *new_context_lens;       // may be context_lens
    const uint8_t *finished;
    int32_t *free_blocks;
    const int32_t *num_free;
    int32_t *new_num_free;           // may be num_free
    unsigned int *err;
    int64_t num_blocks, table_tokens;
    int num_seqs, max_blocks, free_cap, log2_block_size;
};
int launch_blocks_release(const BlocksReleaseParams &p, cudaStream_t stream);

// Rotary positions of the queries and keys of num_tokens tokens: row t of x at x + t * x_stride
// elements, its heads contiguous. With slots, K goes to its slot of the cache k_out
// [slots][num_kv_heads][head_dim] and v, as it is, to that of v_out; without, to row t of k_out
// (strided), and there is no v.
struct RotaryParams {
    const void *q, *k, *v;
    void *q_out, *k_out, *v_out;
    int64_t q_stride, k_stride, v_stride, q_out_stride, k_out_stride;
    const int32_t *positions;
    const double *inv_freq;          // [rotary_dim / 2]
    const int32_t *slots;
    unsigned int *err;
    int64_t num_tokens, num_slots;
    float factor;
    int num_heads, num_kv_heads, head_dim, rotary_dim;
    int interleaved;
};
int launch_rotary(const RotaryParams &p, int dtype, cudaStream_t stream);

}  // namespace pa
