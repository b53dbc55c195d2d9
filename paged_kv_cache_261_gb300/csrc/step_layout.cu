// Block tables and slot maps of a serving step, from the requests' lengths, on the GPU.
//
// The rules are the block manager's: a new block only when a token starts one ("CS349E lecture
// 7: 01_paged_attention.py" demo 1), free ids on a stack whose top is taken
// ("PagedAttention实现" §PagedAttention管理器), slot = block * block_size + offset and packed
// queries with their start locations ("04 - Paged Attention 实现进度" B.2). Here the stack is a
// device array and its height a device integer, so a step needs no answer from the host.
//
// Request b with c tokens held and n new ones needs ceil((c + n) / bs) - ceil(c / bs) blocks; with
// E the sum of the needs before it, its j-th new block is free[num_free - 1 - (E + j)]: the order
// in which requests served one after another would have popped them. Two prefix sums over the
// requests (rows and needs) are all that connects the requests.
//
// Every CTA takes the sums over all requests by itself (they are few), and the tokens and blocks
// are dealt among all threads; a token finds its request by a binary search of the sums in shared
// memory. The new lengths may be written over the old, so their writer has to come after every
// reader: one cluster does a whole call, its barrier between the two, or, where there are many
// tokens, a second launch of one CTA takes the sums again and writes the lengths.
// What bounds it is latency: a chain of loads, the sums, a barrier, a search, loads and stores.
#include "common.cuh"
#include "kernels_step.h"

#include <algorithm>

namespace pa {
namespace {

constexpr int kMaxThreads = 1024;
constexpr int kMaxCluster = 8;
constexpr int kScratch = 66;                     // 64-bit words of the sums
constexpr int kPerThread = 4;                    // table entries of a thread that a release aims at
// An append's tokens that one cluster takes: up to about here its single launch is as fast as the two
// (us on the device: 68 tokens 3.4; 1500 of 300 requests 6.5 against 4.4, 4000 of four 5.6 against 3.7).
constexpr int kClusterTokens = 512;
// Threads of a CTA. Many are slow to start and to agree: maps of 17,500 tokens with 256 3.9 us, 512 4.5,
// 1024 6.4; lengths after 139,000 tokens of 1024 requests with 256 6.4 (the call), 1024 8.2; a release of
// 64 requests with 256 2.8, 512 3.1, 1024 4.2, of 1024 requests 5.1, 4.3, 5.0.
// (More where there are many requests: no thread sums up more than kPerThread of them, or they are 1024.)
constexpr int kCallThreads = 512, kMapThreads = 256, kLengthThreads = 256;
constexpr int kMapCtas = 2;                      // on an SM, at most

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Exclusive prefix sums over the CTA of each thread's (a, b), and the totals. scratch: kScratch
// words, the last two untouched.
struct Sums {
    int64_t a, b;
};
__device__ __forceinline__ Sums prefix_sums(Sums mine, int64_t *scratch, Sums &total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    Sums inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t a = __shfl_up_sync(0xffffffffu, inc.a, o), b = __shfl_up_sync(0xffffffffu, inc.b, o);
        if (lane >= o) {
            inc.a += a;
            inc.b += b;
        }
    }
    if (lane == 31) {
        scratch[2 * warp] = inc.a;
        scratch[2 * warp + 1] = inc.b;
    }
    __syncthreads();
    total = {0, 0};
    Sums before{0, 0};
    for (int w = 0; w < warps; ++w) {
        if (w == warp) before = total;
        total.a += scratch[2 * w];
        total.b += scratch[2 * w + 1];
    }
    return {before.a + inc.a - mine.a, before.b + inc.b - mine.b};
}

// The last b in [0, n) with first[b] <= x, for ascending first with first[0] <= x.
__device__ __forceinline__ int owner(const int *first, int n, int x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// num_free, or 0 with an error where it cannot be the height of the stack: which of its entries are free is
// not known then, so it counts as empty.
__device__ __forceinline__ int stack_height(const int32_t *num_free, int cap, bool report, unsigned int *err) {
    const int n = *num_free;
    if (n >= 0 && n <= cap) return n;
    if (report) raise_error(err, PA_DEVERR_FREE_BLOCKS);
    return 0;
}

// A table entry that names a block, or -1 with an error.
__device__ __forceinline__ int checked_block(int entry, int64_t num_blocks, unsigned int *err) {
    if (entry >= 0 && entry < num_blocks) return entry;
    raise_error(err, PA_DEVERR_BLOCK_ID);
    return -1;
}

// What a launch of blocks_append_kernel does: a whole call by one cluster; all of a call but the
// lengths and the stack's height, by any number of CTAs; or these two, after such a launch.
enum class Append { kCall, kMaps, kLengths };

template <Append kWhat>
__global__ __launch_bounds__(kMaxThreads) void blocks_append_kernel(const BlocksAppendParams p) {
    extern __shared__ __align__(16) unsigned char smem[];
    int64_t *scratch = reinterpret_cast<int64_t *>(smem);
    int *all_taken = reinterpret_cast<int *>(scratch + kScratch - 2);  // blocks that the call takes
    int *start = reinterpret_cast<int *>(scratch + kScratch);          // [B + 1] rows before a request
    int *taken = start + p.num_seqs + 1;                               // [B] blocks needed before it
    int *ctx = taken + p.num_seqs;                                     // [B] tokens held, -1: not served
    // No early signal but to the second launch of a call: a decode launched next reads the new
    // lengths before it waits. That second launch reads what was there before the call, and
    // waits before it writes.
    if constexpr (kWhat != Append::kLengths) asm volatile("griddepcontrol.wait;" ::: "memory");
    if constexpr (kWhat == Append::kMaps) asm volatile("griddepcontrol.launch_dependents;");
    const int B = p.num_seqs, T = p.num_tokens, l2 = p.log2_block_size, bs = 1 << l2;
    const uint32_t gid = blockIdx.x * blockDim.x + threadIdx.x, threads = gridDim.x * blockDim.x;
    const bool report = blockIdx.x == 0 && kWhat != Append::kLengths;
    if (threadIdx.x == 0) *all_taken = 0;
    const int height = stack_height(p.num_free, p.free_cap, report && threadIdx.x == 0, p.err);

    const int per = (B + blockDim.x - 1) / blockDim.x;
    const int b0 = min(B, (int)threadIdx.x * per), b1 = min(B, b0 + per);
    // rows and blocks of a request; one whose lengths are out of range needs none
    auto request = [&](int b, int &c, Sums &s) {
        c = p.context_lens[b];
        const int n = p.query_lens[b];
        const bool good = c >= 0 && n >= 0 && (int64_t)c + n <= p.table_tokens;
        s.a = max(n, 0);
        s.b = good ? (((int64_t)c + n + bs - 1) >> l2) - (((int64_t)c + bs - 1) >> l2) : 0;
        return good;
    };
    Sums mine{0, 0}, total;
    for (int b = b0; b < b1; ++b) {
        int c;
        Sums s;
        request(b, c, s);
        mine.a += s.a;
        mine.b += s.b;
    }
    Sums at = prefix_sums(mine, scratch, total);
    unsigned int bits = 0;
    int mine_taken = 0;
    for (int b = b0; b < b1; ++b) {
        int c;
        Sums s;
        bool good = request(b, c, s);
        start[b] = (int)min(at.a, (int64_t)T);
        taken[b] = (int)min(at.b, (int64_t)height);
        at.a += s.a;
        at.b += s.b;
        if (!good || (s.a > 0 && at.a > T)) {
            good = false;
            bits |= PA_DEVERR_CONTEXT;
        } else if (s.b > 0 && at.b > height) {
            good = false;                        // and so is every later one that needs a block
            bits |= PA_DEVERR_FREE_BLOCKS;
        } else if (s.b > 0) {
            mine_taken = (int)at.b;
        }
        ctx[b] = good ? c : -1;
    }
    if (threadIdx.x == 0) start[B] = (int)min(total.a, (int64_t)T);
    mine_taken = __reduce_max_sync(0xffffffffu, mine_taken);
    bits = __reduce_or_sync(0xffffffffu, bits);
    if ((threadIdx.x & 31) == 0) {
        if (mine_taken) atomicMax(all_taken, mine_taken);
        if (report && bits) raise_error(p.err, bits);
    }
    __syncthreads();
    // every CTA that reads the lengths and the height has done so
    if constexpr (kWhat == Append::kCall) cluster_sync();
    if constexpr (kWhat == Append::kLengths) asm volatile("griddepcontrol.wait;" ::: "memory");

    if constexpr (kWhat != Append::kMaps) {
        for (int b = gid; b < B; b += threads)
            p.new_context_lens[b] = ctx[b] >= 0 ? ctx[b] + start[b + 1] - start[b] : p.context_lens[b];
        if (gid == 0) *p.new_num_free = height - *all_taken;
    }
    if constexpr (kWhat != Append::kLengths) {
        for (int b = gid; b <= B; b += threads) p.query_start_loc[b] = start[b];
        // the entries of the blocks taken
        for (int j = gid; j < *all_taken; j += threads) {
            const int b = owner(taken, B, j), col = ((ctx[b] + bs - 1) >> l2) + j - taken[b];
            p.block_tables[(int64_t)b * p.max_blocks + col] = checked_block(p.free_blocks[height - 1 - j], p.num_blocks, p.err);
        }
        // Slots and positions, a token a thread. (Four tokens in a row a thread, with one search and vector
        // stores where they share a request: 10.2 us against 7.5 for 139,000 tokens of 1024 requests, 6.6
        // against 4.7 for 17,500 of 192.)
        const int live = start[B];
        for (int t = gid; t < T; t += threads) {       // (T is at most 2^30)
            int slot = -1, pos = 0;
            if (t < live) {
                const int b = owner(start, B, t), c = ctx[b];
                if (c >= 0) {
                    pos = c + t - start[b];
                    const int held = (c + bs - 1) >> l2, col = pos >> l2;
                    const int entry = col < held ? p.block_tables[(int64_t)b * p.max_blocks + col]
                                                 : p.free_blocks[height - 1 - (taken[b] + col - held)];
                    const int block = checked_block(entry, p.num_blocks, p.err);
                    if (block >= 0) slot = (block << l2) + (pos & (bs - 1));
                }
            }
            p.slot_mapping[t] = slot;
            p.positions[t] = pos;
        }
    }
}

__global__ __launch_bounds__(kMaxThreads) void blocks_release_kernel(const BlocksReleaseParams p) {
    extern __shared__ __align__(16) unsigned char smem[];
    int64_t *scratch = reinterpret_cast<int64_t *>(smem);
    int *all_back = reinterpret_cast<int *>(scratch + kScratch - 2);   // blocks given back
    int *back = reinterpret_cast<int *>(scratch + kScratch);           // [B] blocks given back before a request
    int *ctx = back + p.num_seqs;                                      // [B] its new length
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int B = p.num_seqs, l2 = p.log2_block_size, bs = 1 << l2;
    const uint32_t gid = blockIdx.x * blockDim.x + threadIdx.x, threads = gridDim.x * blockDim.x;
    const bool report = blockIdx.x == 0;
    if (threadIdx.x == 0) *all_back = 0;
    const int height = stack_height(p.num_free, p.free_cap, report && threadIdx.x == 0, p.err);
    const int room = p.free_cap - height;

    const int per = (B + blockDim.x - 1) / blockDim.x;
    const int b0 = min(B, (int)threadIdx.x * per), b1 = min(B, b0 + per);
    auto request = [&](int b, int &c, Sums &s) {
        c = p.context_lens[b];
        const bool good = c >= 0 && c <= p.table_tokens;
        s.a = 0;
        s.b = p.finished[b] && good ? ((int64_t)c + bs - 1) >> l2 : 0;
        return good;
    };
    Sums mine{0, 0}, total;
    for (int b = b0; b < b1; ++b) {
        int c;
        Sums s;
        request(b, c, s);
        mine.b += s.b;
    }
    Sums at = prefix_sums(mine, scratch, total);
    unsigned int bits = 0;
    int mine_back = 0;
    for (int b = b0; b < b1; ++b) {
        int c;
        Sums s;
        const bool good = request(b, c, s);
        back[b] = (int)min(at.b, (int64_t)room);
        at.b += s.b;
        if (p.finished[b]) {
            if (!good) {
                bits |= PA_DEVERR_CONTEXT;
            } else if (at.b > room && s.b > 0) {
                bits |= PA_DEVERR_FREE_BLOCKS;   // and so is every later one that holds a block
            } else {
                c = 0;
                if (s.b > 0) mine_back = (int)at.b;
            }
        }
        ctx[b] = c;
    }
    mine_back = __reduce_max_sync(0xffffffffu, mine_back);
    bits = __reduce_or_sync(0xffffffffu, bits);
    if ((threadIdx.x & 31) == 0) {
        if (mine_back) atomicMax(all_back, mine_back);
        if (report && bits) raise_error(p.err, bits);
    }
    __syncthreads();
    cluster_sync();                              // every CTA has read the lengths and the height

    for (int b = gid; b < B; b += threads) p.new_context_lens[b] = ctx[b];
    if (gid == 0) *p.new_num_free = height + *all_back;
    for (int j = gid; j < *all_back; j += threads) {
        const int b = owner(back, B, j);
        p.free_blocks[height + j] =
            checked_block(p.block_tables[(int64_t)b * p.max_blocks + j - back[b]], p.num_blocks, p.err);
    }
}

// Launch of `ctas` CTAs, as one cluster or none.
template <typename P>
int launch(void (*kern)(P), const P &p, int ctas, int threads, bool cluster, int words, cudaStream_t stream) {
    const size_t smem = kScratch * 8 + (size_t)words * 4;
    // (set on every call: the attribute is the device's own)
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return -1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess ? 0 : -1;
}

// Threads of a CTA for this much work and as many requests, up to `most` if the work alone asks.
int cta_threads(int64_t work, int num_seqs, int most) {
    const int64_t want = std::max<int64_t>(std::min<int64_t>(work, most), num_seqs / kPerThread);
    return (int)std::min<int64_t>(kMaxThreads, std::max<int64_t>(128, (want + 127) / 128 * 128));
}
int cluster_ctas(int64_t work, int threads) {
    int ctas = 1;
    while (ctas < kMaxCluster && (int64_t)ctas * threads < work) ctas *= 2;
    return ctas;
}

}  // namespace

int launch_blocks_append(const BlocksAppendParams &p, int sms, cudaStream_t stream) {
    const int T = p.num_tokens, words = 3 * p.num_seqs + 1;
    if (T <= kClusterTokens) {
        const int threads = cta_threads(std::max(T, p.num_seqs), p.num_seqs, kCallThreads);
        return launch(blocks_append_kernel<Append::kCall>, p, cluster_ctas(T, threads), threads, true, words, stream);
    }
    const int threads = cta_threads(T, p.num_seqs, kMapThreads);
    const int64_t ctas = ((int64_t)T + threads - 1) / threads;
    const int rc = launch(blocks_append_kernel<Append::kMaps>, p, (int)std::min<int64_t>(kMapCtas * sms, ctas), threads,
                          false, words, stream);
    if (rc != 0) return rc;
    return launch(blocks_append_kernel<Append::kLengths>, p, 1, cta_threads(p.num_seqs, p.num_seqs, kLengthThreads), false,
                  words, stream);
}

int launch_blocks_release(const BlocksReleaseParams &p, cudaStream_t stream) {
    // a thread for every kPerThread entries that the tables could hold: which requests are
    // finished is known on the device alone
    const int64_t work = ((int64_t)p.num_seqs * p.max_blocks + kPerThread - 1) / kPerThread;
    const int threads = cta_threads(std::max<int64_t>(work, p.num_seqs), p.num_seqs, p.num_seqs > 256 ? 512 : 256);
    return launch(blocks_release_kernel, p, cluster_ctas(work, threads), threads, true, 2 * p.num_seqs, stream);
}

}  // namespace pa
