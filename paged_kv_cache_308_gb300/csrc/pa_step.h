// Internal interface between the C-ABI layer of block allocation, rotary put and
// linear attention (pa_step_api.cpp) and their kernels (pa_step.cu, pa_linear.cu).
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "pa_internal.h"

namespace pa {

struct KvAllocParams {
    int32_t* tables;
    int32_t* free_blocks;
    const int32_t* count;
    int32_t* new_count;
    const int32_t* held;
    const int32_t* context;
    const int32_t* query;
    int32_t* loc;
    int32_t* lens;
    int32_t* new_held;  // may be null, or held
    int32_t* slots;
    int32_t* positions;
    int num_blocks, num_seqs, num_tokens, cols;
    int place;  // the cluster places the tokens too; else a launch of their own
    unsigned int* status;
};
constexpr int kAllocThreads = 512;
constexpr int kAllocMaxCluster = 8;
// Up to so many sequences (48 KB) are kept in each block's shared memory, which saves the second launch for their tokens:
// a step of 64 sequences 6.8 us, with each block's own share kept 8.9; of 2048 15.8 / 17.5.
constexpr int kAllocAllSeqs = 2048;
cudaError_t launch_kv_alloc(const KvAllocParams& prm, int cluster, cudaStream_t stream);

struct KvPutParams {
    __half* cache[2];  // null: no cache
    __half* q_out;
    __half* k_out;  // may be null
    const __half* q;
    const __half* k;
    const __half* v;
    const int32_t* slots;
    const int32_t* positions;
    const float* cos_sin;
    long long q_stride, k_stride, v_stride;
    int num_blocks, num_tokens, num_heads, num_kv_heads, rot, max_positions, pairs;
    int rows_per_warp;  // heads (of Q, K and V together) that a warp takes
    unsigned int* status;
};
constexpr int kPutThreads = 128;
cudaError_t launch_kv_put(int head_dim, const KvPutParams& prm, dim3 grid, cudaStream_t stream);

struct LinearParams {
    __half* out;
    const __half* q;
    const __half* k;
    const __half* v;
    float* states;
    const float* log_decay;
    const int32_t* slots;
    const int32_t* context_lens;     // null: every sequence has a state
    const int32_t* query_start_loc;  // null: row b is sequence b's one token
    int num_slots, num_seqs, num_tokens, max_query_len;
    int num_heads, num_kv_heads, group;
    int few;  // > 0: sequences of up to so many tokens go token by token, the others in chunks; 0: all go one way
    float scale;
    unsigned int* status;
};
cudaError_t launch_linear_recurrent(int head_dim, const LinearParams& prm, cudaStream_t stream);

// The chunked form: a sequence's new tokens in blocks of kLinearBlock; block n of
// sequence b is number query_start_loc[b] / kLinearBlock + b + n, so that the
// blocks of packed sequences are numbered without gaps wider than one.
constexpr int kLinearBlock = 256;
constexpr int kLinearTile = 128;  // rows of an output tile; columns and rows of a state tile
struct LinearChunkParams {
    LinearParams lin;
    float* adds;           // [blocks][Hkv][D][D]: what a block's tokens add to the state
    __half* starts;        // [blocks][Hkv][D][D]: the state before a block, times 2^-exponent
    int* exponents;        // [blocks][Hkv]
    float* add_max;        // [blocks][Hkv][tiles]: largest finite magnitude in adds
    float* state_max;      // [B][Hkv]: of the state before the first block
    int* first_bad;        // [blocks][Hkv][D]: first token of a block with a NaN or infinity in that column of v
    int* any_bad;          // [blocks][Hkv][D / tile]: whether a tile's columns have one
    int4* block_info;      // [blocks]: first token, tokens (0: no such block), whether there is a state before it
    int blocks;            // numbers of blocks, those of no block among them
    int wait_limit;
};
// 64 rows of a tile's columns of k and v; of all columns 128 rows of q, and of k, v and starts as many as a
// ring stage of the outputs' kernel has, and of out.
struct LinearMaps {
    CUtensorMap k_group, v_group, q, k, v, starts, out;
};
void linear_out_boxes(int head_dim, int* rows, int* state_rows);
cudaError_t launch_linear_adds(int head_dim, const LinearChunkParams& prm, const LinearMaps& maps, int num_sms,
                               cudaStream_t stream);
cudaError_t launch_linear_scan(int head_dim, const LinearChunkParams& prm, cudaStream_t stream);
cudaError_t launch_linear_out(int head_dim, const LinearChunkParams& prm, const LinearMaps& maps, int num_sms,
                              cudaStream_t stream);

// Tensor map of packed rows [tokens][heads][head_dim] of halves: a box is `rows` tokens of one head by `cols`
// columns, laid out [64-column chunk][rows][128 B] with the 128-byte swizzle; coordinates (0, head, token, chunk).
int make_rows_map(CUtensorMap* map, const void* base, long long tokens, int heads, int head_dim, int rows, int cols);

}  // namespace pa
