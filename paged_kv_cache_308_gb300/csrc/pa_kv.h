// Internal interface between the C-ABI layer of the 8-bit cache and eviction
// calls (pa_kv_api.cpp) and their kernels (pa_kv_decode.cu, pa_kv_cache.cu).
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "pa_decode.h"
#include "pa_internal.h"

namespace pa {

// Defined in pa_api.cpp for the other C-ABI sources.
int sm_count(int* num_sms);                               // of the current device; a PA_* code
int check_prefix(const pa_prefix_args* args, const pa_decode_opts* opts);  // a PA_* code
// pa_prefix_ex whose caches hold the context without its factors, float2 [num_seqs]
// [max_blocks_per_seq][num_kv_heads] of (K, V) (see PrefixParams::factors; null:
// with them); split (null: none) as for pa_prefix_split, its states in `ws`.
int prefix_with_factors(const pa_prefix_args* args, const pa_decode_opts* opts, const float2* factors,
                        const pa_prefix_split_opts* split, void* ws, size_t ws_bytes, cudaStream_t stream);

struct KvDecodeParams {
    __half* out;
    const __half* q;
    const uint8_t* k_cache;
    const uint8_t* v_cache;
    const float* k_scales;  // null for fp16
    const float* v_scales;
    const int32_t* block_tables;
    const int32_t* seq_lens;
    // Partials, `slots` per kv head (slot: see pa_kv_decode.cu):
    float2* sums;  // [Hkv][slots][group]: reference exponent (log2 domain) and sum relative to it
    float* acc;    // [Hkv][slots][group][D], normalised
    int* seq_parts;  // flat: [B][8], where the partials of the sequences with tokens are
    float* scores;   // [B][H][score_stride], log2 domain; null without weights
    long long score_stride;
    const float* weights_in;  // cluster form: null: zeros
    float* weights_out;       // cluster form: null: none
    long long weights_stride;
    long long num_blocks, slots;
    int num_seqs, num_heads, num_kv_heads, group;
    int max_blocks_per_seq, max_seq_len;
    int flat, ctas_per_head;                // flat form
    int partition_size, max_partitions;     // grid form
    int cluster;                            // cluster form: CTAs of a cluster (1: no cluster); else 0
    float scale_log2;
    unsigned int* status;
};

struct KvMergeParams {
    __half* out;
    const float2* sums;
    const float* acc;
    const int* seq_parts;
    const float* scores;
    const float* weights_in;  // null: zeros
    float* weights_out;
    const int32_t* seq_lens;
    long long score_stride, weights_stride, slots;
    int num_heads, num_kv_heads, group, max_seq_len;
    int slices, cols;  // blocks of a (sequence, kv head) that merge, and their columns; the rest add weights
    int flat, partition_size, max_partitions;
    unsigned int* status;
};

constexpr int kKvWarps = 4;                        // of a decode CTA
constexpr int kKvMaxCluster = 8;                   // decode CTAs of a cluster (portable)
int kv_decode_ctas(int format, int head_dim);      // decode CTAs an SM holds at once; -1: not compiled
cudaError_t launch_kv_decode(int format, int head_dim, const KvDecodeParams& prm, dim3 grid, cudaStream_t stream);
constexpr int kKvWeightsTokens = 1024;  // tokens of a CTA that adds weights
cudaError_t launch_kv_merge(int head_dim, const KvMergeParams& prm, dim3 grid, cudaStream_t stream);

struct KvAppendParams {
    void* cache[2];        // K, V
    float* scales[2];
    const __half* fresh[2];
    const int32_t* block_tables;
    const int32_t* context_lens;
    const int32_t* query_start_loc;
    long long num_blocks;
    int num_kv_heads, max_blocks_per_seq, num_tokens, max_query_len, num_seqs;
    int packed;  // the grid's tile slots are packed over the sequences (else one grid layer a sequence)
    unsigned int* status;
};
cudaError_t launch_kv_append(int format, int head_dim, const KvAppendParams& prm, int tiles, cudaStream_t stream);

struct KvExpandParams {
    const uint8_t* cache[2];
    const float* scales[2];
    __half* expanded[2];   // [num_seqs * blocks_per_seq][Hkv][16][D]
    int32_t* tables;       // [num_seqs][blocks_per_seq]: their numbers
    float* factors;        // [num_seqs * blocks_per_seq][Hkv][K, V], or null
    const int32_t* block_tables;
    const int32_t* context_lens;
    long long num_blocks;
    int num_kv_heads, max_blocks_per_seq, blocks_per_seq, max_context_len;
    unsigned int* status;
};
cudaError_t launch_kv_expand(int format, int head_dim, const KvExpandParams& prm, dim3 grid, cudaStream_t stream);

struct KvEvictParams {
    const void* src[2];
    const float* src_scales[2];
    void* dst[2];
    float* dst_scales[2];
    const int32_t* block_tables;
    const int32_t* dst_block_tables;
    const int32_t* seq_lens;
    const int32_t* keep_lens;
    const float* weights;
    float* dst_weights;
    int32_t* kept;
    int32_t* new_lens;  // null: launch_kv_evict_lens writes it
    long long src_blocks, dst_blocks, weights_stride, dst_weights_stride;
    int num_kv_heads, max_blocks_per_seq, dst_max_blocks_per_seq;
    int max_seq_len, max_keep_len, sinks, recent;
    int key_words;  // keys a block of the selection holds in shared memory
    unsigned int* status;
};
constexpr int kEvictThreads = 1024;
constexpr int kEvictKeyWords = 48 * 1024;  // at most: 192 KB
cudaError_t launch_kv_evict_select(const KvEvictParams& prm, int num_seqs, int cluster, cudaStream_t stream);
struct KvEvictLensParams {
    KvEvictParams evict;
    int32_t* new_lens;  // may be evict.seq_lens or evict.keep_lens
    int num_seqs;
};
cudaError_t launch_kv_evict_lens(const KvEvictLensParams& prm, cudaStream_t stream);  // after the move
cudaError_t launch_kv_evict_move(int format, int head_dim, const KvEvictParams& prm, dim3 grid, cudaStream_t stream);

}  // namespace pa
