// C-ABI layer of the calls over a cache in 8 bits and of eviction (see
// include/pa_decode.h): argument checks, decode plan, workspace layout and
// launches.  Shares the device status word, the reduce kernel and the prefill
// kernels with pa_api.cpp.
#include "pa_decode.h"

#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>

#include "pa_internal.h"
#include "pa_kv.h"
#include "pa_prefix.h"

namespace {

constexpr size_t kWsAlign = 256;
// SM count assumed when no device answers (above any GPU's; a call then fails later)
constexpr int kMaxSmsBound = 1024;
// Tokens of a sequence at most: positions and counts of them, rounded up to any
// kernel's step, stay ints.
constexpr int kMaxTokens = 1 << 30;

size_t up(size_t x) { return (x + kWsAlign - 1) / kWsAlign * kWsAlign; }
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int blocks_of(long long tokens) { return static_cast<int>((tokens + pa::kBlockSize - 1) / pa::kBlockSize); }

int check_shape(const pa_kv_cache& c) {
    if (c.num_kv_heads <= 0 || c.head_dim <= 0 || c.block_size <= 0 || c.num_blocks < 0) return PA_ERR_INVALID_ARG;
    if (c.format != PA_KV_F16 && c.format != PA_KV_E4M3 && c.format != PA_KV_INT8) return PA_ERR_INVALID_ARG;
    if (c.head_dim != 64 && c.head_dim != 128 && c.head_dim != 256) return PA_ERR_UNSUPPORTED;
    if (c.block_size != pa::kBlockSize) return PA_ERR_UNSUPPORTED;
    if (c.num_kv_heads > 65535) return PA_ERR_UNSUPPORTED;  // a grid dimension (and x 8 another's)
    // TMA row coordinates are 32-bit
    if (c.num_blocks >= (1ll << 31) || c.num_blocks * c.num_kv_heads * c.block_size >= (1ll << 31))
        return PA_ERR_UNSUPPORTED;
    return PA_OK;
}

int check_pointers(const pa_kv_cache& c) {
    if (!c.k_cache || !c.v_cache || !aligned(c.k_cache, 16) || !aligned(c.v_cache, 16)) return PA_ERR_INVALID_ARG;
    if (c.format != PA_KV_F16 &&
        (!c.k_scales || !c.v_scales || !aligned(c.k_scales, 4) || !aligned(c.v_scales, 4)))
        return PA_ERR_INVALID_ARG;
    return PA_OK;
}

// Whether n and m words of four bytes share memory.
bool overlap(const void* p, long long n, const void* q, long long m) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(p), y = reinterpret_cast<uintptr_t>(q);
    return p && q && n > 0 && m > 0 && (x < y ? y - x < 4ull * n : x - y < 4ull * m);
}

bool bad_ptr(const void* p, uintptr_t a) { return !p || !aligned(p, a); }

// ---- decode

struct DecodePlan {
    bool flat;
    int ctas_per_head;          // flat
    int partition_size, parts;  // grid
    int cluster;                // CTAs of a cluster that has a (sequence, kv head) to itself, else 0; 1: a CTA that
                                // adds its weights itself
    long long slots;            // partials of a kv head
};

// Which form (us per call on GB300, replayed from a graph):
// * up to kSingleMaxLen tokens one CTA per (sequence, kv head), with no merge: 8
//   x 128 tokens of 4 x 256 in e4m3 4.9 against 5.8 in clusters, 16 x 512 of 8 x
//   128 7.7 / 8.1, 128 x 512 30.7 / 34.0 in equal shares;
// * a cluster per pair, which merges over distributed shared memory in the same
//   launch, while it has room and few rounds (see cluster_ctas): 8 x 512 of 4 x
//   256 6.7 against 9.6 with one CTA, 8 x 2048 10.9 / 14.1 in equal shares, 4 x
//   U[1, 2048] of 8 x 128 6.6 / 9.1; with the weights 2 x 512 of 4 x 256 7.4 /
//   12.8, 2 x 2048 10.0 / 11.2;
// * one CTA per pair up to kSingleManyMaxLen where the pairs nearly fill the SMs:
//   32 x 1024 of 8 x 128 19.0 against 19.5 in equal shares, of 4 x 256 17.4 /
//   20.6; 128 x U[1, 1024] 33.4 / 34.3;
// * one sequence: a wave of equal partitions, whose block ids can be read before
//   its length is known;
// * other batches: equal shares for the CTAs the SMs hold at once (against the
//   best of partitions of 256 to 8192 tokens, 8 x 128: 64 log-uniform up to 8192
//   26.5 / 33.5, 16 x U[1, 8192] 27.4 / 30.7, 64 x U[1, 4096] 59.6 / 61.1, 16 x 16384
//   86.9 / 94.4, 64 x 2048 51.5 / 55.8; 4 x 256: 8 x U[1, 8192] 17.2 / 18.0, 16 x U[1,
//   8192] 28.7 / 27.5, 64 x 2048 51.9 / 45.0, which only equal lengths give).
// A caller's partition size gives the grid of partitions.
constexpr int kSingleOneMaxLen = 128, kSingleMaxLen = 512, kSingleManyMaxLen = 1024;

// CTAs of the clusters that take a pair each, or 0 for another form.  The most
// that leave every warp a block, up to the portable 8, that the SMs hold at
// once: clusters fill 85 % of the places, those of 8 with one CTA per SM half
// of them (4 x 1024 of 4 x 256 in fp16, 128 CTAs of 8 on 152 SMs: 12.3 us against
// 8.4 in clusters of 4).  Two CTAs only beat one above 512 tokens (16 of 8 x 128:
// 512 tokens 8.1 / 7.7, 1024 12.5 / 13.7).  A pair's time grows with its blocks
// per warp, as others' do not: up to 8 rounds (4 x 4096 of 4 x 256 13.6 against
// 14.2 in equal shares; at 16, 8 x 4096 of 8 x 128 19.3 / 19.2 and with uniform
// lengths 12.6 / 11.4), with the weights, which need them again, 4 (8 rounds:
// 2 x 4096 of 4 x 256 14.1 / 12.0).  One sequence, whose partitions have more CTAs,
// without weights only and up to 4: 2048 tokens take 7.9 against 7.7, but the
// launch less saves the host 2.
int cluster_ctas(int num_seqs, int max_seq_len, int num_kv_heads, int ctas, int num_sms, bool weights) {
    const int blocks = blocks_of(max_seq_len);
    if (blocks * pa::kBlockSize <= kSingleOneMaxLen) return 0;
    const long long pairs = (long long)num_seqs * num_kv_heads, room = (long long)ctas * num_sms;
    int c = pa::kKvMaxCluster;
    while (c >= 2 && (blocks <= pa::kKvWarps * (c / 2) || pairs * c * 20 > room * (c == 8 && ctas == 1 ? 10 : 17)))
        c /= 2;
    if (c < 2 || (c == 2 && blocks * pa::kBlockSize <= kSingleMaxLen)) return 0;
    const int rounds = (blocks + pa::kKvWarps * c - 1) / (pa::kKvWarps * c);
    const int most = num_seqs == 1 ? (weights ? 0 : 4) : (weights ? 4 : 8);
    return rounds <= most ? c : 0;
}

DecodePlan plan_decode(int num_seqs, int max_seq_len, int num_kv_heads, int head_dim, int format, int num_sms,
                       int partition_size, int mode, bool weights) {
    DecodePlan p{};
    const int whole = std::max(1, blocks_of(max_seq_len)) * pa::kBlockSize;
    const int ctas = pa::kv_decode_ctas(format, head_dim);
    if (mode == PA_MODE_AUTO && partition_size <= 0 &&
        (p.cluster = cluster_ctas(num_seqs, max_seq_len, num_kv_heads, ctas, num_sms, weights))) {
        p.partition_size = whole;
        p.parts = 1;
        return p;
    }
    const bool many = (long long)num_seqs * num_kv_heads * 4 >= num_sms * 3ll;
    // (a batch of empty sequences has nothing to share out, and needs no workspace)
    if (max_seq_len == 0 || mode == PA_MODE_SINGLE || (partition_size <= 0 && mode == PA_MODE_AUTO && num_seqs > 1 &&
                                   max_seq_len <= (many ? kSingleManyMaxLen : kSingleMaxLen)))
        partition_size = whole;
    if (partition_size <= 0 && mode == PA_MODE_AUTO && max_seq_len <= kSingleOneMaxLen) partition_size = whole;
    const long long slots = std::max(1ll, (long long)ctas * num_sms / num_kv_heads);
    if (partition_size <= 0 && num_seqs == 1)  // (one block per warp at least)
        partition_size =
            std::max(blocks_of((max_seq_len + slots - 1) / slots), pa::kKvWarps) * pa::kBlockSize;
    if (partition_size > 0) {
        p.partition_size = std::min(partition_size, whole);
        p.parts = std::max(1, (max_seq_len + p.partition_size - 1) / p.partition_size);
        // A CTA with a whole sequence adds its weights itself while that is short and
        // the grid at most one and a half times what the SMs hold (with and without a
        // launch of their own: 8 x 128 of 4 x 256 in e4m3 7.6 / 6.2 us, 32 x 512 of 8 x
        // 128 15.0 / 14.5; 32 x 1024 23.6 / 25.2, 256 x 300 47.5 / 50.9).
        const long long pairs = (long long)num_seqs * num_kv_heads;
        if (p.parts == 1 && weights && max_seq_len <= kSingleMaxLen && pairs * 2 <= 3ll * ctas * num_sms) p.cluster = 1;
        p.slots = (long long)num_seqs * p.parts;
        return p;
    }
    p.flat = true;
    p.ctas_per_head = static_cast<int>(slots);
    p.slots = (1ll + pa::kKvWarps) * p.ctas_per_head + num_seqs;  // CTAs, warps + sequences
    return p;
}

struct DecodeSpace {
    size_t parts, acc, scores, bytes;  // offsets of seq_parts, acc and scores; the sums are at 0
    long long score_stride;
};

DecodeSpace decode_space(const DecodePlan& p, int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                         int max_seq_len, bool weights) {
    DecodeSpace s;
    const size_t rows = (size_t)p.slots * num_heads;  // slots of a kv head x kv heads x group
    const bool split = p.flat || p.parts > 1;
    s.parts = split || (weights && !p.cluster) ? up(rows * 8) : 0;
    s.acc = s.parts + (p.flat ? up((size_t)num_seqs * 32) : 0);
    s.scores = s.acc + (split ? up(rows * head_dim * 4) : 0);
    s.score_stride = (long long)blocks_of(max_seq_len) * pa::kBlockSize;
    s.bytes = s.scores + (weights ? up((size_t)num_seqs * num_heads * s.score_stride * 4) : 0);
    return s;
}

// Columns of four of a merging block: a power of two, so many that the batch
// gives about two blocks per SM.
int merge_cols(int num_seqs, int num_heads, int num_kv_heads, int head_dim, int num_sms) {
    const int total = num_heads / num_kv_heads * (head_dim / 4);
    int cols = 256;
    while (cols > 8 && (long long)num_seqs * num_kv_heads * ((total + cols - 1) / cols) < 2ll * num_sms) cols /= 2;
    return cols;
}

int check_decode(const pa_kv_decode_args* a, const pa_decode_opts* o) {
    if (!a) return PA_ERR_INVALID_ARG;
    if (a->num_seqs < 0 || a->num_seqs > 65535) return PA_ERR_INVALID_ARG;
    int rc = check_shape(a->cache);
    if (rc == PA_ERR_INVALID_ARG) return rc;
    if (a->num_heads <= 0 || a->num_heads % a->cache.num_kv_heads) return PA_ERR_INVALID_ARG;
    if (!isfinite(a->scale)) return PA_ERR_INVALID_ARG;
    if (a->max_seq_len < 0 || a->max_blocks_per_seq < 0) return PA_ERR_INVALID_ARG;
    if (o && (o->mode < PA_MODE_AUTO || o->mode > PA_MODE_SPLIT)) return PA_ERR_INVALID_ARG;
    if (o && (o->partition_size < 0 || o->partition_size % pa::kBlockSize)) return PA_ERR_INVALID_ARG;
    if (o && (o->warps || o->stages)) return PA_ERR_UNSUPPORTED;
    if (rc) return rc;
    if (a->num_heads / a->cache.num_kv_heads > pa::kMaxGroup) return PA_ERR_UNSUPPORTED;
    if ((long long)a->max_seq_len > (long long)a->max_blocks_per_seq * pa::kBlockSize) return PA_ERR_INVALID_ARG;
    if (a->weights_out && a->weights_stride < a->max_seq_len) return PA_ERR_INVALID_ARG;
    if (a->weights_in && !a->weights_out) return PA_ERR_INVALID_ARG;
    if (a->max_seq_len > kMaxTokens || (o && o->partition_size > kMaxTokens)) return PA_ERR_UNSUPPORTED;
    // the batch's blocks are numbered in 32 bits (with a few more a sequence)
    if ((long long)a->num_seqs * (blocks_of(a->max_seq_len) + 8ll) >= (1ll << 31)) return PA_ERR_UNSUPPORTED;
    if (a->num_seqs == 0) return PA_OK;
    if (bad_ptr(a->out, 16) || bad_ptr(a->q, 16) || bad_ptr(a->block_tables, 4) || bad_ptr(a->seq_lens, 4))
        return PA_ERR_INVALID_ARG;
    if (!aligned(a->weights_in, 4) || !aligned(a->weights_out, 4)) return PA_ERR_INVALID_ARG;
    if ((rc = check_pointers(a->cache))) return rc;
    if (a->cache.num_blocks == 0 && a->max_seq_len > 0) return PA_ERR_INVALID_ARG;
    return PA_OK;
}

int run_decode(const pa_kv_decode_args* a, const pa_decode_opts* o, void* ws, size_t ws_bytes, cudaStream_t stream) {
    int rc = check_decode(a, o);
    if (rc) return rc;
    if (a->num_seqs == 0) return PA_OK;
    const pa_kv_cache& c = a->cache;
    int num_sms = 0;
    if (pa::sm_count(&num_sms) != PA_OK) num_sms = kMaxSmsBound;  // (as for the size)
    const bool weights = a->weights_out && a->max_seq_len > 0;
    const DecodePlan plan = plan_decode(a->num_seqs, a->max_seq_len, c.num_kv_heads, c.head_dim, c.format, num_sms,
                                        o ? o->partition_size : 0, o ? o->mode : PA_MODE_AUTO, weights);
    const DecodeSpace sp =
        decode_space(plan, a->num_seqs, a->num_heads, c.num_kv_heads, c.head_dim, a->max_seq_len, weights);
    if (sp.bytes > 0 && (!ws || ws_bytes < sp.bytes || !aligned(ws, kWsAlign))) return PA_ERR_WORKSPACE;
    const bool split = plan.flat || plan.parts > 1;

    uint8_t* w = static_cast<uint8_t*>(ws);
    pa::KvDecodeParams p{};
    p.out = static_cast<__half*>(a->out);
    p.q = static_cast<const __half*>(a->q);
    p.k_cache = static_cast<const uint8_t*>(c.k_cache);
    p.v_cache = static_cast<const uint8_t*>(c.v_cache);
    p.k_scales = c.k_scales;
    p.v_scales = c.v_scales;
    p.block_tables = a->block_tables;
    p.seq_lens = a->seq_lens;
    p.sums = split || (weights && !plan.cluster) ? reinterpret_cast<float2*>(w) : nullptr;
    p.seq_parts = plan.flat ? reinterpret_cast<int*>(w + sp.parts) : nullptr;
    p.acc = split ? reinterpret_cast<float*>(w + sp.acc) : nullptr;
    p.scores = weights ? reinterpret_cast<float*>(w + sp.scores) : nullptr;
    p.score_stride = sp.score_stride;
    p.weights_in = a->weights_in;
    p.weights_out = weights && plan.cluster ? a->weights_out : nullptr;
    p.weights_stride = a->weights_stride;
    p.num_blocks = c.num_blocks;
    p.slots = plan.slots;
    p.num_seqs = a->num_seqs;
    p.num_heads = a->num_heads;
    p.num_kv_heads = c.num_kv_heads;
    p.group = a->num_heads / c.num_kv_heads;
    p.max_blocks_per_seq = a->max_blocks_per_seq;
    p.max_seq_len = a->max_seq_len;
    p.flat = plan.flat;
    p.ctas_per_head = plan.ctas_per_head;
    p.partition_size = plan.partition_size;
    p.max_partitions = plan.parts;
    p.cluster = plan.cluster;
    p.scale_log2 = static_cast<float>(static_cast<double>(a->scale) * 1.4426950408889634);
    p.status = pa::device_status_ptr();
    if (!p.status) return PA_ERR_CUDA;
    const dim3 grid = plan.flat ? dim3(plan.ctas_per_head * c.num_kv_heads)
                                : dim3(plan.cluster ? plan.cluster : plan.parts, c.num_kv_heads, a->num_seqs);
    if (pa::launch_kv_decode(c.format, c.head_dim, p, grid, stream) != cudaSuccess) return PA_ERR_CUDA;
    if (plan.cluster || (!split && !weights)) return PA_OK;
    pa::KvMergeParams m{};
    m.out = p.out;
    m.sums = p.sums;
    m.acc = p.acc;
    m.seq_parts = p.seq_parts;
    m.scores = p.scores;
    m.weights_in = a->weights_in;
    m.weights_out = a->weights_out;
    m.seq_lens = a->seq_lens;
    m.score_stride = sp.score_stride;
    m.weights_stride = a->weights_stride;
    m.slots = plan.slots;
    m.num_heads = a->num_heads;
    m.num_kv_heads = c.num_kv_heads;
    m.group = p.group;
    m.max_seq_len = a->max_seq_len;
    m.cols = merge_cols(a->num_seqs, a->num_heads, c.num_kv_heads, c.head_dim, num_sms);
    m.slices = split ? (p.group * c.head_dim / 4 + m.cols - 1) / m.cols : 0;
    m.flat = plan.flat;
    m.partition_size = plan.partition_size;
    m.max_partitions = plan.parts;
    m.status = p.status;
    const int chunks = weights ? (a->max_seq_len + pa::kKvWeightsTokens - 1) / pa::kKvWeightsTokens : 0;
    if (m.slices + chunks == 0) return PA_OK;
    return pa::launch_kv_merge(c.head_dim, m, dim3(m.slices + chunks, c.num_kv_heads, a->num_seqs), stream) ==
                   cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

// ---- append

int check_append(const pa_kv_append_args* a) {
    if (!a) return PA_ERR_INVALID_ARG;
    if (a->num_seqs < 0 || a->num_seqs > 65535 || a->num_tokens < 0) return PA_ERR_INVALID_ARG;
    if (a->max_blocks_per_seq < 0 || a->max_query_len < 0) return PA_ERR_INVALID_ARG;
    int rc = check_shape(a->cache);
    if (rc) return rc;
    // the largest position must be an int
    if ((long long)a->max_blocks_per_seq * pa::kBlockSize >= (1ll << 31)) return PA_ERR_UNSUPPORTED;
    if (a->num_tokens > kMaxTokens) return PA_ERR_UNSUPPORTED;
    if (a->num_tokens > 0 && a->max_query_len == 0) return PA_ERR_INVALID_ARG;
    if (a->num_seqs == 0 || a->num_tokens == 0) return PA_OK;
    if (bad_ptr(a->k_new, 16) || bad_ptr(a->v_new, 16) || bad_ptr(a->block_tables, 4) ||
        bad_ptr(a->context_lens, 4) || bad_ptr(a->query_start_loc, 4))
        return PA_ERR_INVALID_ARG;
    return check_pointers(a->cache);
}

// ---- prefill

size_t prefix_copy_bytes(int num_seqs, int blocks_per_seq, int num_kv_heads, int head_dim) {
    return up((size_t)num_seqs * blocks_per_seq * num_kv_heads * pa::kBlockSize * head_dim * 2);
}

// The copy's K and V, its table, INT8's factors; then the states of split query
// tiles, one tile per SM at most (see plan_prefix).
struct PrefixSpace {
    size_t copy, factors, states, bytes;  // bytes of K's copy; offsets; all
};

constexpr int kPrefixSplitMinContext = 512;

PrefixSpace prefix_space(int num_seqs, int max_context_len, int num_kv_heads, int head_dim, int format, int num_sms) {
    PrefixSpace s{};
    if (format == PA_KV_F16 || max_context_len == 0) return s;
    const int n = blocks_of(max_context_len);
    s.copy = prefix_copy_bytes(num_seqs, n, num_kv_heads, head_dim);
    s.factors = 2 * s.copy + up((size_t)num_seqs * n * 4);
    s.states = s.factors + (format == PA_KV_INT8 ? up((size_t)num_seqs * n * num_kv_heads * 8) : 0);
    s.bytes = s.states;
    if (max_context_len >= kPrefixSplitMinContext && 2ll * num_seqs * num_kv_heads <= num_sms)
        s.bytes += up((size_t)num_sms * pa::kPrefixTileRows * head_dim * 4) + up((size_t)num_sms * pa::kPrefixTileRows * 8);
    return s;
}

// Key ranges that each of `tiles` query tiles has its keys cut into (0: none): one
// (query tile, range) per SM at most, four key tiles a range or more, and only
// where the longest tile's walk gets ten key tiles shorter, which pays for the
// merge of the ranges' states (chunks of 37 tokens, whole / split: 8 x 128 after
// 8000 tokens in int8 117.7 / 36.2 us, after 1000 22.8 / 17.5, four such chunks
// after 8000 137.9 / 94.5, after 1000, two ranges each, 26.5 / 27.5; 4 x 256
// after 500 in e4m3 19.3 / 21.9).
int plan_prefix(const pa_prefix_args* a, int num_sms, long long tiles) {
    if (a->max_context_len < kPrefixSplitMinContext || tiles * 2 > num_sms) return 0;
    const int keys = (blocks_of(a->max_context_len) + blocks_of(a->max_query_len) + 3) / 4;  // key tiles of 64
    const int parts = static_cast<int>(std::min<long long>(num_sms / tiles, std::min(64, keys / 4)));
    return parts >= 2 && (long long)keys * (parts - 1) >= 10ll * parts ? parts : 0;
}

int run_prefix(const pa_kv_prefix_args* a, const pa_decode_opts* o, void* ws, size_t ws_bytes, cudaStream_t stream) {
    if (!a) return PA_ERR_INVALID_ARG;
    const pa_kv_cache& c = a->cache;
    int rc = check_shape(c);
    if (rc) return rc;
    pa_prefix_args p;
    p.out = a->out;
    p.q = a->q;
    p.k_new = a->k_new;
    p.v_new = a->v_new;
    p.k_cache = c.k_cache;
    p.v_cache = c.v_cache;
    p.block_tables = a->block_tables;
    p.context_lens = a->context_lens;
    p.query_start_loc = a->query_start_loc;
    p.num_seqs = a->num_seqs;
    p.num_tokens = a->num_tokens;
    p.max_blocks_per_seq = a->max_blocks_per_seq;
    p.max_context_len = a->max_context_len;
    p.max_query_len = a->max_query_len;
    p.num_blocks = c.num_blocks;
    p.num_heads = a->num_heads;
    p.num_kv_heads = c.num_kv_heads;
    p.head_dim = c.head_dim;
    p.block_size = c.block_size;
    p.scale = a->scale;
    if ((rc = pa::check_prefix(&p, o))) return rc;  // as the caller gave it
    if (a->num_seqs == 0 || a->num_tokens == 0) return PA_OK;
    if ((rc = check_pointers(c))) return rc;
    if (c.format == PA_KV_F16) return pa_prefix_ex(&p, o, reinterpret_cast<pa_stream_t>(stream));

    const int n = blocks_of(a->max_context_len);
    int num_sms = 0;
    if (pa::sm_count(&num_sms) != PA_OK) num_sms = kMaxSmsBound;  // (as for the size)
    const PrefixSpace sp =
        prefix_space(a->num_seqs, a->max_context_len, c.num_kv_heads, c.head_dim, c.format, num_sms);
    const bool warp_mma = o && (o->flags & PA_FLAG_PREFIX_WARP_MMA);
    // the copy replaces the cache; it has room for every sequence's longest context
    p.num_blocks = (int64_t)a->num_seqs * n;
    p.max_blocks_per_seq = n;
    float* factors = nullptr;
    if (n > 0) {
        if (p.num_blocks * c.num_kv_heads * pa::kBlockSize >= (1ll << 31)) return PA_ERR_UNSUPPORTED;
        if (!ws || ws_bytes < sp.bytes || !aligned(ws, kWsAlign)) return PA_ERR_WORKSPACE;
        uint8_t* w = static_cast<uint8_t*>(ws);
        pa::KvExpandParams e{};
        e.cache[0] = static_cast<const uint8_t*>(c.k_cache);
        e.cache[1] = static_cast<const uint8_t*>(c.v_cache);
        e.scales[0] = c.k_scales;
        e.scales[1] = c.v_scales;
        e.expanded[0] = reinterpret_cast<__half*>(w);
        e.expanded[1] = reinterpret_cast<__half*>(w + sp.copy);
        e.tables = reinterpret_cast<int32_t*>(w + 2 * sp.copy);
        // INT8 scales have more bits than a product with a code leaves room for in
        // fp16: their significands go to the kernel apart (the warp-level kernel
        // cannot take them; there the values are rounded)
        if (c.format == PA_KV_INT8 && !warp_mma) factors = reinterpret_cast<float*>(w + sp.factors);
        e.factors = factors;
        e.block_tables = a->block_tables;
        e.context_lens = a->context_lens;
        e.num_blocks = c.num_blocks;
        e.num_kv_heads = c.num_kv_heads;
        e.max_blocks_per_seq = a->max_blocks_per_seq;
        e.blocks_per_seq = n;
        e.max_context_len = a->max_context_len;
        e.status = pa::device_status_ptr();
        if (!e.status) return PA_ERR_CUDA;
        p.k_cache = e.expanded[0];
        p.v_cache = e.expanded[1];
        p.block_tables = e.tables;
        if (pa::launch_kv_expand(c.format, c.head_dim, e, dim3(n, c.num_kv_heads, a->num_seqs), stream) !=
            cudaSuccess)
            return PA_ERR_CUDA;
    }
    // Few query tiles: one CTA each, without the counter they would be claimed
    // from (that form takes 1.5 to 2 us less there), and their keys in several
    // ranges where that fills the SMs.
    pa_decode_opts opts = {};
    if (o) opts = *o;
    const int tile_tokens = pa::kPrefixTileRows / (a->num_heads / c.num_kv_heads);
    const long long tiles =
        (long long)((a->max_query_len + tile_tokens - 1) / tile_tokens) * c.num_kv_heads * a->num_seqs;
    if (tiles <= num_sms && !warp_mma) opts.flags |= PA_FLAG_PREFIX_GRID;
    pa_prefix_split_opts split = {};
    if (!warp_mma && n > 0) split.parts = plan_prefix(&p, num_sms, tiles);
    split.units = static_cast<int>(split.parts ? tiles : 0);
    return pa::prefix_with_factors(&p, &opts, reinterpret_cast<const float2*>(factors), split.parts ? &split : nullptr,
                                   static_cast<uint8_t*>(ws) + sp.states, sp.bytes - sp.states, stream);
}

// ---- eviction

int check_evict(const pa_kv_evict_args* a) {
    if (!a) return PA_ERR_INVALID_ARG;
    if (a->num_seqs < 0 || a->num_seqs > 65535) return PA_ERR_INVALID_ARG;
    if (a->max_seq_len < 0 || a->max_keep_len < 0 || a->sinks < 0 || a->recent < 0) return PA_ERR_INVALID_ARG;
    if (a->max_blocks_per_seq < 0 || a->dst_max_blocks_per_seq < 0) return PA_ERR_INVALID_ARG;
    int rc = check_shape(a->src);
    if (rc || (rc = check_shape(a->dst))) return rc;
    if (a->src.format != a->dst.format || a->src.num_kv_heads != a->dst.num_kv_heads ||
        a->src.head_dim != a->dst.head_dim)
        return PA_ERR_INVALID_ARG;
    if ((long long)a->max_seq_len > (long long)a->max_blocks_per_seq * pa::kBlockSize ||
        (long long)a->max_keep_len > (long long)a->dst_max_blocks_per_seq * pa::kBlockSize)
        return PA_ERR_INVALID_ARG;
    if (a->weights_stride < a->max_seq_len || (a->dst_weights && a->dst_weights_stride < a->max_keep_len))
        return PA_ERR_INVALID_ARG;
    if (a->max_seq_len > kMaxTokens || a->max_keep_len > kMaxTokens) return PA_ERR_UNSUPPORTED;
    if (a->num_seqs == 0) return PA_OK;
    if (bad_ptr(a->seq_lens, 4) || bad_ptr(a->keep_lens, 4) || bad_ptr(a->new_lens, 4)) return PA_ERR_INVALID_ARG;
    if (!aligned(a->weights, 4) || !aligned(a->dst_weights, 4) || !aligned(a->kept, 4)) return PA_ERR_INVALID_ARG;
    if (a->max_seq_len > 0 && !a->weights) return PA_ERR_INVALID_ARG;
    if (a->max_seq_len > 0 && a->max_keep_len > 0) {
        if (!a->kept || bad_ptr(a->block_tables, 4) || bad_ptr(a->dst_block_tables, 4)) return PA_ERR_INVALID_ARG;
        if ((rc = check_pointers(a->src)) || (rc = check_pointers(a->dst))) return rc;
        if (a->src.num_blocks == 0 || a->dst.num_blocks == 0) return PA_ERR_INVALID_ARG;
    }
    // new_lens takes seq_lens' or keep_lens' place element by element, or has memory of its own
    for (const int32_t* lens : {a->seq_lens, a->keep_lens})
        if (lens != a->new_lens && overlap(a->new_lens, a->num_seqs, lens, a->num_seqs)) return PA_ERR_INVALID_ARG;
    // in place would read rows that are already overwritten
    if (a->weights && a->weights == a->dst_weights) return PA_ERR_INVALID_ARG;
    if (a->block_tables && a->block_tables == a->dst_block_tables &&
        (a->src.k_cache == a->dst.k_cache || a->src.v_cache == a->dst.v_cache))
        return PA_ERR_INVALID_ARG;
    return PA_OK;
}

// Blocks that share a (sequence, kv head) in the selection.  A cluster costs about
// 3 us more than a block alone and pays for itself above 12,000 tokens (device us
// with the move, 1, 2, 4 and 8 blocks: 8 heads of one sequence of 8192 tokens 10.1,
// 12.3, 11.8, 12.1, of 16384 13.4, 13.9, 12.5, 12.2, of 32768 20.8, 18.1, 15.2,
// 13.8), a pair of blocks above 24,000, as long as the SMs hold the whole grid,
// of clusters of 8 half of it (16 pairs of 16384: 20.3 in clusters of 8, 13.5 of 4).
int evict_cluster(int max_seq_len, long long pairs, int num_sms) {
    int c = max_seq_len <= 12 * 1024 ? 1 : pairs * 16 <= num_sms ? 8 : pairs * 4 <= num_sms ? 4 : 1;
    if (c == 1 && max_seq_len > 24 * 1024 && pairs * 2 <= num_sms) c = 2;
    // more than one block can hold in shared memory is shared out whatever the grid
    while (c < 8 && max_seq_len > (long long)pa::kEvictKeyWords * c) c *= 2;
    return c;
}

}  // namespace

extern "C" {

int pa_kv_append(const pa_kv_append_args* a, pa_stream_t stream) {
    int rc = check_append(a);
    if (rc) return rc;
    if (a->num_seqs == 0 || a->num_tokens == 0) return PA_OK;
    const pa_kv_cache& c = a->cache;
    pa::KvAppendParams p{};
    p.cache[0] = c.k_cache;
    p.cache[1] = c.v_cache;
    p.scales[0] = c.k_scales;
    p.scales[1] = c.v_scales;
    p.fresh[0] = static_cast<const __half*>(a->k_new);
    p.fresh[1] = static_cast<const __half*>(a->v_new);
    p.block_tables = a->block_tables;
    p.context_lens = a->context_lens;
    p.query_start_loc = a->query_start_loc;
    p.num_blocks = c.num_blocks;
    p.num_kv_heads = c.num_kv_heads;
    p.max_blocks_per_seq = a->max_blocks_per_seq;
    p.num_tokens = a->num_tokens;
    p.max_query_len = std::min(a->max_query_len, a->num_tokens);
    p.status = pa::device_status_ptr();
    if (!p.status) return PA_ERR_CUDA;
    // a run of n tokens touches at most ceil((n - 1) / 16) + 1 blocks; packed,
    // the slots of all sequences end below num_tokens / 16 + 2 num_seqs
    p.num_seqs = a->num_seqs;
    const long long each = blocks_of(p.max_query_len - 1) + 1;
    const long long packed = a->num_tokens / pa::kBlockSize + 2ll * a->num_seqs;
    p.packed = packed < each * a->num_seqs;
    return pa::launch_kv_append(c.format, c.head_dim, p, static_cast<int>(p.packed ? packed : each),
                                reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

size_t pa_kv_decode_workspace_size(int num_seqs, int max_seq_len, int num_heads, int num_kv_heads, int head_dim,
                                   int format, int mode, int partition_size, int weights) {
    if (num_seqs <= 0 || max_seq_len <= 0 || num_heads <= 0 || num_kv_heads <= 0 || partition_size < 0 ||
        partition_size % pa::kBlockSize || mode < PA_MODE_AUTO || mode > PA_MODE_SPLIT ||
        max_seq_len > kMaxTokens || partition_size > kMaxTokens || num_heads % num_kv_heads || pa::kv_decode_ctas(format, head_dim) < 0)
        return 0;
    int num_sms = 0;
    if (pa::sm_count(&num_sms) != PA_OK || num_sms <= 0) num_sms = kMaxSmsBound;
    const DecodePlan plan =
        plan_decode(num_seqs, max_seq_len, num_kv_heads, head_dim, format, num_sms, partition_size, mode,
                    weights != 0);
    return decode_space(plan, num_seqs, num_heads, num_kv_heads, head_dim, max_seq_len, weights != 0).bytes;
}

int pa_kv_decode(const pa_kv_decode_args* args, const pa_decode_opts* opts, void* workspace, size_t workspace_bytes,
                 pa_stream_t stream) {
    return run_decode(args, opts, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

size_t pa_kv_prefix_workspace_size(int num_seqs, int max_context_len, int num_kv_heads, int head_dim, int format) {
    if (num_seqs <= 0 || max_context_len <= 0 || num_kv_heads <= 0 || pa::kv_decode_ctas(format, head_dim) < 0)
        return 0;
    int num_sms = 0;
    if (pa::sm_count(&num_sms) != PA_OK || num_sms <= 0) num_sms = kMaxSmsBound;
    return prefix_space(num_seqs, max_context_len, num_kv_heads, head_dim, format, num_sms).bytes;
}

int pa_kv_prefix(const pa_kv_prefix_args* args, const pa_decode_opts* opts, void* workspace, size_t workspace_bytes,
                 pa_stream_t stream) {
    return run_prefix(args, opts, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

int pa_kv_evict(const pa_kv_evict_args* a, pa_stream_t stream_) {
    int rc = check_evict(a);
    if (rc) return rc;
    if (a->num_seqs == 0) return PA_OK;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    pa::KvEvictParams p{};
    p.src[0] = a->src.k_cache;
    p.src[1] = a->src.v_cache;
    p.src_scales[0] = a->src.k_scales;
    p.src_scales[1] = a->src.v_scales;
    p.dst[0] = a->dst.k_cache;
    p.dst[1] = a->dst.v_cache;
    p.dst_scales[0] = a->dst.k_scales;
    p.dst_scales[1] = a->dst.v_scales;
    p.block_tables = a->block_tables;
    p.dst_block_tables = a->dst_block_tables;
    p.seq_lens = a->seq_lens;
    p.keep_lens = a->keep_lens;
    p.weights = a->weights;
    p.dst_weights = a->dst_weights;
    p.kept = a->kept;
    const bool in_place = a->new_lens == a->seq_lens || a->new_lens == a->keep_lens;
    p.new_lens = in_place ? nullptr : a->new_lens;
    p.src_blocks = a->src.num_blocks;
    p.dst_blocks = a->dst.num_blocks;
    p.weights_stride = a->weights_stride;
    p.dst_weights_stride = a->dst_weights_stride;
    p.num_kv_heads = a->src.num_kv_heads;
    p.max_blocks_per_seq = a->max_blocks_per_seq;
    p.dst_max_blocks_per_seq = a->dst_max_blocks_per_seq;
    p.max_seq_len = a->max_seq_len;
    p.max_keep_len = a->max_keep_len;
    p.sinks = a->sinks;
    p.recent = a->recent;
    p.status = pa::device_status_ptr();
    if (!p.status) return PA_ERR_CUDA;
    // lengths that change while blocks read them would part the blocks of a cluster
    const long long pairs = (long long)a->num_seqs * p.num_kv_heads;
    for (const int32_t* lens : {a->seq_lens, a->keep_lens})
        if (overlap(a->kept, pairs * a->max_keep_len, lens, a->num_seqs) ||
            overlap(a->dst_weights, pairs * a->dst_weights_stride, lens, a->num_seqs))
            return PA_ERR_INVALID_ARG;
    int num_sms = 0;
    if (pa::sm_count(&num_sms) != PA_OK) num_sms = 1;
    const int cluster = evict_cluster(a->max_seq_len, pairs, num_sms);
    // (each warp's run is a multiple of 128 keys)
    constexpr int kRound = 4 * pa::kEvictThreads;
    p.key_words = static_cast<int>(std::min<long long>(
        pa::kEvictKeyWords, ((a->max_seq_len + cluster - 1ll) / cluster + kRound - 1) / kRound * kRound));
    if (pa::launch_kv_evict_select(p, a->num_seqs, cluster, stream) != cudaSuccess) return PA_ERR_CUDA;
    const int blocks = blocks_of(std::min(a->max_keep_len, a->max_seq_len));
    if (blocks > 0 && pa::launch_kv_evict_move(a->src.format, a->src.head_dim, p,
                                               dim3(blocks, p.num_kv_heads, a->num_seqs), stream) != cudaSuccess)
        return PA_ERR_CUDA;
    if (in_place && pa::launch_kv_evict_lens({p, a->new_lens, a->num_seqs}, stream) != cudaSuccess) return PA_ERR_CUDA;
    return PA_OK;
}

}  // extern "C"
