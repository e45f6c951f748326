// C-ABI layer of block allocation, rotary put and linear attention (see
// include/pa_decode.h): argument checks, workspace layout and launches.
#include "pa_decode.h"

#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <initializer_list>
#include <iterator>

#include "pa_kv.h"
#include "pa_step.h"

namespace {

constexpr int kMaxTokens = 1 << 30;  // lengths, rounded up to any kernel's step, stay ints
constexpr size_t kWsAlign = 256;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool bad_ptr(const void* p, uintptr_t a) { return !p || !aligned(p, a); }

// An array of words of four bytes that a call reads or writes (n below 2^61, as all memory is).
struct Words {
    const void* p;
    long long n;
};
Words halves(const void* p, long long n) { return {p, n / 2}; }
bool overlap(const Words& a, const Words& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.p && b.p && a.n > 0 && b.n > 0 && (x < y ? y - x < 4ull * a.n : x - y < 4ull * b.n);
}

int check_alloc(const pa_kv_alloc_args* a) {
    if (!a) return PA_ERR_INVALID_ARG;
    if (a->num_seqs < 0 || a->num_seqs > 65535 || a->num_tokens < 0 || a->max_blocks_per_seq < 0 || a->num_blocks < 0 ||
        a->block_size <= 0)
        return PA_ERR_INVALID_ARG;
    if (a->block_size != pa::kBlockSize || a->num_tokens > kMaxTokens) return PA_ERR_UNSUPPORTED;
    if (a->num_blocks >= (1ll << 31) / pa::kBlockSize) return PA_ERR_UNSUPPORTED;  // slots are ints
    if (bad_ptr(a->free_count, 4) || bad_ptr(a->new_free_count, 4) || bad_ptr(a->query_start_loc, 4))
        return PA_ERR_INVALID_ARG;
    if (a->num_seqs > 0 && (bad_ptr(a->context_lens, 4) || bad_ptr(a->query_lens, 4) || bad_ptr(a->seq_lens, 4) ||
                            !aligned(a->held_lens, 4) || !aligned(a->new_held_lens, 4)))
        return PA_ERR_INVALID_ARG;
    if (a->num_seqs > 0 && a->max_blocks_per_seq > 0 && bad_ptr(a->block_tables, 4)) return PA_ERR_INVALID_ARG;
    if (a->num_blocks > 0 && bad_ptr(a->free_blocks, 4)) return PA_ERR_INVALID_ARG;
    if (a->num_tokens > 0 && (bad_ptr(a->slot_map, 4) || bad_ptr(a->positions, 4))) return PA_ERR_INVALID_ARG;
    const long long B = a->num_seqs;
    const Words out[] = {{a->block_tables, B * a->max_blocks_per_seq},
                         {a->free_blocks, a->num_blocks},
                         {a->new_free_count, 1},
                         {a->query_start_loc, B + 1},
                         {a->seq_lens, B},
                         {a->new_held_lens, B},
                         {a->slot_map, a->num_tokens},
                         {a->positions, a->num_tokens}};
    const Words in[] = {{a->free_count, 1}, {a->held_lens, B}, {a->context_lens, B}, {a->query_lens, B}};
    for (const Words& o : out) {
        for (const Words& x : out)
            if (&x != &o && overlap(o, x)) return PA_ERR_INVALID_ARG;
        for (const Words& x : in) {  // (the new count and the new held_lens may take the old ones' place)
            const bool in_place = x.p == o.p && ((o.p == a->new_free_count && x.p == a->free_count) ||
                                                 (o.p == a->new_held_lens && x.p == a->held_lens));
            if (!in_place && overlap(o, x)) return PA_ERR_INVALID_ARG;
        }
    }
    return PA_OK;
}

int check_put(const pa_kv_put_args* a) {
    if (!a) return PA_ERR_INVALID_ARG;
    const pa_kv_cache& c = a->cache;
    if (c.num_kv_heads <= 0 || c.head_dim <= 0 || c.block_size <= 0 || c.num_blocks < 0 || a->num_tokens < 0 ||
        a->num_heads <= 0 || a->rotary_dim < 0 || a->rotary_dim > c.head_dim || a->rotary_dim % 2 ||
        a->max_positions < 0 || (a->pairs != 0 && a->pairs != 1))
        return PA_ERR_INVALID_ARG;
    if (c.format != PA_KV_F16 && c.format != PA_KV_E4M3 && c.format != PA_KV_INT8) return PA_ERR_INVALID_ARG;
    const long long row[3] = {(long long)a->num_heads * c.head_dim, (long long)c.num_kv_heads * c.head_dim,
                              (long long)c.num_kv_heads * c.head_dim};
    const long long stride[3] = {a->q_stride, a->k_stride, a->v_stride};
    for (int i = 0; i < 3; ++i)
        if (stride[i] < 0 || stride[i] % 8 || (stride[i] && stride[i] < row[i])) return PA_ERR_INVALID_ARG;
    if (c.format != PA_KV_F16 || c.block_size != pa::kBlockSize ||
        (c.head_dim != 64 && c.head_dim != 128 && c.head_dim != 256))
        return PA_ERR_UNSUPPORTED;
    // slots are ints; heads a grid dimension
    if (c.num_blocks >= (1ll << 31) / pa::kBlockSize || a->num_heads > 65535 || c.num_kv_heads > 16384 ||
        a->num_tokens > kMaxTokens)
        return PA_ERR_UNSUPPORTED;
    // (so that no array's extent passes 64 bits)
    if (std::max({stride[0], stride[1], stride[2]}) >= (1ll << 31)) return PA_ERR_UNSUPPORTED;
    if (a->num_tokens == 0) return PA_OK;
    if (bad_ptr(a->q, 16) || bad_ptr(a->k, 16) || bad_ptr(a->q_out, 16) || !aligned(a->k_out, 16) ||
        bad_ptr(a->positions, 4) || (a->rotary_dim > 0 && bad_ptr(a->cos_sin, 16)))
        return PA_ERR_INVALID_ARG;
    if (!c.k_cache != !c.v_cache) return PA_ERR_INVALID_ARG;
    if (c.k_cache && (!aligned(c.k_cache, 16) || !aligned(c.v_cache, 16) || bad_ptr(a->v, 16) || bad_ptr(a->slot_map, 4)))
        return PA_ERR_INVALID_ARG;
    // rows of another pitch than the outputs' cannot be rotated in place
    if ((a->q_out == a->q && stride[0] && stride[0] != row[0]) || (a->k_out == a->k && stride[1] && stride[1] != row[1]))
        return PA_ERR_INVALID_ARG;
    const long long T = a->num_tokens, cached = c.num_blocks * row[1] * pa::kBlockSize;
    auto span = [&](int i) { return (T - 1) * (stride[i] ? stride[i] : row[i]) + row[i]; };
    const Words out[] = {halves(a->q_out, T * row[0]), halves(a->k_out, T * row[1]), halves(c.k_cache, cached),
                         halves(c.v_cache, cached)};
    const Words in[] = {halves(a->q, span(0)), halves(a->k, span(1)), halves(c.k_cache ? a->v : nullptr, span(2)),
                        {c.k_cache ? a->slot_map : nullptr, T}, {a->positions, T},
                        {a->cos_sin, (long long)a->max_positions * a->rotary_dim}};
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return PA_ERR_INVALID_ARG;
        for (int j = 0; j < 6; ++j)
            if (!(i == j && i < 2 && out[i].p == in[j].p) && overlap(out[i], in[j])) return PA_ERR_INVALID_ARG;
    }
    return PA_OK;
}

int check_linear(const pa_linear_state& s, int num_heads, float scale) {
    if (s.num_kv_heads <= 0 || s.head_dim <= 0 || s.num_slots < 0 || num_heads <= 0 || num_heads % s.num_kv_heads ||
        !isfinite(scale))
        return PA_ERR_INVALID_ARG;
    if (s.head_dim != 64 && s.head_dim != 128 && s.head_dim != 256) return PA_ERR_UNSUPPORTED;
    if (num_heads / s.num_kv_heads > pa::kMaxGroup || s.num_kv_heads > 65535 || s.num_slots >= (1ll << 31))
        return PA_ERR_UNSUPPORTED;
    return PA_OK;
}

// `read` is what else the call reads, `ws` its workspace.
template <typename Args>
bool bad_linear_pointers(const Args& a, long long tokens, std::initializer_list<Words> read = {}, const Words& ws = {}) {
    if (bad_ptr(a.out, 16) || bad_ptr(a.q, 16) || bad_ptr(a.k, 16) || bad_ptr(a.v, 16) || bad_ptr(a.state.states, 16) ||
        bad_ptr(a.log_decay, 4) || bad_ptr(a.slots, 4))
        return true;
    const long long D = a.state.head_dim, K = a.state.num_kv_heads;
    const Words out = halves(a.out, tokens * a.num_heads * D);
    const Words states{a.state.states, std::min(a.state.num_slots * K * D * D, 1ll << 60)};
    const Words in[] = {halves(a.q, tokens * a.num_heads * D), halves(a.k, tokens * K * D), halves(a.v, tokens * K * D),
                        {a.log_decay, K}, {a.slots, a.num_seqs}};
    auto written = [&](const Words& x) { return overlap(out, x) || overlap(states, x) || overlap(ws, x); };
    return std::any_of(std::begin(in), std::end(in), written) || std::any_of(read.begin(), read.end(), written) ||
           overlap(out, states) || overlap(ws, out) || overlap(ws, states);
}

int check_linear_prefix(const pa_linear_prefix_args* a, const void* ws) {
    if (!a) return PA_ERR_INVALID_ARG;
    if (a->num_seqs < 0 || a->num_seqs > 65535 || a->num_tokens < 0 || a->max_query_len < 0) return PA_ERR_INVALID_ARG;
    int rc = check_linear(a->state, a->num_heads, a->scale);
    if (rc) return rc;
    if (a->num_tokens > kMaxTokens) return PA_ERR_UNSUPPORTED;
    if (a->num_tokens > 0 && a->max_query_len == 0) return PA_ERR_INVALID_ARG;
    if (a->num_seqs == 0 || a->num_tokens == 0) return PA_OK;
    const size_t need = pa_linear_prefix_workspace_size(a->num_seqs, a->num_tokens, a->max_query_len, a->num_heads,
                                                        a->state.num_kv_heads, a->state.head_dim);
    if (bad_ptr(a->context_lens, 4) || bad_ptr(a->query_start_loc, 4) ||
        bad_linear_pointers(*a, a->num_tokens,
                            {{a->context_lens, a->num_seqs}, {a->query_start_loc, a->num_seqs + 1ll}},
                            {ws, (long long)(need / 4)}))
        return PA_ERR_INVALID_ARG;
    return PA_OK;
}

// pa_kv_alloc: up to so many sequences take a cluster of one block, more of them one of kAllocMaxCluster: a step of
// one new token each, 32 sequences 5.2 us in one and 5.4 in eight, 64 of them 6.8 either way, 128 of them 7.5 / 7.0,
// 512 of them 15.6 / 10.2.
constexpr int kAllocOneSeqs = 64;
// Up to so many new tokens for each block of the cluster are placed by it, more of them by a launch of their own:
// 4 sequences of 512 new tokens 5.0 us placed here and 5.1 apart, 8 of them 7.9 / 5.2; in eight blocks 4096 tokens
// 8.6 / 10.0, 16384 of them 10.9 / 10.3, 32768 of them 14.9 / 11.6.
constexpr int kAllocPlaceTokens = 4 * pa::kAllocThreads;

// pa_kv_put: a warp takes all heads of a token, or where there are few tokens a share of them, of at least kPutRows
// and so that there are no more than kPutWarps warps an SM.  64 tokens of 24/4 x 256: 3.2 us with shares of 4 heads,
// 4.1 with 8, 11.0 with all; 32/8 x 128 2.5, 3.1 and 9.5.  1024 tokens: 9.9 and 8.2 us with 16 warps an SM, 10.2 and
// 9.4 with 32, 12.4 and 10.7 with one warp a token (of 12/12 x 64 5.3, 5.8 and 5.6).  A second warp for each of 4096
// tokens gains 10 % there and loses 15 % at 12/12 x 64; at 8192 it gains nothing and loses up to 28 %.
constexpr int kPutRows = 4, kPutWarps = 16;

// Up to so many new tokens a sequence go token by token, by head_dim: where one sequence, with the group that these
// heads usually have, takes as long in chunks.  On the device, us there and in chunks: 1 sequence of 24/4 x 256 with 9
// tokens 19.4 / 21.7 and with 12 25.2 / 21.5; of 32/8 x 128 with 14 tokens 17.7 / 17.8; of 12/12 x 64 with 24 tokens
// 13.6 / 15.3.  Fewer heads a kv head and more sequences move it up, which the limit does not know: 1 sequence of
// 16/16 x 128 breaks even at 26 tokens, of 8/8 x 256 at 34; 64 sequences of 24/4 x 256 at 14 (159 / 169), of 32/8 x 128
// at 26 (with 16 66 / 98), of 12/12 x 64 at 42; 1 sequence of 8/1 x 64 already at 11 (with 24 29.8 / 14.2).
// In a batch whose longest sequence is above it, those that are not have a launch of their own (about 1.5 us; in
// chunks, a block's sums cost a token as much as 256).
int few_tokens(int head_dim) { return head_dim == 256 ? 9 : head_dim == 128 ? 14 : 24; }

// The chunked form's workspace: bytes, offsets (the blocks' sums are at 0).
struct LinearSpace {
    long long blocks;
    size_t starts, exponents, add_max, state_max, first_bad, any_bad, block_info, bytes;
};

LinearSpace linear_space(int num_seqs, int num_tokens, int num_kv_heads, int head_dim) {
    auto up = [](size_t x) { return (x + kWsAlign - 1) / kWsAlign * kWsAlign; };
    LinearSpace s;
    s.blocks = num_tokens / pa::kLinearBlock + (long long)num_seqs;
    const size_t heads = (size_t)s.blocks * num_kv_heads, square = (size_t)head_dim * head_dim;
    const int tiles = std::max(1, head_dim / pa::kLinearTile);
    s.starts = up(heads * square * 4);
    s.exponents = s.starts + up(heads * square * 2);
    s.add_max = s.exponents + up(heads * 4);
    s.state_max = s.add_max + up(heads * tiles * tiles * 4);
    s.first_bad = s.state_max + up((size_t)num_seqs * num_kv_heads * 4);
    s.any_bad = s.first_bad + up(heads * head_dim * 4);
    s.block_info = s.any_bad + up(heads * tiles * 4);
    s.bytes = s.block_info + up((size_t)s.blocks * 16);
    return s;
}

}  // namespace

extern "C" {

int pa_kv_alloc(const pa_kv_alloc_args* a, pa_stream_t stream) {
    int rc = check_alloc(a);
    if (rc) return rc;
    pa::KvAllocParams p{};
    p.tables = a->block_tables;
    p.free_blocks = a->free_blocks;
    p.count = a->free_count;
    p.new_count = a->new_free_count;
    p.held = a->held_lens ? a->held_lens : a->context_lens;
    p.context = a->context_lens;
    p.query = a->query_lens;
    p.loc = a->query_start_loc;
    p.lens = a->seq_lens;
    p.new_held = a->new_held_lens;
    p.slots = a->slot_map;
    p.positions = a->positions;
    p.num_blocks = static_cast<int>(a->num_blocks);
    p.num_seqs = a->num_seqs;
    p.num_tokens = a->num_tokens;
    p.cols = a->max_blocks_per_seq;
    p.status = pa::device_status_ptr();
    if (!p.status) return PA_ERR_CUDA;
    const int cluster = a->num_seqs <= kAllocOneSeqs ? 1 : pa::kAllocMaxCluster;
    p.place = a->num_tokens <= kAllocPlaceTokens * cluster;
    return pa::launch_kv_alloc(p, cluster, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

int pa_kv_put(const pa_kv_put_args* a, pa_stream_t stream) {
    int rc = check_put(a);
    if (rc) return rc;
    if (a->num_tokens == 0) return PA_OK;
    const pa_kv_cache& c = a->cache;
    pa::KvPutParams p{};
    p.cache[0] = static_cast<__half*>(c.k_cache);
    p.cache[1] = static_cast<__half*>(c.v_cache);
    p.q_out = static_cast<__half*>(a->q_out);
    p.k_out = static_cast<__half*>(a->k_out);
    p.q = static_cast<const __half*>(a->q);
    p.k = static_cast<const __half*>(a->k);
    p.v = static_cast<const __half*>(a->v);
    p.slots = a->slot_map;
    p.positions = a->positions;
    p.cos_sin = a->cos_sin;
    p.q_stride = a->q_stride ? a->q_stride : (long long)a->num_heads * c.head_dim;
    p.k_stride = a->k_stride ? a->k_stride : (long long)c.num_kv_heads * c.head_dim;
    p.v_stride = a->v_stride ? a->v_stride : (long long)c.num_kv_heads * c.head_dim;
    p.num_blocks = static_cast<int>(c.num_blocks);
    p.num_tokens = a->num_tokens;
    p.num_heads = a->num_heads;
    p.num_kv_heads = c.num_kv_heads;
    p.rot = a->rotary_dim;
    p.max_positions = a->max_positions;
    p.pairs = a->pairs;
    p.status = pa::device_status_ptr();
    if (!p.status) return PA_ERR_CUDA;
    const int rows = a->num_heads + 2 * c.num_kv_heads, warps = pa::kPutThreads / 32;
    int num_sms = 0;
    if (pa::sm_count(&num_sms) != PA_OK) return PA_ERR_CUDA;
    const long long splits =
        std::max(1ll, std::min((long long)rows / kPutRows, (long long)kPutWarps * num_sms / a->num_tokens));
    p.rows_per_warp = static_cast<int>(std::max((rows + splits - 1) / splits, (rows + 65534ll) / 65535));
    const dim3 grid((a->num_tokens + warps - 1) / warps, (rows + p.rows_per_warp - 1) / p.rows_per_warp);
    return pa::launch_kv_put(c.head_dim, p, grid, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? PA_OK
                                                                                                         : PA_ERR_CUDA;
}

int pa_linear_decode(const pa_linear_decode_args* a, pa_stream_t stream) {
    if (!a || a->num_seqs < 0 || a->num_seqs > 65535) return PA_ERR_INVALID_ARG;
    int rc = check_linear(a->state, a->num_heads, a->scale);
    if (rc || a->num_seqs == 0) return rc;
    if (bad_linear_pointers(*a, a->num_seqs)) return PA_ERR_INVALID_ARG;
    pa::LinearParams p{};
    p.out = static_cast<__half*>(a->out);
    p.q = static_cast<const __half*>(a->q);
    p.k = static_cast<const __half*>(a->k);
    p.v = static_cast<const __half*>(a->v);
    p.states = a->state.states;
    p.log_decay = a->log_decay;
    p.slots = a->slots;
    p.num_slots = static_cast<int>(a->state.num_slots);
    p.num_seqs = p.num_tokens = a->num_seqs;
    p.max_query_len = 1;
    p.num_heads = a->num_heads;
    p.num_kv_heads = a->state.num_kv_heads;
    p.group = a->num_heads / a->state.num_kv_heads;
    p.scale = a->scale;
    p.status = pa::device_status_ptr();
    if (!p.status) return PA_ERR_CUDA;
    return pa::launch_linear_recurrent(a->state.head_dim, p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

size_t pa_linear_prefix_workspace_size(int num_seqs, int num_tokens, int max_query_len, int num_heads,
                                       int num_kv_heads, int head_dim) {
    if (num_seqs <= 0 || num_seqs > 65535 || num_tokens <= 0 || num_tokens > kMaxTokens || max_query_len <= 0 ||
        num_heads <= 0 || num_kv_heads <= 0 || num_kv_heads > 65535 ||
        (head_dim != 64 && head_dim != 128 && head_dim != 256) || max_query_len <= few_tokens(head_dim))
        return 0;
    return linear_space(num_seqs, num_tokens, num_kv_heads, head_dim).bytes;
}

int pa_linear_prefix(const pa_linear_prefix_args* a, void* ws, size_t ws_bytes, pa_stream_t stream_) {
    int rc = check_linear_prefix(a, ws);
    if (rc || a->num_seqs == 0 || a->num_tokens == 0) return rc;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    const int D = a->state.head_dim, K = a->state.num_kv_heads;
    pa::LinearChunkParams c{};
    pa::LinearParams& p = c.lin;
    p.out = static_cast<__half*>(a->out);
    p.q = static_cast<const __half*>(a->q);
    p.k = static_cast<const __half*>(a->k);
    p.v = static_cast<const __half*>(a->v);
    p.states = a->state.states;
    p.log_decay = a->log_decay;
    p.slots = a->slots;
    p.context_lens = a->context_lens;
    p.query_start_loc = a->query_start_loc;
    p.num_slots = static_cast<int>(a->state.num_slots);
    p.num_seqs = a->num_seqs;
    p.num_tokens = a->num_tokens;
    p.max_query_len = a->max_query_len;
    p.num_heads = a->num_heads;
    p.num_kv_heads = K;
    p.group = a->num_heads / K;
    p.scale = a->scale;
    const bool few = a->max_query_len <= few_tokens(D);
    p.few = few || a->num_seqs == 1 ? 0 : few_tokens(D);
    const LinearSpace sp = linear_space(a->num_seqs, a->num_tokens, K, D);
    if (!few) {
        // rows of the tensor maps and CTAs of a grid are 32-bit
        if (sp.blocks * K * D >= (1ll << 31) || sp.blocks * 4 * a->num_heads >= (1ll << 31)) return PA_ERR_UNSUPPORTED;
        if (!ws || ws_bytes < sp.bytes || !aligned(ws, kWsAlign)) return PA_ERR_WORKSPACE;
    }
    p.status = pa::device_status_ptr();
    if (!p.status) return PA_ERR_CUDA;
    if (few) return pa::launch_linear_recurrent(D, p, stream) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
    uint8_t* w = static_cast<uint8_t*>(ws);
    c.adds = reinterpret_cast<float*>(w);
    c.starts = reinterpret_cast<__half*>(w + sp.starts);
    c.exponents = reinterpret_cast<int*>(w + sp.exponents);
    c.add_max = reinterpret_cast<float*>(w + sp.add_max);
    c.state_max = reinterpret_cast<float*>(w + sp.state_max);
    c.first_bad = reinterpret_cast<int*>(w + sp.first_bad);
    c.any_bad = reinterpret_cast<int*>(w + sp.any_bad);
    c.block_info = reinterpret_cast<int4*>(w + sp.block_info);
    c.blocks = static_cast<int>(sp.blocks);
    c.wait_limit = pa::kDefaultWaitLimit;
    const int tile = std::min(D, pa::kLinearTile);
    int num_sms = 0;
    if (pa::sm_count(&num_sms) != PA_OK) return PA_ERR_CUDA;
    pa::LinearMaps maps;
    int rows, state_rows;
    pa::linear_out_boxes(D, &rows, &state_rows);
    if ((rc = pa::make_rows_map(&maps.k_group, a->k, a->num_tokens, K, D, 64, tile)) ||
        (rc = pa::make_rows_map(&maps.v_group, a->v, a->num_tokens, K, D, 64, tile)) ||
        (rc = pa::make_rows_map(&maps.q, a->q, a->num_tokens, a->num_heads, D, 128, D)) ||
        (rc = pa::make_rows_map(&maps.k, a->k, a->num_tokens, K, D, rows, D)) ||
        (rc = pa::make_rows_map(&maps.v, a->v, a->num_tokens, K, D, rows, D)) ||
        (rc = pa::make_rows_map(&maps.out, a->out, a->num_tokens, a->num_heads, D, rows, D)) ||
        (rc = pa::make_rows_map(&maps.starts, c.starts, sp.blocks * K * D, 1, D, state_rows, D)))
        return rc;
    if (p.few > 0 && pa::launch_linear_recurrent(D, p, stream) != cudaSuccess) return PA_ERR_CUDA;
    if (pa::launch_linear_adds(D, c, maps, num_sms, stream) != cudaSuccess ||
        pa::launch_linear_scan(D, c, stream) != cudaSuccess ||
        pa::launch_linear_out(D, c, maps, num_sms, stream) != cudaSuccess)
        return PA_ERR_CUDA;
    return PA_OK;
}

}  // extern "C"
