// Writing, expanding and thinning out the paged cache: kv_append_kernel,
// kv_expand_kernel (8-bit context blocks to an fp16 copy, for the prefill
// kernel), kv_evict_select_kernel and kv_evict_move_kernel.  All of them are
// bound by memory: each moves its rows once, 16 bytes a lane.
#include "pa_kv.h"

#include <cooperative_groups.h>
#include <cuda_fp8.h>
#include <math.h>

#include "pa_decode.h"
#include "pa_device.cuh"

namespace pa {
namespace {

namespace cg = cooperative_groups;

// Block scale of a largest magnitude (a half's value or a scale times a code,
// so a normal number or 0).  E4M3: the smallest 2^k with 448 2^k >= amax; 448
// = 1.75 2^8, so k is amax's exponent less 8, or less 7 above a significand
// of 1.75.  INT8: amax / 127 rounded up to 8 significant bits (the quotient
// of an 11-bit number by 127 is never so close above an 8-bit number that
// rounding it to 24 bits first would lose the difference).
template <int F>
__device__ __forceinline__ float block_scale(float amax) {
    if (!(amax > 0.f)) return 0.f;
    if constexpr (F == PA_KV_E4M3) {
        const uint32_t bits = __float_as_uint(amax);
        const uint32_t e = (bits >> 23) - ((bits & 0x7fffffu) <= 0x600000u ? 8u : 7u);
        return __uint_as_float(e << 23);
    } else {
        const uint32_t bits = __float_as_uint(__fdiv_rn(amax, 127.f));
        return __uint_as_float((bits + 0xffffu) & 0xffff0000u);
    }
}

// x in units of s.  Scales of E4M3 blocks are powers of two unless a caller
// wrote others: then multiplying by 1 / s is the same as dividing.
struct Unit {
    float s, inv;
    bool pow2;
    __device__ explicit Unit(float scale) : s(scale) {
        const uint32_t bits = __float_as_uint(scale);
        pow2 = (bits & 0x7fffffu) == 0 && scale >= 0x1p-100f && scale <= 0x1p100f;
        inv = pow2 ? __uint_as_float((254u << 23) - bits) : 0.f;
    }
    __device__ __forceinline__ float of(float x) const {
        if (pow2) return x * inv;
        return s > 0.f ? __fdiv_rn(x, s) : x;
    }
};

template <int F>
__device__ __forceinline__ uint32_t code_of(float t) {
    if constexpr (F == PA_KV_E4M3) {
        return __nv_cvt_float_to_fp8(t, __NV_SATFINITE, __NV_E4M3);
    } else {
        const int q = __float2int_rn(t);  // NaN: 0
        return static_cast<uint32_t>(max(-127, min(127, q))) & 0xffu;
    }
}

template <int F>
__device__ __forceinline__ float value_of(uint32_t code) {
    if constexpr (F == PA_KV_E4M3) {
        return __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(code), __NV_E4M3)));
    } else {
        return static_cast<float>(static_cast<int8_t>(code));
    }
}

// Four codes of `w` from scale s0 to the unit u.
template <int F>
__device__ __forceinline__ uint32_t recode(uint32_t w, float s0, const Unit& u) {
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) r |= code_of<F>(u.of(value_of<F>((w >> (8 * i)) & 0xffu) * s0)) << (8 * i);
    return r;
}

// K's or V's of a pair of arguments, without indexing the parameter memory.
template <typename T>
__device__ __forceinline__ T of_kv(const T (&two)[2], int kv) {
    return kv ? two[1] : two[0];
}

// One warp per (block, kv head, K or V): the new rows of the block in
// registers (D / 16 loads of 16 bytes a lane, all in flight together), their
// largest magnitude, the scale, then the codes.  Only a block whose scale
// grows has its older rows read and rounded again.
template <int F, int D>
__global__ void __launch_bounds__(64) kv_append_kernel(const KvAppendParams prm) {
    constexpr int kLanes = D / 8;            // lanes of a row: 8 halves each
    constexpr int kRows = 32 / kLanes;       // rows of a pass
    constexpr int kPasses = kBlockSize / kRows;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int kv = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int kvh = blockIdx.y, b = blockIdx.z;
    const int ctx = __ldg(prm.context_lens + b);
    const int q0 = __ldg(prm.query_start_loc + b), q1 = __ldg(prm.query_start_loc + b + 1);
    const long long end = (long long)ctx + q1 - q0;
    if (ctx < 0 || q0 < 0 || q1 < q0 || q1 > prm.num_tokens || q1 - q0 > prm.max_query_len ||
        end > (long long)prm.max_blocks_per_seq * kBlockSize) {
        if (blockIdx.x == 0 && kvh == 0 && threadIdx.x == 0) atomicOr(prm.status, PA_DEV_BAD_SEQ_LEN);
        return;
    }
    const int blk = ctx / kBlockSize + (int)blockIdx.x;
    const long long p0 = (long long)blk * kBlockSize;  // position of the block's slot 0
    if (q1 == q0 || p0 >= end) return;
    const int lo = p0 < ctx ? (int)(ctx - p0) : 0;  // the block's new slots: [lo, hi)
    const int hi = end - p0 < kBlockSize ? (int)(end - p0) : kBlockSize;
    const int phys = __ldg(prm.block_tables + (size_t)b * prm.max_blocks_per_seq + blk);
    if (phys < 0 || (long long)phys >= prm.num_blocks) {
        if (kvh == 0 && threadIdx.x == 0) atomicOr(prm.status, PA_DEV_BAD_BLOCK_ID);
        return;
    }
    const size_t bh = (size_t)phys * prm.num_kv_heads + kvh;
    const int sub = lane / kLanes, col = lane % kLanes;
    const __half* src = of_kv(prm.fresh, kv) + ((size_t)(q0 + (p0 - ctx)) * prm.num_kv_heads + kvh) * D + 8 * col;
    const size_t step = (size_t)prm.num_kv_heads * D;

    uint4 x[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int r = i * kRows + sub;
        x[i] = (r >= lo && r < hi) ? __ldg(reinterpret_cast<const uint4*>(src + r * step)) : make_uint4(0u, 0u, 0u, 0u);
    }
    if constexpr (F == PA_KV_F16) {
        __half* dst = static_cast<__half*>(of_kv(prm.cache, kv)) + bh * kBlockSize * D + 8 * col;
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const int r = i * kRows + sub;
            if (r >= lo && r < hi) *reinterpret_cast<uint4*>(dst + r * D) = x[i];
        }
    } else {
        float* scale = of_kv(prm.scales, kv) + bh;
        const float s0 = lo > 0 ? *scale : 0.f;
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const __half* h = reinterpret_cast<const __half*>(&x[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float a = fabsf(__half2float(h[j]));
                if (a <= 65504.f) amax = fmaxf(amax, a);  // finite ones only
            }
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, off));
        const float s1 = fmaxf(s0, block_scale<F>(amax));
        const Unit u(s1);
        uint8_t* dst = static_cast<uint8_t*>(of_kv(prm.cache, kv)) + bh * kBlockSize * D + 8 * col;
        if (s1 > s0 && lo > 0) {
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                const int r = i * kRows + sub;
                if (r < lo) {
                    uint2 w = *reinterpret_cast<const uint2*>(dst + r * D);
                    w.x = recode<F>(w.x, s0, u);
                    w.y = recode<F>(w.y, s0, u);
                    *reinterpret_cast<uint2*>(dst + r * D) = w;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const int r = i * kRows + sub;
            if (r >= lo && r < hi) {
                const __half* h = reinterpret_cast<const __half*>(&x[i]);
                uint32_t w[2] = {0u, 0u};
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j >> 2] |= code_of<F>(u.of(__half2float(h[j]))) << (8 * (j & 3));
                *reinterpret_cast<uint2*>(dst + r * D) = make_uint2(w[0], w[1]);
            }
        }
        __syncwarp();  // every lane has read the old scale
        if (lane == 0) *scale = s1;
    }
}

// An 8-bit context block to halves (values above fp16's range become its
// largest), and the copy's block table.  One warp per (block, kv head, K or V).
template <int F, int D>
__global__ void __launch_bounds__(64) kv_expand_kernel(const KvExpandParams prm) {
    constexpr int kPasses = kBlockSize * D / (32 * 16);  // 16 codes a lane
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int kv = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int blk = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z;
    const int to = b * prm.blocks_per_seq + blk;
    if (kvh == 0 && threadIdx.x == 0) prm.tables[to] = to;
    const int ctx = __ldg(prm.context_lens + b);
    // a context out of range is reported and skipped by the prefill kernel
    if (ctx < 0 || ctx > prm.max_context_len || blk * kBlockSize >= ctx) return;
    const int phys = __ldg(prm.block_tables + (size_t)b * prm.max_blocks_per_seq + blk);
    if (phys < 0 || (long long)phys >= prm.num_blocks) {
        if (kvh == 0 && threadIdx.x == 0) atomicOr(prm.status, PA_DEV_BAD_BLOCK_ID);
        return;
    }
    const size_t bh = (size_t)phys * prm.num_kv_heads + kvh;
    const uint4* src = reinterpret_cast<const uint4*>(of_kv(prm.cache, kv) + bh * kBlockSize * D) + lane;
    uint4 x[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) x[i] = __ldg(src + 32 * i);
    const float s = __ldg(of_kv(prm.scales, kv) + bh);
    uint4* dst = reinterpret_cast<uint4*>(of_kv(prm.expanded, kv) + ((size_t)to * prm.num_kv_heads + kvh) * kBlockSize * D);
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        __half2 h[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t two = w[j >> 1] >> (16 * (j & 1));
            const float a = value_of<F>(two & 0xffu) * s, c = value_of<F>((two >> 8) & 0xffu) * s;
            // (fminf and fmaxf would turn a NaN code into a number)
            h[j] = __floats2half2_rn(fabsf(a) > 65504.f ? copysignf(65504.f, a) : a,
                                     fabsf(c) > 65504.f ? copysignf(65504.f, c) : c);
        }
        const uint4* r = reinterpret_cast<const uint4*>(h);
        dst[2 * (32 * i + lane)] = r[0];
        dst[2 * (32 * i + lane) + 1] = r[1];
    }
}

// What a sequence keeps (see pa_kv_evict); false: nothing, or out of range.
struct KeepPlan {
    int L, k, sinks, recent;
    bool bad;
    __device__ KeepPlan(const KvEvictParams& prm, int b) {
        L = __ldg(prm.seq_lens + b);
        const int want = __ldg(prm.keep_lens + b);
        bad = L < 0 || L > prm.max_seq_len || L > (long long)prm.max_blocks_per_seq * kBlockSize || want < 0 ||
              want > prm.max_keep_len;
        k = min(want, L);
        recent = min(prm.recent, k);
        sinks = min(prm.sinks, k - recent);
    }
};

// Weights as unsigned numbers of the same order: NaN as -infinity, -0 as +0.
__device__ __forceinline__ uint32_t order_key(float w) {
    if (w != w) w = -INFINITY;
    const uint32_t u = __float_as_uint(w + 0.f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// The k - r - s heaviest tokens between the first s and the last r, by a
// radix select over the weights' ordered bits: three rounds of a histogram
// (11, 11 and 10 bits) find the smallest kept key T and how many of the
// tokens that equal it are kept (the first ones); then a scan over the
// positions writes the kept ones in order.  A cluster of `CS` blocks shares a
// (sequence, kv head): each takes a stretch of the positions, the histograms
// are summed through distributed shared memory, and a block's first output
// follows from its predecessors' counts.  Integer counts only, so the result
// does not depend on the order of the atomics.
constexpr int kBins = 2048;

__global__ void __launch_bounds__(kEvictThreads) kv_evict_select_kernel(const KvEvictParams prm) {
    __shared__ unsigned hist[kBins];
    __shared__ unsigned warp_a[32], warp_b[32];
    __shared__ unsigned found[2];    // bin, tokens above it
    __shared__ unsigned counts[2];   // this block's kept for sure, and ties
    cg::cluster_group cluster = cg::this_cluster();
    const int CS = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int kvh = blockIdx.x / CS, b = blockIdx.y;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const KeepPlan plan(prm, b);
    if (plan.bad) {  // the whole cluster leaves here
        if (blockIdx.x == 0 && tid == 0) atomicOr(prm.status, PA_DEV_BAD_SEQ_LEN);
        return;
    }
    const int L = plan.L, k = plan.k;
    if (blockIdx.x == 0 && tid == 0) prm.new_lens[b] = k;
    const size_t row = (size_t)b * prm.num_kv_heads + kvh;
    const float* w = prm.weights + row * prm.weights_stride;
    int32_t* kept = prm.kept + row * prm.max_keep_len;
    float* dst_w = prm.dst_weights ? prm.dst_weights + row * prm.dst_weights_stride : nullptr;

    // this block's stretch of the tokens between sinks and recent ones
    const int m0 = plan.sinks, m1 = L - plan.recent, mid = m1 - m0;
    const int each = (mid + CS - 1) / CS;
    const int t0 = min(m1, m0 + rank * each), t1 = min(m1, t0 + each);
    unsigned need = (unsigned)(k - plan.recent - plan.sinks);  // of the mid tokens

    // sinks and recent ones keep their order around the rest
    for (int i = rank * kEvictThreads + tid; i < plan.sinks; i += CS * kEvictThreads) {
        kept[i] = i;
        if (dst_w) dst_w[i] = w[i];
    }
    for (int i = rank * kEvictThreads + tid; i < plan.recent; i += CS * kEvictThreads) {
        const int at = k - plan.recent + i, t = L - plan.recent + i;
        kept[at] = t;
        if (dst_w) dst_w[at] = w[t];
    }
    if (need == 0) return;  // the same for the whole cluster

    uint32_t T = 0;       // the keys that are kept for sure are above T
    unsigned ties = need; // of those equal to T, so many
    if (need < (unsigned)mid) {
        uint32_t prefix = 0, mask = 0;
#pragma unroll 1
        for (int round = 0; round < 3; ++round) {
            const int shift = round == 0 ? 21 : round == 1 ? 10 : 0;
            const int bins = round == 2 ? 1024 : 2048;
            for (int i = tid; i < kBins; i += kEvictThreads) hist[i] = 0;
            __syncthreads();
            for (int t = t0 + tid; t < t1; t += kEvictThreads) {
                const uint32_t key = order_key(w[t]);
                if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & (bins - 1)], 1u);
            }
            cluster.sync();
            // bins in descending order: thread i sums bins 2 i, 2 i + 1 from the top
            unsigned v[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int bin = kBins - 1 - (2 * tid + j);
                v[j] = 0;
                for (int r = 0; r < CS; ++r) v[j] += cluster.map_shared_rank(hist, r)[bin];
            }
            unsigned pair = v[0] + v[1], incl = pair;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const unsigned up = __shfl_up_sync(kFull, incl, off);
                if (lane >= off) incl += up;
            }
            if (lane == 31) warp_a[warp] = incl;
            __syncthreads();
            if (warp == 0) {
                unsigned x = warp_a[lane];
                const unsigned own = x;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const unsigned up = __shfl_up_sync(kFull, x, off);
                    if (lane >= off) x += up;
                }
                warp_b[lane] = x - own;
            }
            __syncthreads();
            const unsigned above = warp_b[warp] + incl - pair;  // in the bins before this thread's
            if (above < need && need <= above + pair) {
                const bool first = need <= above + v[0];
                found[0] = (unsigned)(kBins - 1 - (2 * tid + (first ? 0 : 1)));
                found[1] = above + (first ? 0u : v[0]);
            }
            cluster.sync();  // also: every block has read the histograms before they are cleared
            prefix |= found[0] << shift;
            mask |= (uint32_t)(bins - 1) << shift;
            need -= found[1];
            __syncthreads();
        }
        T = prefix;
        ties = need;
    }
    // need == mid: T = 0 is below every key but key 0, which no weight has, so all are kept for sure
    // counts of the stretch, then its start in the output
    unsigned sure = 0, tie = 0;
    for (int t = t0 + tid; t < t1; t += kEvictThreads) {
        const uint32_t key = order_key(w[t]);
        sure += key > T;
        tie += key == T;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        sure += __shfl_xor_sync(kFull, sure, off);
        tie += __shfl_xor_sync(kFull, tie, off);
    }
    if (lane == 0) {
        warp_a[warp] = sure;
        warp_b[warp] = tie;
    }
    __syncthreads();
    if (tid == 0) {
        unsigned a = 0, c = 0;
        for (int i = 0; i < kEvictThreads / 32; ++i) {
            a += warp_a[i];
            c += warp_b[i];
        }
        counts[0] = a;
        counts[1] = c;
    }
    cluster.sync();
    unsigned sure_before = 0, tie_before = 0;
    for (int r = 0; r < rank; ++r) {
        sure_before += cluster.map_shared_rank(counts, r)[0];
        tie_before += cluster.map_shared_rank(counts, r)[1];
    }
    for (int base = t0; base < t1; base += kEvictThreads) {
        const int t = base + tid;
        const float wt = t < t1 ? w[t] : 0.f;
        const uint32_t key = order_key(wt);
        const bool s = t < t1 && key > T, e = t < t1 && key == T;
        const unsigned bs = __ballot_sync(kFull, s), be = __ballot_sync(kFull, e);
        if (lane == 0) {
            warp_a[warp] = __popc(bs);
            warp_b[warp] = __popc(be);
        }
        __syncthreads();
        unsigned a = 0, c = 0, ta = 0, tc = 0;
        for (int i = 0; i < kEvictThreads / 32; ++i) {
            const unsigned x = warp_a[i], y = warp_b[i];
            a += i < warp ? x : 0u;
            c += i < warp ? y : 0u;
            ta += x;
            tc += y;
        }
        const unsigned below = (1u << lane) - 1u;
        const unsigned my_sure = sure_before + a + __popc(bs & below), my_tie = tie_before + c + __popc(be & below);
        if (s || (e && my_tie < ties)) {
            const unsigned at = plan.sinks + my_sure + min(my_tie, ties);
            kept[at] = t;
            if (dst_w) dst_w[at] = wt;
        }
        sure_before += ta;
        tie_before += tc;
        __syncthreads();
    }
    cluster.sync();  // no block leaves while another may still read its counts
}

// The kept rows to their new blocks.  One warp per (destination block, kv
// head, K or V).
template <int F, int D>
__global__ void __launch_bounds__(64) kv_evict_move_kernel(const KvEvictParams prm) {
    constexpr int kElem = F == PA_KV_F16 ? 2 : 1;
    constexpr int kLanes = D * kElem / 16;  // lanes of a row: 16 bytes each
    constexpr int kRows = 32 / kLanes;
    constexpr int kPasses = kBlockSize / kRows;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int kv = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int blk = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z;
    const KeepPlan plan(prm, b);
    if (plan.bad || blk * kBlockSize >= plan.k) return;
    const int n = min(kBlockSize, plan.k - blk * kBlockSize);
    const size_t row = (size_t)b * prm.num_kv_heads + kvh;
    // lane r < 16: where the block's r-th row comes from
    int from = -1, slot = 0;
    if (lane < n) {
        const int t = prm.kept[row * prm.max_keep_len + blk * kBlockSize + lane];
        slot = t % kBlockSize;
        from = __ldg(prm.block_tables + (size_t)b * prm.max_blocks_per_seq + t / kBlockSize);
        if (from < 0 || (long long)from >= prm.src_blocks) {
            atomicOr(prm.status, PA_DEV_BAD_BLOCK_ID);
            from = -1;
        }
    }
    const int to = __ldg(prm.dst_block_tables + (size_t)b * prm.dst_max_blocks_per_seq + blk);
    if (to < 0 || (long long)to >= prm.dst_blocks) {
        if (lane == 0) atomicOr(prm.status, PA_DEV_BAD_BLOCK_ID);
        return;
    }
    const size_t dst_bh = (size_t)to * prm.num_kv_heads + kvh;
    const int sub = lane / kLanes, col = lane % kLanes;
    const uint8_t* src = static_cast<const uint8_t*>(of_kv(prm.src, kv));
    uint8_t* dst = static_cast<uint8_t*>(of_kv(prm.dst, kv)) + dst_bh * kBlockSize * D * kElem + 16 * col;
    uint4 x[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int r = i * kRows + sub;
        const int f = __shfl_sync(kFull, from, r), s = __shfl_sync(kFull, slot, r);
        const size_t at = (((size_t)max(f, 0) * prm.num_kv_heads + kvh) * kBlockSize + s) * D * kElem + 16 * col;
        x[i] = f >= 0 ? __ldg(reinterpret_cast<const uint4*>(src + at)) : make_uint4(0u, 0u, 0u, 0u);
    }
    if constexpr (F != PA_KV_F16) {
        float s0 = from >= 0 ? __ldg(of_kv(prm.src_scales, kv) + (size_t)from * prm.num_kv_heads + kvh) : 0.f;
        float s1 = s0;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s1 = fmaxf(s1, __shfl_xor_sync(kFull, s1, off));
        const Unit u(s1);
        if (lane == 0) of_kv(prm.dst_scales, kv)[dst_bh] = s1;
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const float s = __shfl_sync(kFull, s0, i * kRows + sub);
            if (s != s1) {
                x[i].x = recode<F>(x[i].x, s, u);
                x[i].y = recode<F>(x[i].y, s, u);
                x[i].z = recode<F>(x[i].z, s, u);
                x[i].w = recode<F>(x[i].w, s, u);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int r = i * kRows + sub;
        const int f = __shfl_sync(kFull, from, r);
        if (f >= 0) *reinterpret_cast<uint4*>(dst + r * D * kElem) = x[i];
    }
}

template <typename P>
cudaError_t launch(void (*kern)(P), const P& prm, dim3 grid, int threads, int cluster, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2] = {pdl_attribute(), {}};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cluster > 0) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = cluster;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    return cudaLaunchKernelEx(&cfg, kern, prm);
}

}  // namespace

#define PA_FOR_D(F_, K_)                                                                                    \
    if (format == F_ && head_dim == 64) return launch(K_<F_, 64>, prm, grid, 64, 0, stream);                \
    if (format == F_ && head_dim == 128) return launch(K_<F_, 128>, prm, grid, 64, 0, stream);              \
    if (format == F_ && head_dim == 256) return launch(K_<F_, 256>, prm, grid, 64, 0, stream);

cudaError_t launch_kv_append(int format, int head_dim, const KvAppendParams& prm, dim3 grid, cudaStream_t stream) {
    PA_FOR_D(PA_KV_F16, kv_append_kernel)
    PA_FOR_D(PA_KV_E4M3, kv_append_kernel)
    PA_FOR_D(PA_KV_INT8, kv_append_kernel)
    return cudaErrorInvalidValue;
}

cudaError_t launch_kv_expand(int format, int head_dim, const KvExpandParams& prm, dim3 grid, cudaStream_t stream) {
    PA_FOR_D(PA_KV_E4M3, kv_expand_kernel)
    PA_FOR_D(PA_KV_INT8, kv_expand_kernel)
    return cudaErrorInvalidValue;
}

cudaError_t launch_kv_evict_select(const KvEvictParams& prm, int num_seqs, int cluster, cudaStream_t stream) {
    return launch(kv_evict_select_kernel, prm, dim3(prm.num_kv_heads * cluster, num_seqs), kEvictThreads, cluster,
                  stream);
}

cudaError_t launch_kv_evict_move(int format, int head_dim, const KvEvictParams& prm, dim3 grid, cudaStream_t stream) {
    PA_FOR_D(PA_KV_F16, kv_evict_move_kernel)
    PA_FOR_D(PA_KV_E4M3, kv_evict_move_kernel)
    PA_FOR_D(PA_KV_INT8, kv_evict_move_kernel)
    return cudaErrorInvalidValue;
}

}  // namespace pa
