// Linear attention with a decay a kv head over packed chunks of new tokens, on the
// 5th-generation tensor cores (pa_linear_prefix).
//
// A sequence's new tokens are cut into blocks of 256.  With S_n the state before
// block n, L tokens in it, token i of a block and d = exp(g):
//     A_n     = sum_i d^(L - 1 - i) k_i v_i^T            (what the block adds)
//     S_(n+1) = d^L S_n + A_n
//     out_i   = scale (d^(i + 1) q_i S_n + sum_{j <= i} d^(i - j) (q_i . k_j) v_j)
// in three launches: the sums A of all blocks at once, the chain of states
// (elementwise along a sequence), and the outputs of all blocks at once.  Nothing
// is sequential but the chain, so one long prompt fills the device as a batch does.
// What that costs is the states' traffic, 12 D^2 bytes a block and kv head beside
// the 4 (1 + G) * 256 * D of its tokens: blocks half as long would double it,
// longer ones square the products inside a block.
//
// Precision.  The states are 32-bit values that a user keeps, so A's operand
// d^(L-1-i) v_i goes to the tensor cores as two halves, its nearest and the nearest
// of the rest (22 bits), times a power of two for each column of v that brings the
// column's largest into fp16's upper range; k is exact.  The outputs are fp16:
// their operands d^(i-j) (q_i . k_j) and S_n are rounded once, to fp16 as the outputs
// themselves are, also after powers of two (of a row, of a state) that take
// overflow and underflow out of it.
#include "pa_decode.h"

#include "pa_device.cuh"
#include "pa_step.h"
#include "pa_tcgen05.cuh"

namespace pa {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127
// floor(log2 |x|) for normal x, -127 for less, 128 for infinities
__device__ __forceinline__ int exponent_of(float x) { return (int)((__float_as_uint(x) >> 23) & 255u) - 127; }

// A sequence's rows and slot; false where there is nothing to do for it.
struct Seq {
    int first, count, slot, context;
};
__device__ __forceinline__ bool seq_of(const LinearParams& p, int b, Seq& s, unsigned& status) {
    s.first = __ldg(p.query_start_loc + b);
    const int last = __ldg(p.query_start_loc + b + 1);
    s.slot = __ldg(p.slots + b);
    s.context = __ldg(p.context_lens + b);
    s.count = last - s.first;
    status = 0;
    if (s.slot < 0) return false;
    if (s.slot >= p.num_slots) status |= PA_DEV_BAD_BLOCK_ID;
    if (s.first < 0 || last < s.first || last > p.num_tokens || s.count > p.max_query_len || s.context < 0)
        status |= PA_DEV_BAD_SEQ_LEN;
    return status == 0 && s.count > 0;
}

// The block of a number: sequence, its place in it, its tokens.
struct Block {
    int b, n, first, count, context;
};
__device__ __forceinline__ bool block_of(const LinearParams& p, int number, Block& k) {
    int lo = 0, hi = p.num_seqs;  // the last sequence whose numbers start at or before it
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        (__ldg(p.query_start_loc + mid) / kLinearBlock + mid <= number ? lo : hi) = mid;
    }
    Seq s;
    unsigned status;
    if (!seq_of(p, lo, s, status)) return false;
    k.b = lo;
    k.n = number - s.first / kLinearBlock - lo;
    if (k.n < 0 || (long long)k.n * kLinearBlock >= s.count) return false;
    k.first = s.first + k.n * kLinearBlock;
    k.count = min(kLinearBlock, s.count - k.n * kLinearBlock);
    k.context = s.context;
    return true;
}

// ---- what the blocks add

template <int D>
struct AddShape {
    static constexpr int kTile = D < kLinearTile ? D : kLinearTile;
    static constexpr int kTiles = D / kTile;
    static constexpr int kKBytes = kLinearBlock * kTile * 2;
    // two CTAs an SM, whose TMEM allocations then always fit
    static constexpr int kSmem = (kKBytes > 78 * 1024 ? kKBytes : 78 * 1024) + 2048 + 1024;
    static constexpr int kTmem = 256;  // the sum, and 128 tokens of v in two halves
};

// A CTA has a tile of (128 columns of k) x (128 columns of v) of a block's sum.
// Lane (thread) c of the accumulator is a column of v: the thread reads that column of
// the block's tokens, 64 contiguous bytes a warp and token, scales it and writes it to
// tensor memory as the MMA's A operand (two halves, 128 tokens at a time); k is the B
// operand as TMA brings it, token by token.  CTAs past the blocks find the largest
// entries of the sequences' first states.
template <int D>
__global__ void __launch_bounds__(128, 2)
    linear_adds_kernel(const __grid_constant__ CUtensorMap tmap_k, const LinearChunkParams c) {
    using S = AddShape<D>;
    const LinearParams& p = c.lin;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ks = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    float* w = reinterpret_cast<float*>(ks + S::kKBytes);
    uint64_t* bars = reinterpret_cast<uint64_t*>(w + kLinearBlock);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + 2);
    volatile int* failed = reinterpret_cast<volatile int*>(tslot + 1);
    float* red = reinterpret_cast<float*>(tslot + 2);
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31, kvh = blockIdx.y, number = blockIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");

    auto block_max = [&](float m) {
#pragma unroll
        for (int d = 16; d; d /= 2) m = fmaxf(m, __shfl_xor_sync(kFull, m, d));
        if (lane == 0) red[warp] = m;
        __syncthreads();
        return fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    };
    auto finite_max = [](float m, float x) {
        const float a = fabsf(x);
        return a <= 3.402823466e38f ? fmaxf(m, a) : m;
    };
    if (number >= c.blocks) {
        const int b = number - c.blocks;
        Seq s;
        unsigned status;
        if (blockIdx.z != 0 || !seq_of(p, b, s, status)) return;
        float m = 0.f;
        if (s.context > 0) {
            const float4* st = reinterpret_cast<const float4*>(p.states + ((size_t)s.slot * p.num_kv_heads + kvh) * D * D);
#pragma unroll 8
            for (int i = t; i < D * D / 4; i += 128) {
                const float4 x = st[i];
                m = finite_max(finite_max(finite_max(finite_max(m, x.x), x.y), x.z), x.w);
            }
        }
        m = block_max(m);
        if (t == 0) c.state_max[(size_t)b * p.num_kv_heads + kvh] = m;
        return;
    }
    Block k;
    if (!block_of(p, number, k)) return;
    const int k_tile = blockIdx.z / S::kTiles, v_tile = blockIdx.z % S::kTiles;
    const uint32_t bar_k = smem_addr(bars), bar_mma = bar_k + 8;
    if (t == 0) {
        *failed = 0;
        mbar_init(bar_k, 1);
        mbar_init(bar_mma, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        mbar_arrive_expect_tx(bar_k, S::kKBytes);
        tc_tma_load_4d(smem_addr(ks), &tmap_k, 0, kvh, k.first, k_tile * (S::kTile / 64), bar_k);
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tslot)), "r"(S::kTmem)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    // 64 tokens of the thread's column, in pairs; none past the block.  Read twice, for the column's
    // largest and for the operand: 256 tokens at once would not fit in registers.
    const bool mine = t < S::kTile;
    const size_t row = (size_t)p.num_kv_heads * D;
    const unsigned short* col = reinterpret_cast<const unsigned short*>(p.v) + (size_t)k.first * row + (size_t)kvh * D +
                                v_tile * S::kTile + t;
    auto read = [&](int first, uint32_t(&v)[32]) {
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const int at = first + 2 * i;
            const unsigned a = mine && at < k.count ? __ldg(col + at * row) : 0;
            const unsigned b = mine && at + 1 < k.count ? __ldg(col + (at + 1) * row) : 0;
            v[i] = a | b << 16;
        }
    };
    const float g = fmaxf(__ldg(p.log_decay + kvh), -1e4f);  // (whose exp is 0, and 1 for no tokens)
    for (int i = t; i < kLinearBlock; i += 128) w[i] = i < k.count ? expf(g * (float)(k.count - 1 - i)) : 0.f;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot, lanes = (uint32_t)(warp * 32) << 16;
    const uint32_t t_sum = tmem, t_v = tmem + 128;

    auto halves = [](uint32_t x) { return __half22float2(*reinterpret_cast<const __half2*>(&x)); };
    float m = 0.f;
    int first = kLinearBlock;  // token with a NaN or infinity
#pragma unroll 1
    for (int at = 0; at < k.count; at += 64) {
        uint32_t v[32];
        read(at, v);
        bool bad = false;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const float2 x = halves(v[i]);
            const float2 wi = *reinterpret_cast<const float2*>(w + at + 2 * i);
            bad |= !(fabsf(x.x) <= 65504.f) || !(fabsf(x.y) <= 65504.f);
            m = finite_max(finite_max(m, x.x * wi.x), x.y * wi.y);
        }
        if (bad && first == kLinearBlock) {
#pragma unroll
            for (int i = 31; i >= 0; --i) {
                if ((v[i] & 0x7c000000u) == 0x7c000000u) first = at + 2 * i + 1;
                if ((v[i] & 0x7c00u) == 0x7c00u) first = at + 2 * i;
            }
        }
    }
    const int up = m > 0.f ? min(13 - exponent_of(m), 100) : 0;
    const float raise = pow2(up), lower = pow2(-up);
    if (k_tile == 0 && mine)
        c.first_bad[((size_t)number * p.num_kv_heads + kvh) * D + v_tile * S::kTile + t] = first;

    constexpr uint32_t id = tc_idesc(128, S::kTile, 1);
    const uint64_t kdesc = tc_desc(smem_addr(ks), kLinearBlock * 128, 1024);
    const int steps = (k.count + 15) / 16;
    bool ok = true;
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
        if (half * 128 < k.count) {
            if (half == 1) {  // the operand's memory is read until the first half's MMAs end
                ok = tc_warp_wait(bar_mma, 0, c.wait_limit, failed);
                tc_fence_after();
            }
#pragma unroll 1
            for (int part = 0; part < 2; ++part) {
                const int at = half * 128 + part * 64;
                uint32_t v[32], hi[32], lo[32];
                read(at, v);
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const float2 x = halves(v[i]);
                    const float2 wi = *reinterpret_cast<const float2*>(w + at + 2 * i);
                    const float a = x.x * wi.x * raise, b = x.y * wi.y * raise;
                    const __half2 h = __floats2half2_rn(a, b);
                    const float2 back = __half22float2(h);
                    hi[i] = half2_bits(h);
                    lo[i] = half2_bits(__floats2half2_rn(a - back.x, b - back.y));
                }
                tc_st32x2(t_v + lanes + part * 32, hi, t_v + lanes + 64 + part * 32, lo);
            }
            if (half == 0) {
                ok = tc_warp_wait(bar_k, 0, c.wait_limit, failed);
                // rows of other sequences behind the block's last token: their v is 0 here, but
                // 0 * NaN is not
                const int tail = steps * 16 - k.count;
                for (int i = t; i < tail * (S::kTile / 8); i += 128) {
                    const int r = k.count + i / (S::kTile / 8), u = i % (S::kTile / 8);
                    *reinterpret_cast<uint4*>(ks + (u >> 3) * (kLinearBlock * 128) + r * 128 + (u & 7) * 16) =
                        make_uint4(0u, 0u, 0u, 0u);
                }
                if (tail) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            }
            if (!ok) *failed = 1;
            tc_fence_before();
            __syncthreads();
            if (t == 0 && !*failed) {
                tc_fence_after();
                const int s0 = half * 8, s1 = min(steps, s0 + 8);
                for (int x = 1; x >= 0; --x)  // the small halves first
                    for (int s = s0; s < s1; ++s)
                        tc_mma_ts(t_sum, t_v + x * 64 + (s - s0) * 8, kdesc + (uint64_t)((s * 2048) >> 4), id,
                                  half > 0 || x == 0 || s > s0);
                tc_commit(bar_mma);
            }
            __syncwarp();
        }
    }
    if (!*failed) {
        ok = tc_warp_wait(bar_mma, k.count > 128 ? 1 : 0, c.wait_limit, failed);
        if (!ok) *failed = 1;
    }
    __syncthreads();
    if (*failed) {
        if (t == 0) atomicOr(p.status, PA_DEV_TIMEOUT);
        // what is in flight lands before the CTA's memory is given back
        mbar_wait(bar_k, 0, kDefaultWaitLimit);
        mbar_wait(bar_mma, k.count > 128 ? 1 : 0, kDefaultWaitLimit);
    }
    tc_fence_after();
    m = 0.f;
    float* dst = c.adds + (((size_t)number * p.num_kv_heads + kvh) * D + k_tile * S::kTile) * D + v_tile * S::kTile + t;
#pragma unroll
    for (int c0 = 0; c0 < S::kTile; c0 += 32) {
        uint32_t x[32];
        tc_ld32(t_sum + lanes + c0, x);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const float y = __uint_as_float(x[i]) * lower;
            if (mine) {
                m = finite_max(m, y);
                dst[(size_t)(c0 + i) * D] = y;
            }
        }
    }
    m = block_max(m);
    if (t == 0) c.add_max[((size_t)number * p.num_kv_heads + kvh) * (S::kTiles * S::kTiles) + blockIdx.z] = m;
    tc_fence_before();
    __syncthreads();
    if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::kTmem));
}

// ---- the chain of states

constexpr int kScanThreads = 256;

// A thread takes four entries of a (sequence, kv head)'s state through its blocks.
// The state before each block goes to the outputs' kernel as halves of S 2^-e; e comes
// from a bound on |S| that runs along (no more than a few bits above it), so that no
// block has to look for the largest entry.
template <int D>
__global__ void __launch_bounds__(kScanThreads) linear_scan_kernel(const LinearChunkParams c) {
    const LinearParams& p = c.lin;
    constexpr int kTiles = AddShape<D>::kTiles * AddShape<D>::kTiles;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int t = threadIdx.x, b = blockIdx.z, kvh = blockIdx.y, at = (blockIdx.x * kScanThreads + t) * 4;
    const bool first = t == 0 && blockIdx.x == 0;
    Seq s;
    unsigned status;
    const bool run = seq_of(p, b, s, status);
    if (status && first && kvh == 0) atomicOr(p.status, status);
    if (!run) return;
    const float g = __ldg(p.log_decay + kvh);
    if (first && !(g <= 0.f)) atomicOr(p.status, PA_DEV_BAD_DECAY);

    float4* state = reinterpret_cast<float4*>(p.states + ((size_t)s.slot * p.num_kv_heads + kvh) * D * D + at);
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    float bound = 0.f;
    if (s.context > 0) {
        x = *state;
        bound = __ldg(c.state_max + (size_t)b * p.num_kv_heads + kvh);
    }
    const int blocks = (s.count + kLinearBlock - 1) / kLinearBlock;
    const size_t index = (size_t)(s.first / kLinearBlock + b) * p.num_kv_heads + kvh;  // of the first block
    const float4* add = reinterpret_cast<const float4*>(c.adds + index * D * D + at);
    const size_t step = (size_t)p.num_kv_heads * D * D;
    float4 next = __ldcs(add);
    for (int n = 0; n < blocks; ++n) {
        const float4 a = next;
        if (n + 1 < blocks) next = __ldcs(add + (n + 1) * step / 4);
        const size_t i = index + (size_t)n * p.num_kv_heads;
        if (n > 0 || s.context > 0) {
            const int e = bound > 0.f ? max(min(exponent_of(bound) - 13, 100), -100) : 0;
            const float down = pow2(-e);
            uint2 h;
            h.x = half2_bits(__floats2half2_rn(x.x * down, x.y * down));
            h.y = half2_bits(__floats2half2_rn(x.z * down, x.w * down));
            *reinterpret_cast<uint2*>(c.starts + i * D * D + at) = h;
            if (first) c.exponents[i] = e;
        }
        // d^L S: next to 1 the factor less 1 is what 32 bits hold
        const float y = fmaxf(g, -1e4f) * (float)min(kLinearBlock, s.count - n * kLinearBlock);
        const float whole = y > -0.5f ? 1.f : 0.f, rest = y > -0.5f ? expm1f(y) : expf(y);
        auto chain = [&](float v, float plus) { return fmaf(v, rest, v * whole) + plus; };
        x = make_float4(chain(x.x, a.x), chain(x.y, a.y), chain(x.z, a.z), chain(x.w, a.w));
        float most = 0.f;
#pragma unroll
        for (int j = 0; j < kTiles; ++j) most = fmaxf(most, __ldg(c.add_max + i * kTiles + j));
        bound = (bound * (whole + rest) + most) * 1.0001f;
    }
    *state = x;
}

// ---- the outputs

template <int D>
struct OutShape {
    static constexpr int kCols = D < 128 ? D : 128;      // of v and out, of a CTA
    static constexpr int kSplits = D / kCols;
    static constexpr int kQBytes = 128 * D * 2;
    static constexpr int kStageBytes = 64 * kCols * 2;   // 64 tokens or state rows by kCols columns
    static constexpr int kSlots = D == 256 ? 3 : D == 128 ? 5 : 8;
    static constexpr int kBars = 9 + 2 * kSlots;
    static constexpr int kCtrl = kCols * 4 + kBars * 8 + 16 + 256;  // first_bad, barriers, TMEM address and flag, d^(63-j)
    static constexpr int kSmem = kQBytes + kSlots * kStageBytes + kCtrl;
    static constexpr int kTmem = 256;                    // kCols of the outputs, two buffers of 64 scores
    static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two CTAs an SM");
};
constexpr int kOutRowWarps = 4, kOutThreads = (kOutRowWarps + 2) * 32;

enum : int { kBarQ = 0, kBarInter, kBarScores, kBarP = kBarScores + 2, kBarPV = kBarP + 2, kBarDrain = kBarPV + 2, kBarFull };

// A CTA has 128 tokens (a half of a block) of one query head and 128 columns of v.
// Its 128 rows are the lanes of the accumulator.  Warp 5 brings Q, then in stages of
// 64 rows the K tiles of 64 keys, the state's rows and the V tiles, in the order in
// which warp 4 feeds them to the tensor cores: scores of the first key tile; Q S_n;
// then for each key tile P V and the scores of the tile after the next, in the
// score buffer that P V has left.  Warps 0-3 own a row a thread, turn its scores into
// P, in fp16 over the scores, and keep the accumulator in the row's power of two.  Key
// tiles go from the row's own backwards, where scores only shrink by the decay, so that
// the first one nearly always sets that power.
template <int D>
__global__ void __launch_bounds__(kOutThreads, 2)
    linear_out_kernel(const __grid_constant__ LinearMaps maps, const LinearChunkParams c) {
    using S = OutShape<D>;
    const LinearParams& p = c.lin;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* qs = smem;
    uint8_t* ring = qs + S::kQBytes;
    float* falling = reinterpret_cast<float*>(ring + S::kSlots * S::kStageBytes);  // d^(63 - j)
    int* first_bad = reinterpret_cast<int*>(falling + 64);
    uint64_t* bars = reinterpret_cast<uint64_t*>(first_bad + S::kCols);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + S::kBars);
    volatile int* failed = reinterpret_cast<volatile int*>(tslot + 1);
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int G = p.group, H = p.num_heads, K = p.num_kv_heads;
    unsigned x = blockIdx.x;
    const int split = x % S::kSplits;
    x /= S::kSplits;
    const int head = x % G;
    x /= G;
    const int r = x % 2;  // which half of the block
    x /= 2;
    const int kvh = x % K, number = x / K;
    Block k;
    if (!block_of(p, number, k) || r * 128 >= k.count) return;
    if (smem_addr(smem) & 1023u) {  // (the layouts need it; no launch has been seen to break it)
        if (t == 0) atomicOr(p.status, PA_DEV_TIMEOUT);
        return;
    }
    const size_t index = (size_t)number * K + kvh;
    const bool inter = k.n > 0 || k.context > 0;
    const int tiles = (min(k.count, r * 128 + 128) - 1) / 64 + 1;  // key tiles
    const float l2 = fmaxf(__ldg(p.log_decay + kvh) * kLog2e, -1e6f);
    const uint32_t bar0 = smem_addr(bars);
    auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
    constexpr int kBarEmpty = kBarFull + S::kSlots;
    if (t == 0) {
        *failed = 0;
        for (int i = 0; i < S::kBars; ++i) mbar_init(bar(i), i == kBarP || i == kBarP + 1 ? kOutRowWarps : 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tslot)), "r"(S::kTmem)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    int bad = 0;
    if (t < S::kCols) {
        first_bad[t] = __ldg(c.first_bad + index * D + split * S::kCols + t);
        bad = first_bad[t] < kLinearBlock;
    }
    if (t < 64) falling[t] = exp2f(l2 * (float)(63 - t));
    tc_fence_before();
    const bool dirty = __syncthreads_or(bad);  // a column of v with a NaN or infinity
    tc_fence_after();
    const uint32_t tmem = *tslot, t_out = tmem, t_s = tmem + S::kCols;
    const unsigned limit = c.wait_limit;
    constexpr int kKStages = D / S::kCols;  // stages of a key tile
    const int inter_stages = inter ? D / 64 : 0;
    // stage of V tile j: behind the first two K tiles, the state and the V and K tiles before it
    auto v_stage = [&](int j) { return kKStages * min(tiles, 2) + inter_stages + j + kKStages * min(j, max(tiles - 2, 0)); };

    if (warp == kOutRowWarps + 1) {
        if (lane == 0) {
            int n = 0;
            bool ok = true;
            auto stage = [&](const CUtensorMap* map, int y, int z, int ch) {
                if (!ok) return;
                if (n >= S::kSlots && !(ok = tc_wait(bar(kBarEmpty + n % S::kSlots), (n / S::kSlots - 1) & 1, limit, failed)))
                    return;
                const uint32_t full = bar(kBarFull + n % S::kSlots);
                mbar_arrive_expect_tx(full, S::kStageBytes);
                tc_tma_load_4d(smem_addr(ring + (n % S::kSlots) * S::kStageBytes), map, 0, y, z, ch, full);
                ++n;
            };
            auto key = [&](int j) { return k.first + (tiles - 1 - j) * 64; };
            auto k_tile = [&](int j) {
                for (int ch = 0; ch < kKStages; ++ch) stage(&maps.k, kvh, key(j), ch * (S::kCols / 64));
            };
            mbar_arrive_expect_tx(bar(kBarQ), S::kQBytes);
            tc_tma_load_4d(smem_addr(qs), &maps.q, 0, kvh * G + head, k.first + r * 128, 0, bar(kBarQ));
            k_tile(0);
            for (int d = 0; d < inter_stages; ++d)
                stage(&maps.starts, 0, (int)(index * D) + d * 64, split * (S::kCols / 64));
            if (tiles > 1) k_tile(1);
            for (int j = 0; j < tiles; ++j) {
                stage(&maps.v, kvh, key(j), split * (S::kCols / 64));
                if (j + 2 < tiles) k_tile(j + 2);
            }
            if (!ok) {
                *failed = 1;
                atomicOr(p.status, PA_DEV_TIMEOUT);
            }
            // every copy lands before the CTA's memory is given back
            mbar_wait(bar(kBarQ), 0, kDefaultWaitLimit);
            for (int i = max(0, n - S::kSlots); i < n; ++i)
                mbar_wait(bar(kBarFull + i % S::kSlots), (i / S::kSlots) & 1, kDefaultWaitLimit);
        }
        __syncwarp();
    } else if (warp == kOutRowWarps) {
        if (lane == 0) {
            constexpr uint32_t id_s = tc_idesc(128, 64, 0), id_o = tc_idesc(128, S::kCols, 1);
            const uint64_t qdesc = tc_desc(smem_addr(qs), 16, 1024);
            const uint64_t kdesc = tc_desc(smem_addr(ring), 16, 1024), vdesc = tc_desc(smem_addr(ring), 64 * 128, 1024);
            int n = 0;
            bool ok = tc_wait(bar(kBarQ), 0, limit, failed);
            auto landed = [&] { return ok = ok && tc_wait(bar(kBarFull + n % S::kSlots), (n / S::kSlots) & 1, limit, failed); };
            auto scores = [&](int j) {
                for (int ch = 0; ch < kKStages; ++ch) {
                    if (!landed()) return;
                    tc_fence_after();
                    const uint64_t at = (uint64_t)((n % S::kSlots) * (S::kStageBytes >> 4));
#pragma unroll
                    for (int i = 0; i < S::kCols / 16; ++i)
                        tc_mma_ss(t_s + (j & 1) * 64,
                                  qdesc + (uint64_t)(((ch * (S::kCols / 64) + (i >> 2)) * (128 * 128) + (i & 3) * 32) >> 4),
                                  kdesc + at + (uint64_t)(((i >> 2) * (64 * 128) + (i & 3) * 32) >> 4), id_s, ch > 0 || i > 0);
                    tc_commit(bar(kBarEmpty + n % S::kSlots));
                    ++n;
                }
                tc_commit(bar(kBarScores + (j & 1)));
            };
            scores(0);
            for (int d = 0; d < inter_stages && landed(); ++d) {
                tc_fence_after();
                const uint64_t at = (uint64_t)((n % S::kSlots) * (S::kStageBytes >> 4));
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    tc_mma_ss(t_out, qdesc + (uint64_t)((d * (128 * 128) + i * 32) >> 4), vdesc + at + (uint64_t)((i * 2048) >> 4),
                              id_o, d > 0 || i > 0);
                tc_commit(bar(kBarEmpty + n % S::kSlots));
                ++n;
            }
            if (inter) tc_commit(bar(kBarInter));
            if (tiles > 1) scores(1);
            for (int j = 0; j < tiles && ok; ++j) {
                ok = tc_wait(bar(kBarP + (j & 1)), (j >> 1) & 1, limit, failed);
                if (!landed()) break;
                tc_fence_after();
                const uint64_t at = (uint64_t)((n % S::kSlots) * (S::kStageBytes >> 4));
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    tc_mma_ts(t_out, t_s + (j & 1) * 64 + i * 8, vdesc + at + (uint64_t)((i * 2048) >> 4), id_o,
                              inter || j > 0 || i > 0);
                tc_commit(bar(kBarEmpty + n % S::kSlots));
                tc_commit(bar(kBarPV + (j & 1)));
                ++n;
                if (j + 2 < tiles) {  // over the P that this P V reads
                    ok = tc_wait(bar(kBarPV + (j & 1)), (j >> 1) & 1, limit, failed);
                    if (ok) scores(j + 2);
                }
            }
            if (!ok) {
                *failed = 1;
                atomicOr(p.status, PA_DEV_TIMEOUT);
            }
            tc_commit(bar(kBarDrain));
            mbar_wait(bar(kBarDrain), 0, kDefaultWaitLimit);
        }
        __syncwarp();
    } else {
        const uint32_t lanes = (uint32_t)(warp * 32) << 16;
        const int i = r * 128 + t;  // the row's token in the block
        const float state_log2 = inter ? (float)__ldg(c.exponents + index) + l2 * (float)(i + 1) : 0.f;
        // The accumulator holds the outputs times 2^-e.  Where the state's part is far larger than the
        // scores, e stays so near that this part does not overflow.
        const int e_least = inter ? (int)fmaxf(-100.f, state_log2 - 60.f) : -100;
        int e = max(0, e_least);
        bool set = false, ok = true;
        auto rescale = [&](float f) {
#pragma unroll 1
            for (int c0 = 0; c0 < S::kCols; c0 += 32) {
                uint32_t o[32];
                tc_ld32(t_out + lanes + c0, o);
#pragma unroll
                for (int u = 0; u < 32; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * f);
                tc_st32(t_out + lanes + c0, o);
            }
        };
        for (int j = 0; j < tiles; ++j) {
            const int k0 = (tiles - 1 - j) * 64;  // first key of the tile
            const uint32_t buf = t_s + (j & 1) * 64 + lanes;
            if (!(ok = tc_warp_wait(bar(kBarScores + (j & 1)), (j >> 1) & 1, limit, failed))) break;
            tc_fence_after();
            uint32_t s0[32], s1[32];
            tc_ld32x2(buf, s0, buf + 32, s1);
            float m = 0.f;
            if (k0 + 63 <= r * 128 + warp * 32) {  // every key of the tile is seen by every row of the warp
                const float base = tc_ex2(l2 * (float)(i - k0 - 63));
#pragma unroll
                for (int u = 0; u < 32; ++u) {
                    s0[u] = __float_as_uint(__uint_as_float(s0[u]) * (base * falling[u]));
                    s1[u] = __float_as_uint(__uint_as_float(s1[u]) * (base * falling[32 + u]));
                }
            } else {
#pragma unroll
                for (int u = 0; u < 32; ++u) {
                    const int d0 = i - k0 - u, d1 = d0 - 32;
                    s0[u] = d0 >= 0 ? __float_as_uint(__uint_as_float(s0[u]) * tc_ex2(l2 * (float)d0)) : 0u;
                    s1[u] = d1 >= 0 ? __float_as_uint(__uint_as_float(s1[u]) * tc_ex2(l2 * (float)d1)) : 0u;
                }
            }
#pragma unroll
            for (int u = 0; u < 32; ++u)
                m = fmaxf(m, fmaxf(fabsf(__uint_as_float(s0[u])), fabsf(__uint_as_float(s1[u]))));
            // e moves where the row has its first scores that are not 0, and where later ones
            // would leave fp16 (the first put their largest at 2^10)
            const int e_new = max(exponent_of(m) - 10, e_least);
            const bool move = m > 0.f && (!set || e_new > e + 4);
            const int e_old = e;
            if (move) {
                e = e_new;
                set = true;
            }
            if (j == 0) {
                if (inter) {
                    if (!(ok = tc_warp_wait(bar(kBarInter), 0, limit, failed))) break;
                    tc_fence_after();
                    rescale(exp2f(state_log2 - (float)e));
                }
            } else if (__any_sync(kFull, move && e != e_old)) {
                if (!(ok = tc_warp_wait(bar(kBarPV + ((j - 1) & 1)), ((j - 1) >> 1) & 1, limit, failed))) break;
                tc_fence_after();
                rescale(exp2f((float)(e_old - e)));
            }
            const float down = pow2(-e);
            uint32_t pk[32];
#pragma unroll
            for (int u = 0; u < 16; ++u) {
                pk[u] = half2_bits(__floats2half2_rn(__uint_as_float(s0[2 * u]) * down, __uint_as_float(s0[2 * u + 1]) * down));
                pk[16 + u] = half2_bits(__floats2half2_rn(__uint_as_float(s1[2 * u]) * down, __uint_as_float(s1[2 * u + 1]) * down));
            }
            tc_st32(buf, pk);
            if (dirty || k0 + 64 > k.count) {
                // V rows behind the block's last token belong to other sequences, and a NaN or infinity
                // must not meet the zeros of tokens before it: both become 0 (the latter's column is
                // set from its token on in the end)
                const int n = v_stage(j);
                if (!(ok = tc_warp_wait(bar(kBarFull + n % S::kSlots), (n / S::kSlots) & 1, limit, failed))) break;
                uint8_t* vt = ring + (n % S::kSlots) * S::kStageBytes;
                for (int u = t; u < S::kStageBytes / 16; u += 128) {
                    const int row = (u >> 3) & 63;
                    uint4* at = reinterpret_cast<uint4*>(vt + (size_t)u * 16);
                    uint4 y = *at;
                    auto clean = [](uint32_t h) {
                        if ((h & 0x7c00u) == 0x7c00u) h &= 0xffff0000u;
                        if ((h & 0x7c000000u) == 0x7c000000u) h &= 0xffffu;
                        return h;
                    };
                    y = k0 + row < k.count ? make_uint4(clean(y.x), clean(y.y), clean(y.z), clean(y.w)) : make_uint4(0u, 0u, 0u, 0u);
                    *at = y;
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kBarP + (j & 1)));
        }
        if (ok) ok = tc_warp_wait(bar(kBarPV + ((tiles - 1) & 1)), ((tiles - 1) >> 1) & 1, limit, failed);
        if (ok) {
            tc_fence_after();
            const float f = p.scale * pow2(e);
            __half* out = p.out + ((size_t)(k.first + i) * H + kvh * G + head) * D + split * S::kCols;
#pragma unroll 1
            for (int c0 = 0; c0 < S::kCols; c0 += 32) {
                uint32_t o[32];
                tc_ld32(t_out + lanes + c0, o);
                if (i < k.count) {
                    if (dirty) {
#pragma unroll
                        for (int u = 0; u < 32; ++u)
                            if (i >= first_bad[c0 + u]) o[u] = 0x7fffffffu;
                    }
#pragma unroll
                    for (int u = 0; u < 32; u += 8) {
                        uint4 y;
                        uint32_t* yp = reinterpret_cast<uint32_t*>(&y);
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            yp[q] = half2_bits(__floats2half2_rn(__uint_as_float(o[u + 2 * q]) * f, __uint_as_float(o[u + 2 * q + 1]) * f));
                        *reinterpret_cast<uint4*>(out + c0 + u) = y;
                    }
                }
            }
        } else if (lane == 0) {
            *failed = 1;
            atomicOr(p.status, PA_DEV_TIMEOUT);
        }
    }
    tc_fence_before();
    __syncthreads();  // no copy or MMA is in flight
    if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::kTmem));
}

template <typename... P, typename... A>
cudaError_t launch(void (*kern)(P...), dim3 grid, int threads, int smem, cudaStream_t stream, const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <int D>
cudaError_t adds(const LinearChunkParams& prm, const LinearMaps& maps, cudaStream_t stream) {
    using S = AddShape<D>;
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = once_per_device(done, [] {
        return cudaFuncSetAttribute(linear_adds_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    });
    if (e != cudaSuccess) return e;
    return launch(linear_adds_kernel<D>, dim3(prm.blocks + prm.lin.num_seqs, prm.lin.num_kv_heads, S::kTiles * S::kTiles), 128,
                  S::kSmem, stream, maps.k_block, prm);
}

template <int D>
cudaError_t out(const LinearChunkParams& prm, const LinearMaps& maps, cudaStream_t stream) {
    using S = OutShape<D>;
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = once_per_device(done, [] {
        return cudaFuncSetAttribute(linear_out_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    });
    if (e != cudaSuccess) return e;
    return launch(linear_out_kernel<D>, dim3((unsigned)prm.blocks * 2 * prm.lin.num_heads * S::kSplits), kOutThreads, S::kSmem,
                  stream, maps, prm);
}

}  // namespace

cudaError_t launch_linear_adds(int head_dim, const LinearChunkParams& prm, const LinearMaps& maps, cudaStream_t stream) {
    switch (head_dim) {
        case 64: return adds<64>(prm, maps, stream);
        case 128: return adds<128>(prm, maps, stream);
        case 256: return adds<256>(prm, maps, stream);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_linear_scan(int head_dim, const LinearChunkParams& prm, cudaStream_t stream) {
    const dim3 grid(head_dim * head_dim / (4 * kScanThreads), prm.lin.num_kv_heads, prm.lin.num_seqs);
    switch (head_dim) {
        case 64: return launch(linear_scan_kernel<64>, grid, kScanThreads, 0, stream, prm);
        case 128: return launch(linear_scan_kernel<128>, grid, kScanThreads, 0, stream, prm);
        case 256: return launch(linear_scan_kernel<256>, grid, kScanThreads, 0, stream, prm);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_linear_out(int head_dim, const LinearChunkParams& prm, const LinearMaps& maps, cudaStream_t stream) {
    switch (head_dim) {
        case 64: return out<64>(prm, maps, stream);
        case 128: return out<128>(prm, maps, stream);
        case 256: return out<256>(prm, maps, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace pa
