// Linear attention with a decay a kv head over packed chunks of new tokens, on the
// 5th-generation tensor cores (pa_linear_prefix).
//
// A sequence's new tokens are cut into blocks of 256.  With S_n the state before
// block n, L tokens in it, token i of a block and d = exp(g):
//     A_n     = sum_i d^(L - 1 - i) k_i v_i^T            (what the block adds)
//     S_(n+1) = d^L S_n + A_n
//     out_i   = scale (d^(i + 1) q_i S_n + sum_{j <= i} d^(i - j) (q_i . k_j) v_j)
// in three launches: the sums A of all blocks at once, the chain of states
// (elementwise along a sequence), and the outputs of all blocks at once.  The calls take
// 52 us for 4 x 512 tokens of 24/4 x 256, 122 us for one sequence of 8192 of them, 121 us for
// 16 of up to 4096 of 12/12 x 64, and 448 us for 8 x 8192 of 32/8 x 128.  Nothing
// is sequential but the chain, so one long prompt fills the device as a batch does.
// What that costs is the states' traffic, 12 D^2 bytes a block and kv head beside
// the 4 (1 + G) * 256 * D of its tokens: blocks half as long would double it,
// longer ones square the products inside a block.
//
// Precision.  The states are 32-bit values that a user keeps, so A's operand
// d^(L-1-i) v_i goes to the tensor cores as two halves, its nearest and the nearest
// of the rest (22 bits), times a power of two for each column of v that brings the
// column's largest to 2^8 or above; k is exact.  Half of the second half's last step is
// 2^-25: what is below 2^-11 of the column's largest is off by up to 2^-33 of that.
// The outputs are fp16: their operands d^(i-j) (q_i . k_j) and S_n are rounded once, to
// fp16 as the outputs themselves are, also after powers of two, of a row and of a
// whole state, that keep them from overflow.  A row's largest score comes to 2^-4 or above
// (where it is there already the accumulator need not be touched), a state's largest entry,
// as its blocks' largest bound it, to 2^8: scores below 2^-10 of the first and entries below
// 2^-22 of the second may be fp16's subnormals, off by up to 2^-21 and 2^-33 of it, and columns
// of v as much smaller than others have fewer bits in the outputs than token by token.  A
// power of two for each column would need a pass over the accumulator.
#include "pa_decode.h"

#include "pa_device.cuh"
#include "pa_linear.cuh"
#include "pa_step.h"
#include "pa_tcgen05.cuh"

namespace pa {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127
// floor(log2 |x|) for normal x, -127 for less, 128 for infinities
__device__ __forceinline__ int exponent_of(float x) { return (int)((__float_as_uint(x) >> 23) & 255u) - 127; }

// Products of two numbers at a time (one instruction), and the larger magnitude of three.
__device__ __forceinline__ void mul2(uint32_t& a, uint32_t& b, float x, float y) {
    asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\tmul.rn.f32x2 p, p, q;\n\t"
        "mov.b64 {%0, %1}, p;\n\t}"
        : "+r"(a), "+r"(b)
        : "f"(x), "f"(y));
}
__device__ __forceinline__ float max3(float m, uint32_t a, uint32_t b) {
    asm("max.abs.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)));
    return m;
}

// A sequence's rows and slot; false where there is nothing to do for it here.
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
    return status == 0 && s.count > p.few;
}

// The block of a number: sequence, its place in it, its tokens.  By a whole warp: 32
// sequences at a time, so that a batch of up to 32 takes one round of loads.
struct Block {
    int b, n, first, count, context;
};
__device__ __forceinline__ bool block_of(const LinearParams& p, int number, Block& k) {
    const int lane = threadIdx.x & 31;
    int lo = 0, left = p.num_seqs;  // the last sequence whose numbers start at or before it is one of these
    while (left > 1) {
        const int step = (left + 31) / 32, at = lo + lane * step;
        const bool before = lane == 0 || (at < lo + left && __ldg(p.query_start_loc + at) / kLinearBlock + at <= number);
        const int skip = (31 - __clz(__ballot_sync(kFull, before))) * step;
        lo += skip;
        left = min(step, left - skip);
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
    static constexpr int kGroup = 64;                     // tokens of a stage
    static constexpr int kHalf = kGroup * kTile * 2;      // bytes of a stage's k, and of its v
    static constexpr int kSlots = 3;
    static constexpr int kRing = kSlots * 2 * kHalf;
    // two CTAs an SM, whose TMEM allocations then always fit
    static constexpr int kSmem = (kRing > 78 * 1024 ? kRing : 78 * 1024) + 4 * 1024;
    static constexpr int kTmem = 256;  // the sum, and 64 tokens of v in two halves, twice
    static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two CTAs an SM");
};
constexpr int kAddThreads = 6 * 32;

// A tile of (128 columns of k) x (128 columns of v) of a block's sum.
struct AddUnit {
    int first, count;  // of the block; count 0: no more units
    int number, kvh, tile;
};

// A grid of the CTAs that the SMs hold takes the tiles in turn, a block's tokens 64 at a time, the last ones
// first.  Warp 5 finds the blocks and brings their tokens, running ahead into the next unit;
// lane (thread) c of warps 0-3 is a column of v, whose tokens it scales and writes to tensor
// memory as the MMA's A operand (two halves); warp 4 multiplies by k, the B operand, as TMA
// laid it out.  The column's power of two is set by the first tokens that are not 0 (the
// decay makes earlier ones smaller) with room above, and moves, with the column's sum so far,
// where later ones would not fit.  The first CTAs find the largest entries of the sequences'
// first states.
// 8 x 8192 tokens of 8 x 128: 74.5 us for 402 MB of tokens and sums, 80 % of the measured
// bandwidth (a CTA a tile, without the run ahead: 86 us).  One sequence of 8192 of 4 x 256: 25.5 us,
// 512 tiles for 304 CTAs, where the scaling of a column's 64 tokens (two halves each) bounds it;
// two threads a column take 25.5 too, and 79.5 us for the 8 sequences: their warps wait for each other.
// Looking for keys of 0 costs 2 of 53 us for 16 sequences of up to 4096 of 12 x 64, and less than 1 elsewhere.
template <int D>
__global__ void __launch_bounds__(kAddThreads, 2)
    linear_adds_kernel(const __grid_constant__ LinearMaps maps, const LinearChunkParams c) {
    using S = AddShape<D>;
    const LinearParams& p = c.lin;
    constexpr int kTiles2 = S::kTiles * S::kTiles;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    float* weights = reinterpret_cast<float*>(ring + S::kRing);  // of the tokens, two units
    AddUnit* units = reinterpret_cast<AddUnit*>(weights + 2 * kLinearBlock);
    uint64_t* bars = reinterpret_cast<uint64_t*>(units + 4);  // (two are used: 16-byte multiples)
    uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + 20);
    volatile int* failed = reinterpret_cast<volatile int*>(tslot + 1);
    float* red = reinterpret_cast<float*>(tslot + 2);   // of the warps, two units
    int* bad_sm = reinterpret_cast<int*>(red + 8);      // as many
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31, K = p.num_kv_heads;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");

    auto warp_max = [&](float m) {
#pragma unroll
        for (int d = 16; d; d /= 2) m = fmaxf(m, __shfl_xor_sync(kFull, m, d));
        return m;
    };
    auto finite_max = [](float m, float x) {
        const float a = fabsf(x);
        return a <= 3.402823466e38f ? fmaxf(m, a) : m;
    };
    const int state_ctas = p.num_seqs * K;
    if ((int)blockIdx.x < state_ctas) {
        const int b = blockIdx.x / K, kvh = blockIdx.x % K;
        Seq s;
        unsigned status;
        if (!seq_of(p, b, s, status)) return;
        float m = 0.f;
        if (s.context > 0) {
            const float4* st = reinterpret_cast<const float4*>(p.states + ((size_t)s.slot * K + kvh) * D * D);
#pragma unroll 8
            for (int i = t; i < D * D / 4; i += kAddThreads) {
                const float4 x = st[i];
                m = finite_max(finite_max(finite_max(finite_max(m, x.x), x.y), x.z), x.w);
            }
        }
        m = warp_max(m);
        if (lane == 0) red[warp] = m;
        __syncthreads();
        if (t == 0) {
            for (int i = 1; i < kAddThreads / 32; ++i) m = fmaxf(m, red[i]);
            c.state_max[(size_t)b * K + kvh] = m;
        }
        return;
    }
    // barriers: a stage has landed, has been used; the operand of a group in buffer i is written, has been read;
    // a unit is in its slot, has been taken from it; the column warps meet; they have read the sums
    const uint32_t bar_full = smem_addr(bars), bar_empty = bar_full + 8 * S::kSlots, bar_v = bar_empty + 8 * S::kSlots,
                   bar_mma = bar_v + 16, bar_unit = bar_mma + 16, bar_free = bar_unit + 16, bar_meet = bar_free + 16,
                   bar_read = bar_meet + 8;
    static_assert(2 * S::kSlots + 2 + 2 + 2 + 2 + 1 + 1 <= 20, "barriers");
    if (t == 0) {
        *failed = 0;
        for (int i = 0; i < S::kSlots; ++i) {
            mbar_init(bar_full + 8 * i, 1);
            mbar_init(bar_empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar_v + 8 * i, 4);
            mbar_init(bar_mma + 8 * i, 1);
            mbar_init(bar_unit + 8 * i, 1);
            mbar_init(bar_free + 8 * i, 5);
        }
        mbar_init(bar_meet, 4);
        mbar_init(bar_read, 4);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tslot)), "r"(S::kTmem)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot, t_sum = tmem, t_v = tmem + 128;
    const unsigned limit = c.wait_limit;
    auto fail = [&] {
        *failed = 1;
        atomicOr(p.status, PA_DEV_TIMEOUT);
    };
    // group x of a block holds its tokens from 64 * (groups - 1 - x) on
    auto groups_of = [](int count) { return (count + S::kGroup - 1) / S::kGroup; };

    if (warp == 5) {
        const unsigned total = (unsigned)c.blocks * K * kTiles2, ctas = gridDim.x - state_ctas;
        int n = 0, done = 0, last = -1;  // stages; units; the block looked up last
        bool ok = true, valid = false;
        Block k;
        for (unsigned x = blockIdx.x - state_ctas;; x += ctas) {
            AddUnit u;
            u.count = 0;
            if (x < total) {
                u.tile = x % kTiles2;
                u.kvh = x / kTiles2 % K;
                u.number = x / kTiles2 / K;
                if (u.number != last) valid = block_of(p, u.number, k);
                last = u.number;
                if (lane == 0 && u.kvh == 0 && u.tile == 0)
                    c.block_info[u.number] = valid ? make_int4(k.first, k.count, k.n > 0 || k.context > 0, 0) : make_int4(0, 0, 0, 0);
                if (!valid) continue;
                u.first = k.first;
                u.count = k.count;
            }
            const int s = done & 1;
            if (done >= 2 && !(ok = tc_warp_wait(bar_free + 8 * s, ((done - 2) >> 1) & 1, limit, failed))) break;
            if (lane == 0) {
                units[s] = u;
                mbar_arrive(bar_unit + 8 * s);
            }
            __syncwarp();
            if (u.count == 0) break;
            const int groups = groups_of(u.count), k_tile = u.tile / S::kTiles, v_tile = u.tile % S::kTiles;
#pragma unroll 1
            for (int y = 0; y < groups; ++y, ++n) {
                const int slot = n % S::kSlots;
                if (n >= S::kSlots && !(ok = tc_warp_wait(bar_empty + 8 * slot, (n / S::kSlots - 1) & 1, limit, failed))) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar_full + 8 * slot, 2 * S::kHalf);
                    const uint32_t dst = smem_addr(ring + slot * 2 * S::kHalf);
                    const int at = u.first + (groups - 1 - y) * S::kGroup;
                    tc_tma_load_4d(dst, &maps.k_group, 0, u.kvh, at, k_tile * (S::kTile / 64), bar_full + 8 * slot);
                    tc_tma_load_4d(dst + S::kHalf, &maps.v_group, 0, u.kvh, at, v_tile * (S::kTile / 64), bar_full + 8 * slot);
                }
                __syncwarp();
            }
            if (!ok) break;
            ++done;
        }
        if (lane == 0) {
            if (!ok) fail();
            // every copy lands before the CTA's memory is given back
            for (int i = max(0, n - S::kSlots); i < n; ++i)
                mbar_wait(bar_full + 8 * (i % S::kSlots), (i / S::kSlots) & 1, kDefaultWaitLimit);
        }
        __syncwarp();
    } else if (warp == 4) {
        if (tc_elect()) {
            constexpr uint32_t id = tc_idesc(128, S::kTile, 1);
            bool ok = true;
            int x = 0;  // groups
            for (int done = 0; ok; ++done) {
                const int s = done & 1;
                if (!(ok = tc_wait(bar_unit + 8 * s, (done >> 1) & 1, limit, failed))) break;
                const int count = units[s].count;
                mbar_arrive(bar_free + 8 * s);
                if (count == 0) break;
                const int groups = groups_of(count);
                // the last unit's sums have been read
                if (done > 0 && !(ok = tc_wait(bar_read, (done - 1) & 1, limit, failed))) break;
#pragma unroll 1
                for (int y = 0; y < groups; ++y, ++x) {
                    // (the columns' threads wait for the group's copies before they write the operand)
                    if (!(ok = tc_wait(bar_v + 8 * (x & 1), (x >> 1) & 1, limit, failed))) break;
                    tc_fence_after();
                    const int slot = x % S::kSlots;
                    const uint64_t kd = tc_desc(smem_addr(ring + slot * 2 * S::kHalf), S::kGroup * 128, 1024);
                    const int steps = (min(count - (groups - 1 - y) * S::kGroup, S::kGroup) + 15) / 16;
                    for (int part = 1; part >= 0; --part)  // the small halves first
                        for (int i = 0; i < steps; ++i)
                            tc_mma_ts(t_sum, t_v + (x & 1) * 64 + part * 32 + i * 8, kd + (uint64_t)((i * 2048) >> 4), id,
                                      y > 0 || part == 0 || i > 0);
                    tc_commit(bar_empty + 8 * slot);
                    tc_commit(bar_mma + 8 * (x & 1));
                }
            }
            if (!ok) fail();
            // every MMA is done before the CTA's memory is given back
            if (x > 0) mbar_wait(bar_mma + 8 * ((x - 1) & 1), ((x - 1) >> 1) & 1, kDefaultWaitLimit);
        }
        __syncwarp();
    } else {
        const uint32_t lanes = (uint32_t)(warp * 32) << 16;
        const bool mine = t < S::kTile;
        const int chunk = t >> 6, unit = (t & 63) >> 3, in_unit = t & 7;  // of the column in a row's 64-column chunk
        // (the 128-byte swizzle: 16-byte units exchanged by the row's number)
        auto column = [&](const uint8_t* tile, int i) {
            return __half2float(*reinterpret_cast<const __half*>(tile + i * 128 + ((unit ^ (i & 7)) << 4) + in_unit * 2));
        };
        bool ok = true;
        int x = 0, meets = 0;  // groups; meetings of the columns' warps
        auto meet = [&] {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_meet);
            return ok = tc_warp_wait(bar_meet, meets++ & 1, limit, failed);
        };
        for (int done = 0;; ++done) {
            const int s = done & 1;
            if (!(ok = tc_warp_wait(bar_unit + 8 * s, (done >> 1) & 1, limit, failed))) break;
            const AddUnit u = units[s];
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_free + 8 * s);
            if (u.count == 0) break;
            const int groups = groups_of(u.count), k_tile = u.tile / S::kTiles, v_tile = u.tile % S::kTiles;
            float* w = weights + s * kLinearBlock;
            const float g = fmaxf(__ldg(p.log_decay + u.kvh), -1e4f);  // (whose exp is 0, and 1 for no tokens)
            for (int i = t; i < kLinearBlock; i += 128) w[i] = i < u.count ? expf(g * (float)(u.count - 1 - i)) : 0.f;
            if (t == 0) bad_sm[s] = 0;
            if (!meet()) break;  // (who writes these again has met the others, done with this unit, once more)
            int up = 0, first = kLinearBlock;
            bool set = false;
#pragma unroll 1
            for (int y = 0; y < groups; ++y, ++x) {
                const int at = (groups - 1 - y) * S::kGroup, count = min(u.count - at, S::kGroup);
                uint8_t* ks = ring + (x % S::kSlots) * 2 * S::kHalf;
                const uint8_t* vs = ks + S::kHalf + chunk * (S::kGroup * 128);
                if (!(ok = tc_warp_wait(bar_full + 8 * (x % S::kSlots), (x / S::kSlots) & 1, limit, failed))) break;
                // rows of other sequences behind the block's last token: nothing of them, whatever they hold
                const int tail = (count + 15) / 16 * 16 - count;
                for (int i = t; i < tail * (S::kTile / 8); i += 128) {
                    const int r = count + i / (S::kTile / 8), q = i % (S::kTile / 8);
                    *reinterpret_cast<uint4*>(ks + (q >> 3) * (S::kGroup * 128) + r * 128 + (q & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                }
                if (tail) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                // Tokens whose keys (of this tile) are all 0 add nothing and have no say in the power of two: masked
                // ones may follow others that the decay has made smaller than their v's last bit.  A lane looks at two
                // tokens, 16 bytes of each where these are not 0.
                auto key = [&](int r, int q) {
                    const uint4 z = *reinterpret_cast<const uint4*>(ks + (q >> 3) * (S::kGroup * 128) + r * 128 +
                                                                    (((q & 7) ^ (r & 7)) << 4));
                    return ((z.x | z.y | z.z | z.w) & 0x7fff7fffu) != 0;
                };
                bool some[2] = {lane >= count || key(lane, 0), lane + 32 >= count || key(lane + 32, 0)};
                float a[64];
                float m = 0.f;
                bool bad = false;
#pragma unroll
                for (int i = 0; i < 64; i += 2) {
#pragma unroll
                    for (int j = i; j < i + 2; ++j) {
                        const float v = mine && j < count ? column(vs, j) : 0.f;
                        bad |= !(fabsf(v) <= 65504.f);
                        a[j] = v * w[at + j];
                    }
                    m = max3(m, __float_as_uint(a[i]), __float_as_uint(a[i + 1]));
                }
                if (!__all_sync(kFull, some[0] && some[1])) {
                    m = 0.f;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
#pragma unroll 1
                        for (int q = 1; q < S::kTile / 8 && !some[h]; ++q) some[h] = key(h * 32 + lane, q);
                        const unsigned live = __ballot_sync(kFull, some[h]);
#pragma unroll
                        for (int i = h * 32; i < h * 32 + 32; ++i) {
                            // (0 times a NaN or an infinity stays NaN)
                            if (!(live >> (i & 31) & 1u) && fabsf(a[i]) <= 65504.f) a[i] = 0.f;
                            m = fmaxf(m, fabsf(a[i]));
                        }
                    }
                }
                if (bad) {  // the power of two is that of the others
                    m = 0.f;
#pragma unroll
                    for (int i = 63; i >= 0; --i) {
                        const bool there = mine && i < count;
                        if (there && !(fabsf(column(vs, i)) <= 65504.f))
                            first = at + i;
                        else
                            m = fmaxf(m, fabsf(a[i]));
                    }
                }
                const int e = exponent_of(m);
                const bool move = m > 0.f && (!set || e + up > 14);
                const int was = up;
                if (move) up = min(8 - e, 118);  // (moves down by 125 at most, from there to 65504)
                if (x >= 2) {  // the operand's buffer has been read
                    if (!(ok = tc_warp_wait(bar_mma + 8 * (x & 1), ((x - 2) >> 1) & 1, limit, failed))) break;
                    tc_fence_after();
                }
                if (y > 0 && __any_sync(kFull, move && set)) {
                    if (!(ok = tc_warp_wait(bar_mma + 8 * ((x - 1) & 1), ((x - 1) >> 1) & 1, limit, failed))) break;
                    tc_fence_after();
                    const float f = move && set ? pow2(up - was) : 1.f;
#pragma unroll 1
                    for (int c0 = 0; c0 < S::kTile; c0 += 32) {
                        uint32_t o[32];
                        tc_ld32(t_sum + lanes + c0, o);
#pragma unroll
                        for (int q = 0; q < 32; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * f);
                        tc_st32(t_sum + lanes + c0, o);
                    }
                }
                set |= move;
                const float raise = pow2(up);
                uint32_t hi[32], lo[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const float y0 = a[2 * i] * raise, y1 = a[2 * i + 1] * raise;
                    const __half2 h = __floats2half2_rn(y0, y1);
                    const float2 back = __half22float2(h);
                    hi[i] = half2_bits(h);
                    lo[i] = half2_bits(__floats2half2_rn(y0 - back.x, y1 - back.y));
                }
                tc_st32x2(t_v + lanes + (x & 1) * 64, hi, t_v + lanes + (x & 1) * 64 + 32, lo);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_v + 8 * (x & 1));
            }
            if (!ok) break;
            const size_t index = (size_t)u.number * K + u.kvh;
            if (k_tile == 0 && mine) {
                c.first_bad[index * D + v_tile * S::kTile + t] = first;
                if (first < kLinearBlock) bad_sm[s] = 1;
            }
            if (!(ok = tc_warp_wait(bar_mma + 8 * ((x - 1) & 1), ((x - 1) >> 1) & 1, limit, failed))) break;
            tc_fence_after();
            float m = 0.f;
            const float lower = pow2(-up);
            float* dst = c.adds + (index * D + k_tile * S::kTile) * D + v_tile * S::kTile + t;
#pragma unroll 1
            for (int c0 = 0; c0 < S::kTile; c0 += 32) {
                uint32_t o[32];
                tc_ld32(t_sum + lanes + c0, o);
                if (mine) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const float z = __uint_as_float(o[i]) * lower;
                        m = finite_max(m, z);
                        dst[(size_t)(c0 + i) * D] = z;
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_read);
            m = warp_max(m);
            if (lane == 0) red[s * 4 + warp] = m;
            if (!meet()) break;
            if (t == 0) {
                const float* r = red + s * 4;
                c.add_max[index * kTiles2 + u.tile] = fmaxf(fmaxf(r[0], r[1]), fmaxf(r[2], r[3]));
                if (k_tile == 0) c.any_bad[index * S::kTiles + v_tile] = bad_sm[s];
            }
        }
        if (!ok && lane == 0) fail();
    }
    tc_fence_before();
    __syncthreads();  // no copy or MMA is in flight
    if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::kTmem));
}

// ---- the chain of states

constexpr int kScanThreads = 256;

// A thread takes four entries of a (sequence, kv head)'s state through its blocks.
// The state before each block goes to the outputs' kernel as halves of S 2^-e; e comes
// from a bound on |S| that runs along (no more than a few bits above it), so that no
// block has to look for the largest entry.  Bound by memory, 6 D^2 bytes a block and kv head:
// 8 x 8192 tokens of 8 x 128 (201 MB) 36 us, 82 % of the measured bandwidth (with 70 registers,
// three blocks an SM, 41); where one sequence has all blocks, by the trips along it (8192 of
// 4 x 256, 50 MB: 19.4 us).
template <int D>
__global__ void __launch_bounds__(kScanThreads, 4) linear_scan_kernel(const LinearChunkParams c) {
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
    Decay d = decay_of(fmaxf(g, -1e4f) * (float)kLinearBlock);  // d^L
    // four blocks ahead: what a round of the loop waits for has long been asked for (eight: 8 prompts of 8192 tokens of
    // 8 x 128 43 -> 55 us, one of 4 x 256 20 either way)
    constexpr int kAhead = 4;
    float4 next[kAhead];
    float most_next[kAhead];
    auto fetch = [&](int n, float4& a, float& most) {
        if (n >= blocks) return;
        a = __ldcs(add + n * step / 4);
        most = 0.f;
#pragma unroll
        for (int j = 0; j < kTiles; ++j) most = fmaxf(most, __ldg(c.add_max + (index + (size_t)n * p.num_kv_heads) * kTiles + j));
    };
#pragma unroll
    for (int n = 0; n < kAhead; ++n) fetch(n, next[n], most_next[n]);
    auto one = [&](int n, float4& slot, float& most_slot) {
        const float4 a = slot;
        const float most = most_slot;
        fetch(n + kAhead, slot, most_slot);
        const size_t i = index + (size_t)n * p.num_kv_heads;
        if (n > 0 || s.context > 0) {
            const int e = bound > 0.f ? max(min(exponent_of(bound) - 8, 119), -100) : 0;
            const float down = pow2(-e);
            uint2 h;
            h.x = half2_bits(__floats2half2_rn(x.x * down, x.y * down));
            h.y = half2_bits(__floats2half2_rn(x.z * down, x.w * down));
            *reinterpret_cast<uint2*>(c.starts + i * D * D + at) = h;
            if (first) c.exponents[i] = e;
        }
        if (n == blocks - 1) d = decay_of(fmaxf(g, -1e4f) * (float)(s.count - n * kLinearBlock));
        auto chain = [&](float v, float plus) { return fmaf(v, d.whole, v * d.rest) + plus; };
        x = make_float4(chain(x.x, a.x), chain(x.y, a.y), chain(x.z, a.z), chain(x.w, a.w));
        bound = (bound * (d.whole + d.rest) + most) * 1.0001f;
    };
    for (int n = 0; n < blocks; n += kAhead) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (n + j < blocks) one(n + j, next[j], most_next[j]);
    }
    *state = x;
}

// ---- the outputs

template <int D>
struct OutShape {
    // two CTAs an SM up to head_dim 128; at 256 the accumulator takes half of the tensor memory
    static constexpr int kCtas = D == 256 ? 1 : 2;
    static constexpr int kSides = D == 256 ? 4 : 2;       // threads of a row
    static constexpr int kRowWarps = 4 * kSides;
    static constexpr int kThreads = (kRowWarps + 2) * 32;
    static constexpr int kStageRows = D == 256 ? 64 : 128;  // keys or state rows of a ring slot, 16 or 32 KB
    static constexpr int kStateRows = D < kStageRows ? D : kStageRows;
    static constexpr int kStepStages = 128 / kStageRows;
    static constexpr int kQBytes = 128 * D * 2;
    static constexpr int kStageBytes = kStageRows * D * 2;
    static constexpr int kSlots = D == 256 ? 5 : D == 128 ? 2 : 4;
    static constexpr int kScores = D == 256 ? 2 : 1;  // steps whose scores or P are in tensor memory
    static constexpr int kBars = 22 + 2 * kSlots;
    // barriers, TMEM address and flag, two units, the exponents of the rows' largest scores by threads
    static constexpr int kCtrl = kBars * 8 + 16 + 2 * 64 + 2 * kSides * 128;
    static constexpr int kSmemNeed = kQBytes + kSlots * kStageBytes + kCtrl;
    // (so much that no more CTAs fit, and their TMEM allocations always do)
    static constexpr int kSmem = kSmemNeed > 80 * 1024 ? kSmemNeed : 80 * 1024;
    static constexpr int kTmem = D == 256 ? 512 : 256;    // D of the outputs, 128 for each step's scores
    static_assert(kCtas * (kSmem + 1024) <= 228 * 1024, "CTAs an SM");
    static_assert(D + 128 * kScores <= kTmem && kCtas * kTmem <= 512, "tensor memory of an SM");
};

// 128 tokens (a half of a block) of one query head.
struct OutUnit {
    int first, count;  // of the block; count 0: no more units
    int index;         // of the block and kv head
    int half, kvh, head;
    int inter;         // whether there is a state before the block
    int dirty;         // whether a column of v has a NaN or infinity
    int exponent;      // of that state
    float l2;          // log2 of the decay
};

// mbarriers of a CTA
enum : int {
    kBarQ = 0,                 // Q has landed
    kBarQFree,                 // and its MMAs are done
    kBarInter,                 // the accumulator holds Q S
    kBarRead,                  // the rows have read the accumulator
    kBarScores,                // a step's scores are there, 2 (in turn, where the next step's may come before they
                               // are used)
    kBarP = kBarScores + 2,    // P over them, 2 (a warp may be a step ahead of another)
    kBarPV = kBarP + 2,        // P V is done, 2 (so may the products be)
    kBarUnit = kBarPV + 2,     // a unit's slot is written, 2
    kBarUnitFree = kBarUnit + 2,  // and read by the MMAs' warp and the rows', 2
    kBarDrain = kBarUnitFree + 2,
    kBarV,                        // V tiles that the rows clean have landed
    kBarSwap,                     // the threads of a quarter of the rows meet, 4
    kBarOut = kBarSwap + 4,       // a unit's outputs are in its last V stages, 2 (in turn: the unit after the next
                                  // starts when this one's have gone)
    kBarFull = kBarOut + 2
};

// A grid of the CTAs that the SMs hold takes the units in turn, the two halves of a block
// (one and two steps of 128 keys) neighbours in that order.  A unit's 128 rows are the
// lanes of the accumulator.  The last warp finds the units and brings Q, then in ring stages a
// step's keys, the state's rows (behind the first step's keys; at head_dim 256 the second step's
// follow them) and the step's values, in the
// order in which the warp before it feeds them to the tensor cores: a step's scores; Q S_n;
// P V.  Both run ahead into the next unit while the row warps, two or four threads a
// row, turn a step's scores into P, in fp16 over the scores, keep the accumulator in the
// row's power of two, and write the outputs.  Steps go from the row's own keys backwards,
// where scores only shrink by the decay, so that the first one nearly always sets that
// power.  What bounds it is the chain of hand-overs between the roles, each of which takes
// longer than its products: hence steps of 128 keys, whole steps a stage where they fit (stages of
// 64 keys at head_dim 128: the call on 8 x 8192 of 32/8 463 -> 520 us), and one elected thread for
// the copies and one for the MMAs (in a branch of `lane == 0` the compiler does not know that it
// is one).  At head_dim 256, where tensor memory has room for them, a unit's second scores are
// multiplied while the rows work on the first (without: 81 us where it takes 76 below).
// 8 x 8192 tokens of 32/8 x 128: 312 us for 1.41 GB, 66 % of the measured bandwidth, and 880
// TFLOP/s of its tiles' products, 46 % of the measured rate; the hand-overs alone, without the row
// warps' arithmetic, take half of that.  One sequence of 8192 of 24/4 x 256: 76 us (one CTA an SM,
// whose hand-overs nothing else covers), and 5 to 27 us more with outputs stored by the row warps.
template <int D>
__global__ void __launch_bounds__(OutShape<D>::kThreads, OutShape<D>::kCtas)
    linear_out_kernel(const __grid_constant__ LinearMaps maps, const LinearChunkParams c) {
    using S = OutShape<D>;
    const LinearParams& p = c.lin;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* qs = smem;
    uint8_t* ring = qs + S::kQBytes;
    uint64_t* bars = reinterpret_cast<uint64_t*>(ring + S::kSlots * S::kStageBytes);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + S::kBars);
    volatile int* failed = reinterpret_cast<volatile int*>(tslot + 1);
    OutUnit* units = reinterpret_cast<OutUnit*>(tslot + 4);
    static_assert(sizeof(OutUnit) <= 64, "unit slots");
    uint8_t* largest = reinterpret_cast<uint8_t*>(tslot + 4 + 2 * 16);
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int G = p.group, H = p.num_heads, K = p.num_kv_heads;
    if (smem_addr(smem) & 1023u) {  // (the layouts need it; dynamic shared memory starts there)
        if (t == 0) atomicOr(p.status, PA_DEV_TIMEOUT);
        return;
    }
    const uint32_t bar0 = smem_addr(bars);
    auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
    constexpr int kBarEmpty = kBarFull + S::kSlots;
    if (t == 0) {
        *failed = 0;
        for (int i = 0; i < S::kBars; ++i)
            mbar_init(bar(i), i == kBarP || i == kBarP + 1 || i == kBarRead || i == kBarOut || i == kBarOut + 1 ? S::kRowWarps
                              : i >= kBarSwap && i < kBarOut               ? S::kSides
                              : i == kBarUnitFree || i == kBarUnitFree + 1 ? S::kRowWarps + 1
                                                                           : 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tslot)), "r"(S::kTmem)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot, t_out = tmem, t_s = tmem + D;
    const unsigned limit = c.wait_limit;
    auto fail = [&] {
        *failed = 1;
        atomicOr(p.status, PA_DEV_TIMEOUT);
    };
    // A unit's steps are of 128 keys, the last ones first: half + 1 of them.  Whether the rows change a
    // step's V before it is multiplied (see there):
    auto cleaned = [](bool dirty, int count, int half, int j) { return dirty || (j == 0 && count < half * 128 + 128); };
    constexpr int kStateStages = D / S::kStateRows;

    if (warp == S::kRowWarps + 1) {
        int n = 0, slot = 0, turn = 0;  // stages; the next one's slot of the ring and its phase
        bool ok = true;
        int done = 0, q_tiles = 0;  // units; Q tiles
        if (tc_elect()) {
            // The CTA's units are every gridDim.x-th, counted by the halves, the heads of a group, the kv heads and
            // the blocks, each with a carry (divisions took this thread longer than its copies).
            auto digits = [&](unsigned x, int& half, int& h, int& kvh, int& number) {
                half = x % 2;
                x /= 2;
                h = x % G;
                x /= G;
                kvh = x % K;
                number = x / K;
            };
            int half, h, kvh, number, d_half, d_h, d_kvh, d_number;
            digits(blockIdx.x, half, h, kvh, number);
            digits(gridDim.x, d_half, d_h, d_kvh, d_number);
            // What a unit takes from memory is asked for a unit ahead of when it is needed.
            int4 info;
            int dirty, exponent;
            float decay;
            auto ask = [&] {
                if (number >= c.blocks) return;
                const size_t y = (size_t)number * K + kvh;
                info = __ldg(c.block_info + number);
                dirty = __ldg(c.any_bad + y * AddShape<D>::kTiles);
                if (AddShape<D>::kTiles == 2) dirty |= __ldg(c.any_bad + y * 2 + 1);
                exponent = __ldg(c.exponents + y);
                decay = __ldg(p.log_decay + kvh);
            };
            auto advance = [&] {
                half += d_half;
                h += d_h + (half >> 1);
                half &= 1;
                const int c1 = h >= G;
                h -= c1 ? G : 0;
                kvh += d_kvh + c1;
                const int c2 = kvh >= K;
                kvh -= c2 ? K : 0;
                number += d_number + c2;
            };
            ask();
            // The last unit's outputs lie in its last V stages (from owed_stage on) until they are copied
            // out; its stages are then free.
            bool owed = false, owed_whole = false;
            int owed_stage = 0, owed_head = 0, owed_row = 0, settled = 0;
            auto settle = [&] {
                owed = false;
                if (!tc_wait(bar(kBarOut + (settled & 1)), (settled >> 1) & 1, limit, failed)) return false;
                ++settled;
#pragma unroll
                for (int y = 0; y < S::kStepStages; ++y) {
                    const int from = (owed_stage + y) % S::kSlots;
                    if (owed_whole)
                        asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(&maps.out),
                                     "r"(0), "r"(owed_head), "r"(owed_row + y * S::kStageRows), "r"(0),
                                     "r"(smem_addr(ring) + from * S::kStageBytes)
                                     : "memory");
                }
                asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group.read 0;" ::: "memory");
#pragma unroll
                for (int y = 0; y < S::kStepStages; ++y) mbar_arrive(bar(kBarEmpty + (owed_stage + y) % S::kSlots));
                return true;
            };
            for (;;) {
                while (number < c.blocks && half * 128 >= info.y) {  // no such half of a block
                    advance();
                    ask();
                }
                OutUnit u;
                u.count = 0;
                if (number < c.blocks) {
                    u.first = info.x;
                    u.count = info.y;
                    u.index = number * K + kvh;
                    u.half = half;
                    u.kvh = kvh;
                    u.head = kvh * G + h;
                    u.inter = info.z;
                    u.dirty = dirty;
                    u.exponent = exponent;
                    u.l2 = fmaxf(decay * kLog2e, -1e6f);
                    advance();
                    ask();
                }
                const int s = done & 1;
                if (done >= 2 && !(ok = tc_wait(bar(kBarUnitFree + s), ((done - 2) >> 1) & 1, limit, failed))) break;
                units[s] = u;
                mbar_arrive(bar(kBarUnit + s));
                if (u.count == 0) break;
                auto stage = [&](const CUtensorMap* map, int y, int z, int bytes) {
                    if (!ok) return;
                    if (n >= S::kSlots) {
                        if (owed && n - S::kSlots == owed_stage && !(ok = settle())) return;
                        if (!(ok = tc_wait(bar(kBarEmpty + slot), turn ^ 1, limit, failed))) return;
                    }
                    const uint32_t full = bar(kBarFull + slot);
                    mbar_arrive_expect_tx(full, bytes);
                    tc_tma_load_4d(smem_addr(ring) + slot * S::kStageBytes, map, 0, y, z, 0, full);
                    ++n;
                    if (++slot == S::kSlots) {
                        slot = 0;
                        turn ^= 1;
                    }
                };
                auto step = [&](const CUtensorMap* map, int j) {
#pragma unroll
                    for (int y = 0; y < S::kStepStages; ++y)
                        stage(map, u.kvh, u.first + (u.half - j) * 128 + y * S::kStageRows, S::kStageBytes);
                };
                if (done >= 1 && !(ok = tc_wait(bar(kBarQFree), (done - 1) & 1, limit, failed))) break;
                mbar_arrive_expect_tx(bar(kBarQ), S::kQBytes);
                tc_tma_load_4d(smem_addr(qs), &maps.q, 0, u.head, u.first + u.half * 128, 0, bar(kBarQ));
                ++q_tiles;
#pragma unroll 1
                for (int j = 0; j <= u.half; ++j) {
                    if (S::kScores == 1 || j == 0) step(&maps.k, j);
                    if (j == 0 && u.inter)
#pragma unroll
                        for (int d = 0; d < kStateStages; ++d)
                            stage(&maps.starts, 0, u.index * D + d * S::kStateRows, S::kStateRows * D * 2);
                    if (S::kScores == 2 && j < u.half) step(&maps.k, j + 1);
                    step(&maps.v, j);
                }
                // (a unit may have fewer stages than the ring has slots)
                if (!ok || (owed && !(ok = settle()))) break;
                owed = true;
                owed_stage = n - S::kStepStages;
                owed_whole = u.half * 128 + 128 <= u.count;
                owed_head = u.head;
                owed_row = u.first + u.half * 128;
                ++done;
            }
            if (ok && owed) ok = settle();
            if (!ok) fail();
            // every copy lands before the CTA's memory is given back
            if (q_tiles > 0) mbar_wait(bar(kBarQ), (q_tiles - 1) & 1, kDefaultWaitLimit);
            for (int i = max(0, n - S::kSlots); i < n; ++i)
                mbar_wait(bar(kBarFull + i % S::kSlots), (i / S::kSlots) & 1, kDefaultWaitLimit);
        }
        __syncwarp();
    } else if (warp == S::kRowWarps) {
        if (tc_elect()) {
            constexpr uint32_t id_s = tc_idesc(128, S::kStageRows, 0), id_o = tc_idesc(128, D, 1);
            const uint64_t qdesc = tc_desc(smem_addr(qs), 16, 1024), kdesc = tc_desc(smem_addr(ring), 16, 1024);
            // columns of V and of the state 64 at a time, one 64-column chunk behind the other
            const uint64_t vdesc = tc_desc(smem_addr(ring), S::kStageRows * 128, 1024);
            const uint64_t sdesc = tc_desc(smem_addr(ring), S::kStateRows * 128, 1024);
            int slot = 0, turn = 0;  // of the ring: the next stage's slot, and its phase
            int x = 0, inters = 0;   // steps, units with a state
            bool ok = true;
            auto wait = [&](int b, int parity) { return ok = ok && tc_wait(bar(b), parity & 1, limit, failed); };
            auto landed = [&] { return wait(kBarFull + slot, turn); };
            auto at = [&] { return (uint64_t)(slot * (S::kStageBytes >> 4)); };
            auto next = [&] {
                if (++slot == S::kSlots) {
                    slot = 0;
                    turn ^= 1;
                }
            };
            auto release = [&] {
                tc_commit(bar(kBarEmpty + slot));
                next();
            };
            for (int done = 0;; ++done) {
                const int s = done & 1;
                if (!wait(kBarUnit + s, done >> 1)) break;
                const int count = units[s].count, half = units[s].half;
                const bool inter = units[s].inter, dirty = units[s].dirty;
                mbar_arrive(bar(kBarUnitFree + s));
                if (count == 0) break;
                if (!wait(kBarQ, done)) break;
                // The scores of step x + ahead, over the P of kScores steps before, whose P V was the last one issued
                // or came before that one.
                auto scores = [&](int ahead) {
                    const int z = x + ahead, buffer = z % S::kScores;
                    if (x > 0 && !wait(kBarPV + (x - 1) % S::kScores, (x - 1) / S::kScores)) return false;
#pragma unroll
                    for (int y = 0; y < S::kStepStages; ++y) {
                        if (!landed()) return false;
                        tc_fence_after();
                        const uint64_t kd = kdesc + at();
#pragma unroll
                        for (int i = 0; i < D / 16; ++i)
                            tc_mma_ss(t_s + buffer * 128 + y * S::kStageRows,
                                      qdesc + (uint64_t)(((i >> 2) * (128 * 128) + (i & 3) * 32) >> 4),
                                      kd + (uint64_t)(((i >> 2) * (S::kStageRows * 128) + (i & 3) * 32) >> 4), id_s, i > 0);
                        release();
                    }
                    tc_commit(bar(kBarScores + buffer));
                    return true;
                };
#pragma unroll 1
                for (int j = 0; j <= half; ++j, ++x) {
                    if ((S::kScores == 1 || j == 0) && !scores(0)) break;
                    if (j == 0 && inter) {
                        // the accumulator's last outputs have been read
                        if (done >= 1 && !wait(kBarRead, done - 1)) break;
#pragma unroll 1
                        for (int d = 0; d < kStateStages && landed(); ++d) {
                            tc_fence_after();
                            const uint64_t sd = sdesc + at();
                            const uint64_t qd = qdesc + (uint64_t)((d * (S::kStateRows / 64) * (128 * 128)) >> 4);
#pragma unroll
                            for (int i = 0; i < S::kStateRows / 16; ++i)
                                tc_mma_ss(t_out, qd + (uint64_t)(((i >> 2) * (128 * 128) + (i & 3) * 32) >> 4),
                                          sd + (uint64_t)((i * 2048) >> 4), id_o, d > 0 || i > 0);
                            release();
                        }
                        if (!ok) break;
                        tc_commit(bar(kBarInter));
                        ++inters;
                    }
                    if (S::kScores == 2 && j < half && !scores(1)) break;  // while the rows make P
                    if (j == (S::kScores == 2 ? 0 : half)) tc_commit(bar(kBarQFree));
                    // (the rows cannot tell a ring slot's phases apart: they may be two behind)
                    if (cleaned(dirty, count, half, j)) {
                        if (!landed()) break;
                        if (S::kStepStages == 2) {
                            const bool wraps = slot + 1 == S::kSlots;
                            if (!wait(kBarFull + (wraps ? 0 : slot + 1), turn ^ (int)wraps)) break;
                        }
                        mbar_arrive(bar(kBarV));
                    }
                    // (rows that have written P have read the last outputs too)
                    if (!wait(kBarP + x % S::kScores, x / S::kScores)) break;
                    // Q S, whose operand comes from shared memory, is done before P V, whose comes from
                    // tensor memory, adds to it: nothing orders the two kinds in the tensor cores
                    if (j == 0 && inter && !wait(kBarInter, inters - 1)) break;
                    const uint32_t add = inter || j > 0;
#pragma unroll
                    for (int y = 0; y < S::kStepStages; ++y) {
                        if (!landed()) break;
                        tc_fence_after();
                        const uint64_t vd = vdesc + at();
#pragma unroll
                        for (int i = 0; i < S::kStageRows / 16; ++i) {
                            // each of a row's threads has its P over its own 128 / kSides scores
                            constexpr int kPer = 8 / S::kSides;
                            const int k = y * (S::kStageRows / 16) + i;
                            tc_mma_ts(t_out, t_s + x % S::kScores * 128 + k / kPer * (128 / S::kSides) + k % kPer * 8,
                                      vd + (uint64_t)((i * 2048) >> 4), id_o,
                                      k > 0 ? 1u : add);
                        }
                        // (the unit's last V goes to the rows, who put the outputs there)
                        if (j < half) tc_commit(bar(kBarEmpty + slot));
                        next();
                    }
                    if (!ok) break;
                    tc_commit(bar(kBarPV + x % S::kScores));
                }
                if (!ok) break;
            }
            if (!ok) fail();
            tc_commit(bar(kBarDrain));
            mbar_wait(bar(kBarDrain), 0, kDefaultWaitLimit);
        }
        __syncwarp();
    } else {
        // Warps w, w + 4, ... have the same 32 rows (tensor memory gives a warp those of its number
        // modulo 4), each a share of a step's keys and of the outputs' columns.
        const int quarter = warp & 3, side = warp >> 2;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        constexpr int kMine = D / S::kSides, kKeys = 128 / S::kSides;
        const uint32_t acc = t_out + lanes + side * kMine, scores0 = t_s + lanes + side * kKeys;
        bool ok = true;
        int x = 0, inters = 0;  // steps; units with a state
        int stages = 0;         // ring stages of earlier steps
        int cleans = 0;         // steps whose V was cleaned
        int swaps = 0;          // meetings of the quarter's warps
        // (by an mbarrier, whose waits are bounded: a warp that gave up elsewhere would leave others at a hardware
        // barrier for good)
        auto meet = [&] {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kBarSwap + quarter));
            return ok = tc_warp_wait(bar(kBarSwap + quarter), swaps++ & 1, limit, failed);
        };
        auto product = [&](int step) {  // a step's P V is done
            return tc_warp_wait(bar(kBarPV + step % S::kScores), step / S::kScores & 1, limit, failed);
        };
        for (int done = 0;; ++done) {
            const int s = done & 1;
            if (!(ok = tc_warp_wait(bar(kBarUnit + s), (done >> 1) & 1, limit, failed))) break;
            const OutUnit u = units[s];
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kBarUnitFree + s));
            if (u.count == 0) break;
            const int row0 = u.half * 128 + quarter * 32, i = row0 + lane;  // the warp's first token in the block; the row's
            // The accumulator holds the outputs times 2^-level.  It starts out with Q S, whose row is so
            // many times the state's part as `state` says; where that number is moderate the scores
            // simply go by it, and the accumulator is not touched.
            const float state = u.inter ? (float)u.exponent + u.l2 * (float)(i + 1) : 0.f;
            float level = u.inter ? fminf(fmaxf(state, -6.f), 60.f) : 0.f;
            // The level stays where nothing overflows: the state's part (from state - 60 on), and 2^-level itself, the
            // factor of keys next to the row, whose scores may be 0 (and of an accumulator that holds nothing yet).  At
            // -119 the smallest largest score, 2^-126, is still a normal number of fp16, 2^-7.
            const float least = u.inter ? fmaxf(state - 60.f, -119.f) : -119.f;
            float pending = u.inter ? state - level : 0.f;        // by how much the accumulator is behind
            bool set = false;
            float within[8];  // decays inside a group of 8 keys
#pragma unroll
            for (int v = 0; v < 8; ++v) within[v] = tc_ex2(u.l2 * (float)(7 - v));
#pragma unroll 1
            for (int j = 0; j <= u.half; ++j, ++x) {
                const int kc = (u.half - j) * 128 + side * kKeys;  // first key of the warp's share of the step
                const uint32_t own = scores0 + x % S::kScores * 128;
                if (!(ok = tc_warp_wait(bar(kBarScores + x % S::kScores), x / S::kScores & 1, limit, failed))) break;
                tc_fence_after();
                uint32_t pk[kKeys / 2];
                // A second time where a row's level has to move: 64 scores a thread kept beside their P would not
                // fit in its registers.
#pragma unroll 1
                for (bool again = false;;) {
                    float m = 0.f;
#pragma unroll
                    for (int h = 0; h < kKeys / 32; ++h) {
                        const int k0 = kc + h * 32;
                        uint32_t sc[32];
                        if (k0 > row0) {  // keys behind all of the rows
#pragma unroll
                            for (int v = 0; v < 16; ++v) pk[h * 16 + v] = 0u;
                            continue;
                        }
                        tc_ld32(own + h * 32, sc);
                        // times d^(i - key) 2^-level
                        if (k0 < row0) {
                            // for groups of 8 keys up to the last of them, and the one within
#pragma unroll
                            for (int v = 0; v < 32; v += 8) {
                                const float to = tc_ex2(fmaf(u.l2, (float)(i - k0 - v - 7), -level));
#pragma unroll
                                for (int y = 0; y < 8; y += 2) {
                                    uint32_t d0 = __float_as_uint(within[y]), d1 = __float_as_uint(within[y + 1]);
                                    mul2(d0, d1, to, to);
                                    mul2(sc[v + y], sc[v + y + 1], __uint_as_float(d0), __uint_as_float(d1));
                                }
                            }
                        } else {  // the diagonal
#pragma unroll
                            for (int v = 0; v < 32; ++v)
                                sc[v] = lane >= v ? __float_as_uint(__uint_as_float(sc[v]) *
                                                                    tc_ex2(fmaf(u.l2, (float)(lane - v), -level)))
                                                  : 0u;
                        }
#pragma unroll
                        for (int v = 0; v < 32; v += 2) {
                            m = max3(m, sc[v], sc[v + 1]);
                            pk[h * 16 + v / 2] = half2_bits(__floats2half2_rn(__uint_as_float(sc[v]), __uint_as_float(sc[v + 1])));
                        }
                    }
                    if (again) break;
                    // the exponent of the row's largest, of all its threads (what is not a normal number counts as 0)
                    uint8_t* row = largest + (x & 1) * (S::kSides * 128) + quarter * 32 + lane;
                    int e = exponent_of(m) + 127;
                    row[side * 128] = (uint8_t)e;
                    if (!meet()) break;
#pragma unroll
                    for (int y = 0; y < S::kSides; ++y) e = max(e, (int)row[y * 128]);
                    e -= 127;
                    // The level moves where the row's first scores that are not 0 are not of a middling size, and
                    // where later ones would leave fp16.
                    const bool move = e > -127 && (e >= 15 || (!set && e < -4));
                    set |= e > -127;
                    if (!__any_sync(kFull, move)) break;
                    const float by = move ? fmaxf((float)(e - 8), least - level) : 0.f;
                    level += by;
                    pending -= by;
                    again = true;
                }
                if (!ok) break;
                // over the thread's own scores
                if constexpr (kKeys == 64)
                    tc_st32(own, pk);
                else
                    tc_st16(own, pk);
                if (__any_sync(kFull, pending != 0.f)) {
                    // (the accumulator holds nothing before a first step without a state)
                    if (j == 0 && u.inter) {
                        ok = tc_warp_wait(bar(kBarInter), inters & 1, limit, failed);
                    } else if (j > 0) {
                        ok = product(x - 1);
                    }
                    if (!ok) break;
                    if (j > 0 || u.inter) {
                        tc_fence_after();
                        const float f = exp2f(pending);
#pragma unroll 1
                        for (int c0 = 0; c0 < kMine; c0 += 32) {
                            uint32_t o[32];
                            tc_ld32(acc + c0, o);
#pragma unroll
                            for (int v = 0; v < 32; v += 2) mul2(o[v], o[v + 1], f, f);
                            tc_st32(acc + c0, o);
                        }
                    }
                    pending = 0.f;
                }
                // (behind the step's keys and, where they come early, the next one's)
                const int v_stage = stages + (S::kScores == 1 ? 1 : j > 0 ? 0 : u.half + 1) * S::kStepStages +
                                    (j == 0 && u.inter ? kStateStages : 0);
                if (cleaned(u.dirty, u.count, u.half, j)) {
                    // V rows behind the block's last token belong to other sequences, and a NaN or
                    // infinity must not meet the zeros of tokens before it: both become 0 (the latter's column
                    // is set from its token on in the end)
                    if (!(ok = tc_warp_wait(bar(kBarV), cleans & 1, limit, failed))) break;
                    ++cleans;
#pragma unroll 1
                    for (int y = 0; y < S::kStepStages; ++y) {
                        uint8_t* vt = ring + ((v_stage + y) % S::kSlots) * S::kStageBytes;
                        const int k0 = (u.half - j) * 128 + y * S::kStageRows;
                        for (int v = t; v < S::kStageBytes / 16; v += S::kRowWarps * 32) {
                            const int row = (v >> 3) % S::kStageRows;
                            uint4* cell = reinterpret_cast<uint4*>(vt + (size_t)v * 16);
                            const uint4 z = *cell;
                            auto clean = [](uint32_t h) {
                                if ((h & 0x7c00u) == 0x7c00u) h &= 0xffff0000u;
                                if ((h & 0x7c000000u) == 0x7c000000u) h &= 0xffffu;
                                return h;
                            };
                            *cell = k0 + row < u.count ? make_uint4(clean(z.x), clean(z.y), clean(z.z), clean(z.w))
                                                       : make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
                stages = v_stage + S::kStepStages;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kBarP + x % S::kScores));
            }
            if (!ok) break;
            if (!(ok = product(x - 1))) break;
            tc_fence_after();
            const float f = p.scale * exp2f(level);
            // Whole tiles go out through the memory of the unit's last V stages, which hold as many rows
            // and columns: 16 bytes a thread by the 128-byte swizzle, and from there by the copy engine,
            // which the copies' warp asks before it loads those stages again.  (Stores of the threads' own
            // rows, 32 rows a warp, kept the load-store unit busy for a third of the kernel's time.)  In a
            // sequence's last tile, whose other rows are not its own, each thread stores its row.
            const bool whole = u.half * 128 + 128 <= u.count;
            const int last = (stages - S::kStepStages + quarter * 32 / S::kStageRows) % S::kSlots;
            uint8_t* tile = ring + last * S::kStageBytes + side * kMine / 64 * (S::kStageRows * 128) +
                            quarter * 32 % S::kStageRows * 128;
            __half* out = p.out + ((size_t)(u.first + i) * H + u.head) * D + side * kMine;
#pragma unroll 1
            for (int c0 = 0; c0 < kMine; c0 += 32) {
                uint32_t o[32], y[16];
                tc_ld32(acc + c0, o);
                if (u.dirty) {
                    const int* bad = c.first_bad + (size_t)u.index * D + side * kMine + c0;
#pragma unroll
                    for (int v = 0; v < 32; ++v)
                        if (i >= __ldg(bad + v)) o[v] = 0x7fffffffu;
                }
#pragma unroll
                for (int v = 0; v < 16; ++v) {
                    mul2(o[2 * v], o[2 * v + 1], f, f);
                    y[v] = half2_bits(__floats2half2_rn(__uint_as_float(o[2 * v]), __uint_as_float(o[2 * v + 1])));
                }
                const int unit0 = (side * kMine + c0) % 64 / 8;  // of the row's eight 16-byte units in the chunk
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const uint4 z = make_uint4(y[4 * v], y[4 * v + 1], y[4 * v + 2], y[4 * v + 3]);
                    if (whole)
                        *reinterpret_cast<uint4*>(tile + lane * 128 + (((unit0 + v) ^ (lane & 7)) << 4)) = z;
                    else if (i < u.count)
                        *reinterpret_cast<uint4*>(out + c0 + 8 * v) = z;
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kBarRead));
            if (whole) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kBarOut + s));  // the copies' warp takes it from here
            inters += u.inter;
        }
        if (!ok && lane == 0) fail();
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
cudaError_t adds(const LinearChunkParams& prm, const LinearMaps& maps, int num_sms, cudaStream_t stream) {
    using S = AddShape<D>;
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = once_per_device(done, [] {
        return cudaFuncSetAttribute(linear_adds_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    });
    if (e != cudaSuccess) return e;
    const long long units = (long long)prm.blocks * prm.lin.num_kv_heads * S::kTiles * S::kTiles, room = 2ll * num_sms;
    const unsigned grid = (unsigned)prm.lin.num_seqs * prm.lin.num_kv_heads + (unsigned)(units < room ? units : room);
    return launch(linear_adds_kernel<D>, dim3(grid), kAddThreads, S::kSmem, stream, maps, prm);
}

template <int D>
cudaError_t out(const LinearChunkParams& prm, const LinearMaps& maps, int num_sms, cudaStream_t stream) {
    using S = OutShape<D>;
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = once_per_device(done, [] {
        return cudaFuncSetAttribute(linear_out_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    });
    if (e != cudaSuccess) return e;
    // An odd number of CTAs, so that each takes first and second halves of blocks in turn.
    const long long units = (long long)prm.blocks * 2 * prm.lin.num_heads;
    const long long room = (long long)S::kCtas * num_sms - (S::kCtas * num_sms % 2 == 0);
    const unsigned grid = (unsigned)(units < room ? units : room);
    return launch(linear_out_kernel<D>, dim3(grid), S::kThreads, S::kSmem, stream, maps, prm);
}

}  // namespace

void linear_out_boxes(int head_dim, int* rows, int* state_rows) {
    *rows = head_dim == 256 ? OutShape<256>::kStageRows : head_dim == 128 ? OutShape<128>::kStageRows : OutShape<64>::kStageRows;
    *state_rows = head_dim == 256   ? OutShape<256>::kStateRows
                  : head_dim == 128 ? OutShape<128>::kStateRows
                                    : OutShape<64>::kStateRows;
}

cudaError_t launch_linear_adds(int head_dim, const LinearChunkParams& prm, const LinearMaps& maps, int num_sms,
                               cudaStream_t stream) {
    switch (head_dim) {
        case 64: return adds<64>(prm, maps, num_sms, stream);
        case 128: return adds<128>(prm, maps, num_sms, stream);
        case 256: return adds<256>(prm, maps, num_sms, stream);
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

cudaError_t launch_linear_out(int head_dim, const LinearChunkParams& prm, const LinearMaps& maps, int num_sms,
                              cudaStream_t stream) {
    switch (head_dim) {
        case 64: return out<64>(prm, maps, num_sms, stream);
        case 128: return out<128>(prm, maps, num_sms, stream);
        case 256: return out<256>(prm, maps, num_sms, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace pa
