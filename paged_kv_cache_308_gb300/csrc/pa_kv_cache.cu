// Writing, expanding and thinning out the paged cache: kv_append_kernel,
// kv_expand_kernel (8-bit context blocks to an fp16 copy, for the prefill
// kernel), kv_evict_select_kernel, kv_evict_move_kernel and
// kv_evict_lens_kernel.  Those that move rows are bound by memory: each moves
// its rows once, 16 bytes a lane.
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

__device__ __forceinline__ bool power_of_two(float s) {
    return (__float_as_uint(s) & 0x7fffffu) == 0 && s >= 0x1p-100f && s <= 0x1p100f;
}

// A scale to divide by: E4M3 scales are powers of two and INT8 scales have 8
// significant bits unless a caller wrote others.
struct Unit {
    float s, inv;
    bool pow2;
    bool short8;  // positive, at most 8 significant bits
    __device__ explicit Unit(float scale) : s(scale), pow2(power_of_two(scale)) {
        short8 = (__float_as_uint(scale) & 0xffffu) == 0 && scale >= 0x1p-60f && scale <= 0x1p60f;
        inv = pow2 ? __uint_as_float((254u << 23) - __float_as_uint(scale)) : scale > 0.f ? __fdiv_rn(1.f, scale) : 0.f;
    }
    __device__ __forceinline__ float of(float x) const {  // x / s; x itself for s = 0
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

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// Codes of eight values in the unit u.
// INT8, for a scale of 8 significant bits and |x| <= 127 s of at most 15 (a
// half, or a code times such a scale), without a division: t = x / s with one
// residual step, t + (x - t s) / s, is within 2^-23 t of the quotient and equal
// to it where that is a number of 24 bits.  The quotient is N / M with N <
// 2^15, so it is either a tie exactly, and then t is that tie, or at least
// 1 / (2 M) > 2^-16 t away from one: rounding t rounds the quotient.  Adding
// 1.5 * 2^23 does that (ties to even), and the sum's low byte is the code.
// Plain: what that needs is known; else a scale of more bits, infinities and
// NaN take the division.
template <int F, bool Plain>
__device__ __forceinline__ uint2 codes8(const float (&x)[8], const Unit& u) {
    uint32_t w[2];
    if constexpr (F == PA_KV_E4M3) {
        if (u.pow2) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
                w[j] = e4m3x2(x[4 * j] * u.inv, x[4 * j + 1] * u.inv) |
                       e4m3x2(x[4 * j + 2] * u.inv, x[4 * j + 3] * u.inv) << 16;
            return make_uint2(w[0], w[1]);
        }
    } else if constexpr (Plain) {
        uint32_t r[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float t = x[j] * u.inv;
            t = fmaf(fmaf(-t, u.s, x[j]), u.inv, t);
            r[j] = __float_as_uint(t + 12582912.f);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
            w[j] = __byte_perm(__byte_perm(r[4 * j], r[4 * j + 1], 0x0040),
                               __byte_perm(r[4 * j + 2], r[4 * j + 3], 0x0040), 0x5410);
        return make_uint2(w[0], w[1]);
    }
    w[0] = w[1] = 0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j >> 2] |= code_of<F>(u.of(x[j])) << (8 * (j & 3));
    return make_uint2(w[0], w[1]);
}

// Eight codes as numbers.
template <int F>
__device__ __forceinline__ void values8(uint2 w, float (&x)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t v = j < 4 ? w.x : w.y;
        if constexpr (F == PA_KV_E4M3) {
            if (j & 1) continue;
            const __half2_raw h =
                __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(v >> (8 * (j & 2))), __NV_E4M3);
            const float2 f = __half22float2(__half2(h));
            x[j] = f.x;
            x[j + 1] = f.y;
        } else {  // the byte plus 128 under the exponent of 2^23
            const uint32_t b = __byte_perm(v ^ 0x80808080u, 0x4b000000u, 0x7540 + (j & 3));
            x[j] = __uint_as_float(b) - (8388608.f + 128.f);
        }
    }
}

// Eight codes from scale s0 to the unit u.
template <int F>
__device__ __forceinline__ uint2 recode8(uint2 w, float s0, const Unit& u) {
    if constexpr (F == PA_KV_E4M3) {
        const float ratio = s0 * u.inv;
        if (u.pow2 && power_of_two(s0) && ratio <= 1.f) {
            // halves do: a code times a power of two is exact in them unless it is
            // far below the smallest code, where both round to zero
            const __half2 k = __float2half2_rn(ratio);
            uint32_t r[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t v = j ? w.y : w.x;
                uint32_t two[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const __half2 h = __half2(
                        __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(v >> (16 * i)), __NV_E4M3));
                    two[i] = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(__hmul2(h, k)), __NV_SATFINITE,
                                                        __NV_E4M3);
                }
                r[j] = two[0] | two[1] << 16;
            }
            return make_uint2(r[0], r[1]);
        }
    }
    float x[8];
    values8<F>(w, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] *= s0;
    // (a code of -128, which only a caller writes, may not fit)
    const bool low = F == PA_KV_INT8 && (__vcmpeq4(w.x, 0x80808080u) | __vcmpeq4(w.y, 0x80808080u));
    const bool plain = u.short8 && (__float_as_uint(s0) & 0xffffu) == 0 && s0 >= 0.f && s0 <= u.s && !low;
    return plain ? codes8<F, true>(x, u) : codes8<F, false>(x, u);
}

// 16 read-only bytes, loaded before any store that follows in the source (left
// to itself the compiler takes one load and one store at a time where that
// saves registers, and a warp then has one load in flight).
__device__ __forceinline__ uint4 load_ahead(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

// K's or V's of a pair of arguments, without indexing the parameter memory.
template <typename T>
__device__ __forceinline__ T of_kv(const T (&two)[2], int kv) {
    return kv ? two[1] : two[0];
}

// One warp per (block, kv head, K or V), kAppendHeads kv heads a CTA (their rows
// of a token are neighbours in memory; 1, 2 and 4 measured 32.8, 32.7 and 34.1
// us on 16 ragged chunks of up to 4096 tokens, 8 x 128): the new rows of the block
// in registers (D / 16 loads of 16 bytes a lane, all in flight together), their
// largest magnitude, the scale, then the codes.  Only a block whose scale
// grows has its older rows read and rounded again.
constexpr int kAppendHeads = 2;

template <int F, int D>
__global__ void __launch_bounds__(64 * kAppendHeads) kv_append_kernel(const KvAppendParams prm) {
    constexpr int kLanes = D / 8;            // lanes of a row: 8 halves each
    constexpr int kRows = 32 / kLanes;       // rows of a pass
    constexpr int kPasses = kBlockSize / kRows;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int kv = warp & 1, kvh = blockIdx.y * kAppendHeads + (warp >> 1);
    int b, tile, ctx, q0, q1;
    // bad tables or lengths of a sequence
    auto bad = [&](int c, int s, int e) {
        return c < 0 || s < 0 || e < s || e > prm.num_tokens || e - s > prm.max_query_len ||
               (long long)c + e - s > (long long)prm.max_blocks_per_seq * kBlockSize;
    };
    if (prm.packed) {
        if (blockIdx.x == 0 && blockIdx.y == 0) {
            // (a table out of order may hide a sequence from the search below)
            for (int i = threadIdx.x; i < prm.num_seqs; i += blockDim.x)
                if (bad(__ldg(prm.context_lens + i), __ldg(prm.query_start_loc + i), __ldg(prm.query_start_loc + i + 1)))
                    atomicOr(prm.status, PA_DEV_BAD_SEQ_LEN);
        }
        // Tile slots of sequence b from floor(q0 / 16) + 2 b on: n tokens touch at
        // most floor(n / 16) + 2 blocks, and floor(q1 / 16) - floor(q0 / 16) >=
        // floor(n / 16).  The last b whose slots begin at or before this one, by
        // 32 probes at a time; the last round's probes hold its lengths too.
        int lo = 0, hi = prm.num_seqs, step, at, loc;  // the answer is in [lo, hi)
        unsigned m;
        do {
            step = (hi - lo + 31) / 32;
            at = min(lo + lane * step, prm.num_seqs);
            loc = __ldg(prm.query_start_loc + at);
            ctx = step == 1 ? __ldg(prm.context_lens + min(at, prm.num_seqs - 1)) : 0;
            const bool before = at < hi && max(loc, 0) / kBlockSize + 2ll * at <= (long long)blockIdx.x;
            m = __ballot_sync(kFull, before) | 1u;  // (a bad table may begin anywhere)
            lo += (31 - __clz(m)) * step;
            hi = min(hi, lo + step);
        } while (step > 1);
        const int probe = 31 - __clz(m);
        b = lo;
        ctx = __shfl_sync(kFull, ctx, probe);
        q0 = __shfl_sync(kFull, loc, probe);
        q1 = __shfl_sync(kFull, loc, (probe + 1) & 31);
        if (probe == 31) q1 = __ldg(prm.query_start_loc + b + 1);
        const long long t = (long long)blockIdx.x - max(q0, 0) / kBlockSize - 2ll * b;
        if (t < 0) return;
        tile = (int)t;
    } else {
        b = blockIdx.z;
        tile = blockIdx.x;
        ctx = __ldg(prm.context_lens + b);
        q0 = __ldg(prm.query_start_loc + b);
        q1 = __ldg(prm.query_start_loc + b + 1);
    }
    if (bad(ctx, q0, q1)) {
        if (blockIdx.y == 0 && threadIdx.x == 0) atomicOr(prm.status, PA_DEV_BAD_SEQ_LEN);
        return;
    }
    const long long end = (long long)ctx + q1 - q0;
    const int blk = ctx / kBlockSize + tile;
    const long long p0 = (long long)blk * kBlockSize;  // position of the block's slot 0
    if (q1 == q0 || p0 >= end || kvh >= prm.num_kv_heads) return;
    const int lo = p0 < ctx ? (int)(ctx - p0) : 0;  // the block's new slots: [lo, hi)
    const int hi = end - p0 < kBlockSize ? (int)(end - p0) : kBlockSize;
    const int phys = __ldg(prm.block_tables + (size_t)b * prm.max_blocks_per_seq + blk);
    const int sub = lane / kLanes, col = lane % kLanes;
    const __half* src =
        of_kv(prm.fresh, kv) + ((long long)(q0 + (p0 - ctx)) * prm.num_kv_heads + kvh) * D + 8 * col;
    const size_t step = (size_t)prm.num_kv_heads * D;

    uint4 x[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int r = i * kRows + sub;
        x[i] = make_uint4(0u, 0u, 0u, 0u);
        if (r >= lo && r < hi) x[i] = load_ahead(src + r * step);
    }
    if (phys < 0 || (long long)phys >= prm.num_blocks) {
        if (blockIdx.y == 0 && threadIdx.x == 0) atomicOr(prm.status, PA_DEV_BAD_BLOCK_ID);
        return;
    }
    const size_t bh = (size_t)phys * prm.num_kv_heads + kvh;
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
        // the largest magnitude of the finite ones: bits of |x|, two halves at a time
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < kPasses; ++i)
            top = __vmaxu2(top, __vmaxu2(__vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu),
                                         __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu)));
        uint32_t amax = max(top & 0xffffu, top >> 16);
        const bool special = __any_sync(kFull, amax >= 0x7c00u);
        if (special) {
            amax = 0;
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t v = (w[j >> 1] >> (16 * (j & 1))) & 0x7fffu;
                    amax = v < 0x7c00u ? max(amax, v) : amax;
                }
            }
        }
        amax = __reduce_max_sync(kFull, amax);
        const float s1 = fmaxf(s0, block_scale<F>(__half2float(__ushort_as_half(static_cast<unsigned short>(amax)))));
        const Unit u(s1);
        const bool plain = u.short8 && !special;
        uint8_t* dst = static_cast<uint8_t*>(of_kv(prm.cache, kv)) + bh * kBlockSize * D + 8 * col;
        if (s1 > s0 && lo > 0) {
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                const int r = i * kRows + sub;
                if (r < lo) {
                    uint2* w = reinterpret_cast<uint2*>(dst + r * D);
                    *w = recode8<F>(*w, s0, u);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const int r = i * kRows + sub;
            if (r >= lo && r < hi) {
                const __half2* h = reinterpret_cast<const __half2*>(&x[i]);
                float f[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 two = __half22float2(h[j]);
                    f[2 * j] = two.x;
                    f[2 * j + 1] = two.y;
                }
                *reinterpret_cast<uint2*>(dst + r * D) = plain ? codes8<F, true>(f, u) : codes8<F, false>(f, u);
            }
        }
        __syncwarp();  // every lane has read the old scale
        if (lane == 0) *scale = s1;
    }
}

// An 8-bit context block to halves (values above fp16's range become its
// largest), and the copy's block table; with factors only the power of two of
// the block's scale goes into the halves.  One warp per (block, kv head, K or V).
template <int F, int D>
__global__ void __launch_bounds__(64) kv_expand_kernel(const KvExpandParams prm) {
    constexpr int kPasses = kBlockSize * D / (32 * 16);  // 16 codes a lane
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int kv = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int blk = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z;
    const int to = b * prm.blocks_per_seq + blk;
    const bool first = kvh == 0 && threadIdx.x == 0;
    if (first) prm.tables[to] = to;
    const int ctx = __ldg(prm.context_lens + b);
    // a context out of range is reported and skipped by the prefill kernel
    if (ctx < 0 || ctx > prm.max_context_len || blk * kBlockSize >= ctx) return;
    const int phys = __ldg(prm.block_tables + (size_t)b * prm.max_blocks_per_seq + blk);
    if (phys < 0 || (long long)phys >= prm.num_blocks) {
        // the prefill kernel treats it like a bad block of its own
        if (first) {
            prm.tables[to] = -1;
            atomicOr(prm.status, PA_DEV_BAD_BLOCK_ID);
        }
        if (prm.factors && lane == 0) prm.factors[2 * ((size_t)to * prm.num_kv_heads + kvh) + kv] = 1.f;
        return;
    }
    const size_t bh = (size_t)phys * prm.num_kv_heads + kvh;
    const uint4* src = reinterpret_cast<const uint4*>(of_kv(prm.cache, kv) + bh * kBlockSize * D) + lane;
    // through shared memory, each lane its own pieces: every load in flight
    // without a register (held in registers, the compiler took one or two at a
    // time: 43 us for 4 x 8192 tokens of 4 x 256)
    __shared__ uint4 held[2][kPasses][32];
#pragma unroll
    for (int i = 0; i < kPasses; ++i)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(&held[kv][i][lane])), "l"(src + 32 * i)
                     : "memory");
    float s = __ldg(of_kv(prm.scales, kv) + bh);
    if (prm.factors) {
        // s = f 2^e, 1 <= f < 2: the copy holds code 2^e, exact in fp16 for e from
        // -24 to 9, and f goes into the factors
        const uint32_t bits = __float_as_uint(s);
        float f = 1.f;
        if (s >= 0x1p-126f && s <= 0x1p126f) {
            f = __uint_as_float((bits & 0x7fffffu) | 0x3f800000u);
            s = __uint_as_float(bits & 0x7f800000u);
        }
        if (lane == 0) prm.factors[2 * ((size_t)to * prm.num_kv_heads + kvh) + kv] = f;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    uint8_t* dst = reinterpret_cast<uint8_t*>(of_kv(prm.expanded, kv) +
                                              ((size_t)to * prm.num_kv_heads + kvh) * kBlockSize * D);
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const uint4 x = held[kv][i][lane];
        uint32_t h[8];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float f[8];
            values8<F>(j ? make_uint2(x.z, x.w) : make_uint2(x.x, x.y), f);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                // saturated; NaN stays NaN
                const float a = f[2 * k] * s, c = f[2 * k + 1] * s;
                h[4 * j + k] = half2_bits(__hmax2_nan(
                    __hmin2_nan(__floats2half2_rn(a, c), __float2half2_rn(65504.f)), __float2half2_rn(-65504.f)));
            }
        }
        // a lane's 32 bytes in one store: as two of 16 each would write half a sector
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + 32 * (32 * i + lane)),
                     "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]), "r"(h[4]), "r"(h[5]), "r"(h[6]), "r"(h[7])
                     : "memory");
    }
}

// What a sequence keeps (see pa_kv_evict); false: nothing, or out of range.
struct KeepPlan {
    int L, k, sinks, recent;
    bool bad;
    __device__ KeepPlan(const KvEvictParams& prm, int b)
        : KeepPlan(prm, __ldg(prm.seq_lens + b), __ldg(prm.keep_lens + b)) {}
    __device__ KeepPlan(const KvEvictParams& prm, int len, int want) : L(len) {
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

// The weight of a key; NaN and the zeros, which share keys, are read again.
__device__ __forceinline__ float weight_of(uint32_t key, const float* w) {
    const uint32_t bits = (key & 0x80000000u) ? key & 0x7fffffffu : ~key;
    return bits == 0u || bits == 0xff800000u ? *w : __uint_as_float(bits);
}

// The k - r - s heaviest tokens between the first s and the last r, by a
// radix select over the weights' ordered bits: three rounds of a histogram
// (11, 11 and 10 bits) find the smallest kept key T and how many of the
// tokens that equal it are kept (the first ones); then a scan over the
// positions gives each kept token its place.  The rounds end where a bin is kept
// whole.  A (sequence, kv head) has a block to itself, or a cluster of them: each
// takes a stretch of the positions, whose keys stay in its shared memory (the
// weights are read once), the histograms are summed through distributed shared
// memory, and a block's first output follows from its predecessors' counts.  Integer counts only, so the result does not
// depend on the order of the atomics.  Bound by latency: per round three
// barriers of the block, or two and one of the cluster.
constexpr int kHistWords = 2048 + 2048 + 1024;
constexpr int kMaxCluster = 8;  // blocks of a cluster

// Exclusive prefix sums of a pair of counts over the block's threads (in
// their order), and the block's totals.  One barrier; `part` (2 x 32 words)
// must not be in use.
__device__ __forceinline__ uint2 block_scan(uint2 v, unsigned (*part)[32], uint2* total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint2 incl = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const unsigned a = __shfl_up_sync(kFull, incl.x, off), c = __shfl_up_sync(kFull, incl.y, off);
        if (lane >= off) incl.x += a, incl.y += c;
    }
    if (lane == 31) part[0][warp] = incl.x, part[1][warp] = incl.y;
    __syncthreads();
    uint2 w = make_uint2(part[0][lane], part[1][lane]);  // 32 warps: every warp scans their totals
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const unsigned a = __shfl_up_sync(kFull, w.x, off), c = __shfl_up_sync(kFull, w.y, off);
        if (lane >= off) w.x += a, w.y += c;
    }
    *total = make_uint2(__shfl_sync(kFull, w.x, 31), __shfl_sync(kFull, w.y, 31));
    const unsigned bx = __shfl_sync(kFull, w.x, (warp + 31) & 31), by = __shfl_sync(kFull, w.y, (warp + 31) & 31);
    return make_uint2((warp ? bx : 0u) + incl.x - v.x, (warp ? by : 0u) + incl.y - v.y);
}

// One: no cluster, a block has a (sequence, kv head) to itself; two share an SM,
// in 32 registers (768 pairs of up to 1024 tokens: 32.0 instead of 40.0 device us
// with the move; 32 pairs of up to 8192 21.2 instead of 21.0), a cluster's do not (27.4
// instead of 24.3).
template <bool One>
__global__ void __launch_bounds__(kEvictThreads, One ? 2 : 1) kv_evict_select_kernel(const KvEvictParams prm) {
    extern __shared__ __align__(16) uint32_t keys[];  // prm.key_words of them
    __shared__ __align__(8) unsigned hist[kHistWords];
    __shared__ __align__(8) unsigned coarse[3][64];
    __shared__ unsigned part[2][32];
    __shared__ unsigned found[3][3];  // per round: bin, tokens to take from it on, tokens in it
    __shared__ __align__(8) unsigned counts[2];  // this block's kept for sure, and ties
    cg::cluster_group cluster = cg::this_cluster();
    const int CS = One ? 1 : (int)cluster.num_blocks(), rank = One ? 0 : (int)cluster.block_rank();
    auto of_block = [&](unsigned* p, int r) {  // a shared array of block r of the cluster
        if constexpr (One) return p;
        else return cluster.map_shared_rank(p, r);
    };
    const int kvh = blockIdx.x / CS, b = blockIdx.y;
    const int tid = threadIdx.x, lane = tid & 31;
    for (int i = tid; i < kHistWords; i += kEvictThreads) hist[i] = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const KeepPlan plan(prm, b);
    if (plan.bad) {  // the whole cluster leaves here
        if (blockIdx.x == 0 && tid == 0) atomicOr(prm.status, PA_DEV_BAD_SEQ_LEN);
        return;
    }
    const int L = plan.L, k = plan.k;
    if (prm.new_lens && blockIdx.x == 0 && tid == 0) prm.new_lens[b] = k;
    const size_t row = (size_t)b * prm.num_kv_heads + kvh;
    const float* w = prm.weights + row * prm.weights_stride;
    int32_t* kept = prm.kept + row * prm.max_keep_len;
    float* dst_w = prm.dst_weights ? prm.dst_weights + row * prm.dst_weights_stride : nullptr;
    auto put = [&](int at, int t) {
        kept[at] = t;
        if (dst_w) dst_w[at] = w[t];
    };

    // sinks and recent ones keep their order around the rest
    auto put_protected = [&]() {
        for (int i = rank * kEvictThreads + tid; i < plan.sinks; i += CS * kEvictThreads) put(i, i);
        for (int i = rank * kEvictThreads + tid; i < plan.recent; i += CS * kEvictThreads)
            put(k - plan.recent + i, L - plan.recent + i);
    };

    // this block's stretch of the tokens between them
    const int m0 = plan.sinks, m1 = L - plan.recent, mid = m1 - m0;
    const int each = (mid + CS - 1) / CS;
    const int t0 = min(m1, m0 + rank * each), n = min(m1 - t0, each);
    unsigned need = (unsigned)(k - plan.recent - plan.sinks);  // of the mid tokens
    if (need == 0 || need == (unsigned)mid) put_protected();
    if (need == 0) return;        // the same for the whole cluster
    if (need == (unsigned)mid) {  // all of them: L <= the budget
        for (int i = tid; i < n; i += kEvictThreads) put(t0 + i, t0 + i);
        return;
    }
    // Each warp takes a run of the stretch, a lane four neighbours at a time;
    // keys past the stretch are 0, below every weight's.
    const int warp = tid >> 5;
    const int run = (n + 4 * kEvictThreads - 1) / (4 * kEvictThreads) * 128;
    const int i0 = warp * run + 4 * lane, i1 = min(n, (warp + 1) * run);
    const bool held = 32 * run <= prm.key_words;
    auto fresh_keys = [&](int i) {
        const float* p = w + t0 + i;
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = i + j < n ? p[j] : 0.f;
        return make_uint4(i < n ? order_key(v[0]) : 0u, i + 1 < n ? order_key(v[1]) : 0u,
                          i + 2 < n ? order_key(v[2]) : 0u, i + 3 < n ? order_key(v[3]) : 0u);
    };
    auto keys_of = [&](int i) { return held ? *reinterpret_cast<const uint4*>(keys + i) : fresh_keys(i); };
    __syncthreads();  // the histograms are clear
    uint32_t T = 0, mask = 0;  // the key so far, and its bits
#pragma unroll
    for (int round = 0; round < 3; ++round) {
        unsigned* h = hist + 2048 * round;
        const int shift = round == 0 ? 21 : round == 1 ? 10 : 0, bins = round == 2 ? 1024 : 2048;
        if (round == 0) {
            // Weights that underflowed to zero can be most of them: counted apart,
            // lest every atomic of a warp queue on their bin.
            unsigned zeros = 0;
#pragma unroll 2
            for (int i = i0; i < (warp + 1) * run; i += 128) {  // to the run's end: keys past n become 0
                const uint4 q = fresh_keys(i);
                if (held) *reinterpret_cast<uint4*>(keys + i) = q;
                const uint32_t k4[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    zeros += k4[j] == 0x80000000u;
                    if (k4[j] != 0u && k4[j] != 0x80000000u) atomicAdd(h + (k4[j] >> 21), 1u);
                }
            }
            zeros = __reduce_add_sync(kFull, zeros);
            if (lane == 0 && zeros) atomicAdd(h + (0x80000000u >> 21), zeros);
        } else {
            for (int i = i0; i < i1; i += 128) {
                const uint4 q = keys_of(i);
                const uint32_t k4[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if ((k4[j] & mask) == T) atomicAdd(h + ((k4[j] >> shift) & (bins - 1)), 1u);
            }
        }
        // Sums over the cluster of 64 groups of bins find the group, then of the
        // group's bins the bin: reading all bins of all blocks was bound by the
        // network between the SMs (2.4 us a round with 8 blocks).
        __syncthreads();
        const int per = bins / 64;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const unsigned sum = __reduce_add_sync(kFull, lane < per ? h[(2 * warp + j) * per + lane] : 0u);
            if (lane == 0) coarse[round][2 * warp + j] = sum;
        }
        if constexpr (One) {
            if (round == 0) put_protected();
            __syncthreads();
        } else {
            cluster.barrier_arrive();
            if (round == 0) put_protected();  // while the others arrive
            cluster.barrier_wait();
        }
        if (warp == 0) {
            // in descending order: lane i has groups 63 - 2 i and 62 - 2 i, then bin per - 1 - i
            auto pick = [&](unsigned a, unsigned c, unsigned& above) {  // the lane whose counts reach `need`
                unsigned incl = a + c;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const unsigned up = __shfl_up_sync(kFull, incl, off);
                    if (lane >= off) incl += up;
                }
                above = incl - a - c;
                return __ffs(__ballot_sync(kFull, above < need && need <= incl)) - 1;
            };
            unsigned a = 0, c = 0, above;
            uint2 two[kMaxCluster];  // all reads on their way at once
#pragma unroll
            for (int r = 0; r < kMaxCluster; ++r)
                two[r] = r < CS ? *reinterpret_cast<const uint2*>(of_block(coarse[round], r) + 62 - 2 * lane)
                                : make_uint2(0u, 0u);
#pragma unroll
            for (int r = 0; r < kMaxCluster; ++r) a += two[r].y, c += two[r].x;
            int who = pick(a, c, above);
            const bool second = need > above + a;
            const int group = 63 - 2 * who - (int)__shfl_sync(kFull, (unsigned)second, who);
            need -= __shfl_sync(kFull, above + (second ? a : 0u), who);  // less the groups above
            a = 0;
            unsigned one[kMaxCluster];
#pragma unroll
            for (int r = 0; r < kMaxCluster; ++r)
                one[r] = r < CS && lane < per ? of_block(h, r)[group * per + per - 1 - lane] : 0u;
#pragma unroll
            for (int r = 0; r < kMaxCluster; ++r) a += one[r];
            who = pick(a, 0u, above);
            need -= __shfl_sync(kFull, above, who);
            a = __shfl_sync(kFull, a, who);
            if (lane == 0)
                found[round][0] = (unsigned)(group * per + per - 1 - who), found[round][1] = need, found[round][2] = a;
        }
        __syncthreads();
        T |= found[round][0] << shift;
        mask |= (uint32_t)(bins - 1) << shift;
        need = found[round][1];
        if (need == found[round][2]) {  // the bin is kept whole, whatever its keys' other bits
            T -= 1;                     // (no weight's key is below 2^22)
            need = 0;
            break;
        }
    }
    // Kept: the keys above T, and of those equal to it the first `need`.
    unsigned sure = 0, tie = 0;
    for (int i = i0; i < i1; i += 128) {
        const uint4 q = keys_of(i);
        const uint32_t k4[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            sure += k4[j] > T;
            tie += k4[j] == T;
        }
    }
    uint2 total;
    uint2 before = block_scan(make_uint2(sure, tie), part, &total);
    before = make_uint2(__shfl_sync(kFull, before.x, 0), __shfl_sync(kFull, before.y, 0));  // the warp's first
    if (tid == 0) counts[0] = total.x, counts[1] = total.y;
    if constexpr (!One) {
        cluster.sync();
        uint2 others[kMaxCluster];
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
            others[r] = r < rank ? *reinterpret_cast<const uint2*>(of_block(counts, r)) : make_uint2(0u, 0u);
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) before.x += others[r].x, before.y += others[r].y;
    }
    // the warp's run again, a key a lane
    const unsigned below = (1u << lane) - 1u;
    const float* from = w + t0;
    kept += plan.sinks;
    if (dst_w) dst_w += plan.sinks;
    for (int i = warp * run + lane; i - lane < i1; i += 32) {
        const uint32_t key = i >= n ? 0u : held ? keys[i] : order_key(from[i]);
        const unsigned bs = __ballot_sync(kFull, key > T), be = __ballot_sync(kFull, key == T);
        const unsigned my_tie = before.y + __popc(be & below);
        if (key > T || (key == T && my_tie < need)) {
            const unsigned at = before.x + __popc(bs & below) + min(my_tie, need);
            kept[at] = t0 + i;
            if (dst_w) dst_w[at] = weight_of(key, from + i);
        }
        before.x += __popc(bs);
        before.y += __popc(be);
    }
    if constexpr (!One) cluster.sync();  // no block leaves while another may still read its counts
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
    const size_t row = (size_t)b * prm.num_kv_heads + kvh;
    // what the lengths allow is known later: these loads stay inside the arrays
    const int i = blk * kBlockSize + (lane & (kBlockSize - 1));
    const int t = i < prm.max_keep_len ? prm.kept[row * prm.max_keep_len + i] : 0;
    const int to = __ldg(prm.dst_block_tables + (size_t)b * prm.dst_max_blocks_per_seq + blk);
    const KeepPlan plan(prm, b);
    if (plan.bad || blk * kBlockSize >= plan.k) return;
    const int n = min(kBlockSize, plan.k - blk * kBlockSize);
    // lane r < 16: where the block's r-th row comes from
    int from = -1, slot = 0;
    if (lane < n) {
        slot = t % kBlockSize;
        from = __ldg(prm.block_tables + (size_t)b * prm.max_blocks_per_seq + t / kBlockSize);
        if (from < 0 || (long long)from >= prm.src_blocks) {
            atomicOr(prm.status, PA_DEV_BAD_BLOCK_ID);
            from = -1;
        }
    }
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
        x[i] = make_uint4(0u, 0u, 0u, 0u);
        if (f >= 0) x[i] = load_ahead(src + at);
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
                const uint2 a = recode8<F>(make_uint2(x[i].x, x[i].y), s, u);
                const uint2 c = recode8<F>(make_uint2(x[i].z, x[i].w), s, u);
                x[i] = make_uint4(a.x, a.y, c.x, c.y);
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

// new_lens in place of seq_lens or keep_lens: the selection's and the move's
// blocks read those, so it is written when all of them have ended (3 sequences of
// 300 tokens 7.2 instead of 6.2 us on the device).
__global__ void __launch_bounds__(256) kv_evict_lens_kernel(const KvEvictLensParams prm) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int b = blockIdx.x * blockDim.x + threadIdx.x;
    if (b >= prm.num_seqs) return;
    const KeepPlan plan(prm.evict, prm.evict.seq_lens[b], prm.evict.keep_lens[b]);
    if (!plan.bad) prm.new_lens[b] = plan.k;
}

template <typename P>
cudaError_t launch(void (*kern)(P), const P& prm, dim3 grid, int threads, int cluster, cudaStream_t stream,
                   size_t smem = 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
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

#define PA_FOR_D(F_, K_, THREADS_)                                                                          \
    if (format == F_ && head_dim == 64) return launch(K_<F_, 64>, prm, grid, THREADS_, 0, stream);          \
    if (format == F_ && head_dim == 128) return launch(K_<F_, 128>, prm, grid, THREADS_, 0, stream);        \
    if (format == F_ && head_dim == 256) return launch(K_<F_, 256>, prm, grid, THREADS_, 0, stream);

cudaError_t launch_kv_append(int format, int head_dim, const KvAppendParams& prm, int tiles, cudaStream_t stream) {
    const dim3 grid(tiles, (prm.num_kv_heads + kAppendHeads - 1) / kAppendHeads, prm.packed ? 1 : prm.num_seqs);
    const int threads = 64 * (prm.num_kv_heads < kAppendHeads ? prm.num_kv_heads : kAppendHeads);
    PA_FOR_D(PA_KV_F16, kv_append_kernel, threads)
    PA_FOR_D(PA_KV_E4M3, kv_append_kernel, threads)
    PA_FOR_D(PA_KV_INT8, kv_append_kernel, threads)
    return cudaErrorInvalidValue;
}

cudaError_t launch_kv_expand(int format, int head_dim, const KvExpandParams& prm, dim3 grid, cudaStream_t stream) {
    PA_FOR_D(PA_KV_E4M3, kv_expand_kernel, 64)
    PA_FOR_D(PA_KV_INT8, kv_expand_kernel, 64)
    return cudaErrorInvalidValue;
}

template <bool One>
static cudaError_t launch_select(const KvEvictParams& prm, int num_seqs, int cluster, cudaStream_t stream) {
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = once_per_device(done, [] {
        return cudaFuncSetAttribute(kv_evict_select_kernel<One>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    kEvictKeyWords * 4);
    });
    if (e != cudaSuccess) return e;
    return launch(kv_evict_select_kernel<One>, prm, dim3(prm.num_kv_heads * cluster, num_seqs), kEvictThreads,
                  One ? 0 : cluster, stream, prm.key_words * 4);
}

cudaError_t launch_kv_evict_select(const KvEvictParams& prm, int num_seqs, int cluster, cudaStream_t stream) {
    return cluster == 1 ? launch_select<true>(prm, num_seqs, cluster, stream)
                        : launch_select<false>(prm, num_seqs, cluster, stream);
}

cudaError_t launch_kv_evict_lens(const KvEvictLensParams& prm, cudaStream_t stream) {
    return launch(kv_evict_lens_kernel, prm, dim3((prm.num_seqs + 255) / 256), 256, 0, stream);
}

cudaError_t launch_kv_evict_move(int format, int head_dim, const KvEvictParams& prm, dim3 grid, cudaStream_t stream) {
    PA_FOR_D(PA_KV_F16, kv_evict_move_kernel, 64)
    PA_FOR_D(PA_KV_E4M3, kv_evict_move_kernel, 64)
    PA_FOR_D(PA_KV_INT8, kv_evict_move_kernel, 64)
    return cudaErrorInvalidValue;
}

}  // namespace pa
