// Decode attention over a cache in 8 bits (or fp16), and the accumulation of
// its attention weights.
//
// kv_partition_kernel<F, D, NS, Cluster>: the decomposition of pa_partition_kernel
// (partitions of a sequence, by kv head) over cache format F.  The math
// per 16-token block, for the <= 8 query heads of a kv head (log2 domain,
// c = scale * log2 e):
//     s[t, h] = c ks sum_d k8[t, d] q[h, d]             ks, vs: the block's scales
//     m'      = max(m, max_t s),  p = 2^(s - m' + kShift)
//     l       = l 2^(m - m') + sum_t p
//     o[d, h] = o 2^(m - m') + sum_t v8[t, d] p16[t, h],  p16 = half(p vs / vr)
// The scales stay outside the products, so K and V enter the tensor cores as
// exact halves (a code is at most 448).  ks costs one multiply per score.  vs
// multiplies the probabilities, relative to vr, the largest block scale so
// far, which o is kept in units of (when it grows, o is rescaled along with
// the change of m): one multiply per probability instead of one per output.
// A block whose vs is below 2^-20 vr, where p16 could lose bits, adds vs / vr
// times its product to o instead.
// p is rounded to fp16 for the product (relative 2^-11; the shift keeps
// products of probability and scale ratio down to 2^-28 normal and 2^-38 above
// zero); l adds the unrounded p, in 32 bits as m and o are.  So the weights of
// the accumulation have the error of a score (a dot product in 32 bits) and of
// the exponential (2^-22), and none of the rounding to fp16.
//
// From 8 bits to MMA fragments: a 32-bit register of ldmatrix holds four
// consecutive d of one token (K), or two d of two neighbouring tokens (V,
// transposed form).  The order of the k index of an MMA is free as long as
// both operands agree, and so is the order of the output's rows: K's four d
// become the k pairs (2c, 2c+1) and (2c+8, 2c+9), for which Q is loaded in
// the same order, and V's two d become rows g and g+8.  So no byte crosses
// lanes: e4m3 takes one cvt per two elements (plus one byte permute per
// register of V), int8 two byte permutes and two subtractions per four (bytes
// with the sign bit flipped, placed under the exponent of 1024, minus 1152).
//
// How the work is dealt out.  Flat form: a grid of the CTAs the SMs hold at
// once, C per kv head.  The blocks of the batch's sequences form one list, in
// which each sequence counts kLead units more than it has blocks (what it costs
// to begin one); CTA c takes the c-th of equal runs of units.  So the CTAs end
// together whatever the lengths, none is launched for a partition that its
// sequence does not have, and the host never reads the lengths: every warp
// finds its run from seq_lens itself.  A run within one sequence is dealt
// round-robin to the CTA's warps, which merge their states into one partial
// (slot c).  A run that crosses sequences is cut into one run per warp; the
// warps then work alone, sequence by sequence, the copies running on from one
// into the next, and each segment leaves a partial (slot C + warp + b, for the
// b-th sequence: from one segment to the next either the warp's number or b
// grows, so slots never collide) or, if it is the whole sequence, the output.
// Grid form (one sequence, a partition size was given, or every sequence fits
// one CTA): one CTA per (partition, kv head, sequence).
// Cluster form (few and short sequences): a cluster of CTAs per (kv head,
// sequence), whose warps take the blocks in turns.  It merges over distributed
// shared memory and adds the weights itself: no second launch, which costs
// about 3 us on the device and 2 on the host.
//
// kv_merge_kernel: the log-sum-exp merge of the partials, and in further CTAs
// of the same launch weights_out = weights_in + sum_h 2^(s - lse) from the
// scores that the partition kernel left: 4 bytes per (token, head) written
// and read again, instead of K's D bytes a second time.
#include "pa_kv.h"

#include <cooperative_groups.h>
#include <cuda_fp8.h>
#include <math.h>

#include "pa_decode.h"
#include "pa_device.cuh"

namespace pa {
namespace {

namespace cg = cooperative_groups;

constexpr float kShift = 14.f;
constexpr int kLead = 6;  // units a sequence counts beyond its blocks

// The flat form's runs: `ctas` of them over `units` units, q each and one more
// for the first r, at least kMinUnits long while there are as many units.
struct FlatRuns {
    static constexpr int kMinUnits = 2 * kKvWarps;
    int most, ctas, q, r;
    __device__ FlatRuns(int units, int most_) : most(most_) {
        ctas = min(most, units / kMinUnits);
        if (ctas == 0) ctas = units > 0 ? 1 : 0;
        q = ctas ? units / ctas : 0;
        r = units - q * ctas;
    }
    __device__ int begin(int c) const { return c * q + min(c, r); }
    __device__ int of(int u) const { return u < r * (q + 1) ? u / (q + 1) : r + (u - r * (q + 1)) / q; }
    // a warp's part of a run that crosses sequences
    static __device__ int warp_begin(int u0, int u1, int w) {
        return u0 + (int)((long long)(u1 - u0) * w / kKvWarps);
    }
    __device__ int warp_of(int c, int u) const {
        const int u0 = begin(c), u1 = begin(c + 1);
        int w = 0;
        while (w + 1 < kKvWarps && warp_begin(u0, u1, w + 1) <= u) ++w;
        return w;
    }
};

// The partial slots of a sequence with n blocks whose units begin at `first`:
// three stretches (some empty), in the order of its tokens -- warps of a first
// CTA that it shares with the sequence before, CTAs of its own, warps of a
// last one.
struct SeqParts {
    int first[3], count[3];
    __device__ SeqParts(const FlatRuns& runs, int at, int n, int b) {
        const int ua = at + kLead, uz = ua + n - 1;  // units of its first and last block
        int ca = runs.of(ua), cz = runs.of(uz);
        auto whole = [&](int c) { return runs.begin(c) >= at && runs.begin(c + 1) <= uz + 1; };
        auto slot = [&](int c, int w) { return runs.most + c * kKvWarps + w + b; };
        first[0] = first[1] = first[2] = count[0] = count[1] = count[2] = 0;
        if (ca == cz && !whole(ca)) {
            const int wa = runs.warp_of(ca, ua);
            first[0] = slot(ca, wa);
            count[0] = runs.warp_of(ca, uz) - wa + 1;
            return;
        }
        if (!whole(ca)) {
            const int wa = runs.warp_of(ca, ua);
            first[0] = slot(ca, wa);
            count[0] = kKvWarps - wa;
            ++ca;
        }
        if (!whole(cz)) {
            first[2] = slot(cz, 0);
            count[2] = runs.warp_of(cz, uz) + 1;
            --cz;
        }
        first[1] = ca;
        count[1] = cz - ca + 1;
    }
};

template <int F, int D, int NS>
struct KvShape {
    static constexpr int kNW = kKvWarps;
    static constexpr int kRow = D * (F == PA_KV_F16 ? 2 : 1);    // bytes of a token's row
    static constexpr int kTile = kBlockSize * kRow;              // K (or V) of a block
    static constexpr int kStage = 2 * kTile;
    static constexpr int kStageArea = kNW * NS * kStage;
    static constexpr int kTilesM = D / 16;                       // m-tiles of P.V
    static constexpr int kRedStride = D + 4;
    static constexpr int kRedBytes = kNW * kMaxGroup * kRedStride * 4;
    static constexpr int kArea = kStageArea > kRedBytes ? kStageArea : kRedBytes;
    static constexpr int kSmem = kArea + 2 * kNW * kMaxGroup * 4;  // + (m, l) of the warps
    static_assert(kSmem <= 227 * 1024, "shared memory budget of one CTA");
};

// Byte offset of 16-byte unit `unit` of row `row` in a staged tile: 128-byte
// columns, the units of a row exchanged by the row's number modulo 8 (64-byte
// rows: modulo 4, every other row), so that the eight rows of an ldmatrix
// matrix lie in different banks.
template <int F, int D>
__device__ __forceinline__ uint32_t unit_at(int row, int unit) {
    if constexpr (F != PA_KV_F16 && D == 64)
        return static_cast<uint32_t>(row * 64 + ((unit ^ ((row >> 1) & 3)) << 4));
    else
        return static_cast<uint32_t>((unit >> 3) * (kBlockSize * 128)) + swz(row, unit & 7);
}

// Start copying a tile (contiguous in memory) to `stage`, 16 bytes a lane and
// instruction.  Pass i begins kRows i rows on; as kRows is a power of two, row
// & 7 is (kRows i & 7) ^ (the row in the pass), so the swizzle of a pass is the
// first one's, exclusive-or a constant.
template <int F, int D>
__device__ __forceinline__ void copy_tile(uint32_t stage, const uint8_t* src) {
    constexpr int kRow = D * (F == PA_KV_F16 ? 2 : 1);
    constexpr int kRows = 512 / kRow;  // rows of a pass (1 to 8)
    const int lane = threadIdx.x & 31;
    const uint32_t first = stage + unit_at<F, D>(lane * 16 / kRow, lane * 16 % kRow / 16);
    src += lane * 16;
#pragma unroll
    for (int i = 0; i < kBlockSize / kRows; ++i) {
        constexpr bool kPlain = F != PA_KV_F16 && D == 64;  // 8 rows a pass: nothing changes
        const uint32_t at = kPlain ? first + i * 512 : (first ^ ((kRows * i & 7) << 4)) + kRows * i * 128;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(src + 512 * i) : "memory");
    }
}

__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void copies_wait() {  // all but the latest N groups have landed
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Halves of the four bytes of w: bytes 0 and 1, bytes 2 and 3.  INT8 bytes come
// with the sign bit flipped (v + 128).
template <int F>
__device__ __forceinline__ void to_halves(uint32_t w, uint32_t& lo, uint32_t& hi) {
    if constexpr (F == PA_KV_E4M3) {
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
    } else {
        const __half2 k = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152
        const uint32_t a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);
        lo = half2_bits(__hsub2(*reinterpret_cast<const __half2*>(&a), k));
        hi = half2_bits(__hsub2(*reinterpret_cast<const __half2*>(&b), k));
    }
}

template <int F>
__device__ __forceinline__ uint32_t unsign(uint32_t w) {
    return F == PA_KV_INT8 ? w ^ 0x80808080u : w;
}

// D = A . B (no accumulator read).
__device__ __forceinline__ void mma_16816_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// 2^x by the hardware's approximation (relative error about 2^-22; results
// below 2^-126 are 0, which no sum here would notice).
__device__ __forceinline__ float pow2_of(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// (d of o[mt][0..1], d of o[mt][2..3]) of a lane with row group g.
template <int F>
__device__ __forceinline__ int out_dim(int mt, int g, int hi) {
    return F == PA_KV_F16 ? 16 * mt + g + 8 * hi : 16 * mt + 2 * g + hi;
}

// Stages per warp, and the CTAs an SM holds, within its registers (D / 4 of O and
// D / 8 of Q a thread) and 228 KB of shared memory.  More copies in flight than
// the latency asks for only queue in memory and let the SMs drift apart: 3
// instead of 2 stages at head_dim 256 in 8 bits (192 against 128 KB per SM)
// took 132.0 instead of 126.1 us for 400,000 tokens of 4 kv heads, 3 and 4
// instead of 2 at 128 (144, 192 / 96 KB) 133.1 and 138.5 instead of 128.4.  At
// 64, whose blocks are small next to a block's latency, 3 were slower than 4
// (152.0 / 149.9), and 16-bit tiles want 192 KB.
template <int F, int D>
constexpr int stages_of() {
    return F == PA_KV_F16 ? (D == 64 ? 4 : 3) : (D == 64 ? 4 : 2);
}
template <int F, int D>
constexpr int ctas_of() {
    return F == PA_KV_F16 ? (D == 256 ? 1 : D == 128 ? 2 : 3) : (D == 256 ? 2 : D == 128 ? 3 : 5);
}

// Scores are read again by the next kernel: K and V passing through L2 should
// not push them out.
__device__ __forceinline__ uint64_t keep_in_l2() {
    uint64_t policy;
    asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(policy));
    return policy;
}
__device__ __forceinline__ void store_kept(float* p, float v, uint64_t policy) {
    asm volatile("st.global.L2::cache_hint.f32 [%0], %1, %2;" ::"l"(p), "f"(v), "l"(policy) : "memory");
}

// A warp's online softmax over the heads of a kv head: lane (g, c) of an MMA
// fragment holds heads 2c and 2c + 1.
template <int D>
struct WarpState {
    float o[D / 16][4];
    float m0, m1;  // running maximum
    float l0, l1;  // this lane's share of the exp sums
    float vr, rvr; // V unit of o, and its reciprocal (0: no block yet)
    __device__ void clear() {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        m0 = m1 = -INFINITY;
        l0 = l1 = 0.f;
        vr = rvr = 0.f;
    }
};

// One 16-token block.  `kst`, `vst`: its staged K and V, `vgen` V as a generic
// pointer.  `ks`: softmax scale (log2) times K's block scale.  `score0`: where
// the scores of head 2c from the block's first token on go (null: nowhere),
// head 2c + 1's `score_stride` further if `two`.
template <int F, int D>
__device__ __forceinline__ void block_update(WarpState<D>& st, const uint32_t (&qb)[D / 16][2], uint32_t kst,
                                             uint32_t vst, uint8_t* vgen, int nvalid, float ks, float vs,
                                             float* score0, long long score_stride, bool two) {
    constexpr int kRow = D * (F == PA_KV_F16 ? 2 : 1);
    const int lane = threadIdx.x & 31;
    const int g = lane >> 2;
    const int mi = lane >> 3, r8 = lane & 7;

    // S^T = K . Q^T, in several accumulators for shorter chains
    constexpr int kAcc = D == 256 ? 4 : 2;
    float sa[kAcc][4];
    const int rq = r8 + ((mi & 1) << 3);
    if constexpr (F == PA_KV_F16) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            uint32_t a[4];
            ldsm_x4(a, kst + unit_at<F, D>(rq, 2 * k + (mi >> 1)));
            if (k < kAcc)
                mma_16816_first(sa[k], a, qb[k][0], qb[k][1]);
            else
                mma_16816(sa[k % kAcc], a, qb[k][0], qb[k][1]);
        }
    } else {
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {  // 16-byte units 2k and 2k + 1
            uint32_t w[4], a[4], e[4];
            ldsm_x4(w, kst + unit_at<F, D>(rq, 2 * k + (mi >> 1)));
#pragma unroll
            for (int x = 0; x < 4; ++x) w[x] = unsign<F>(w[x]);
            to_halves<F>(w[0], a[0], a[2]);
            to_halves<F>(w[1], a[1], a[3]);
            to_halves<F>(w[2], e[0], e[2]);
            to_halves<F>(w[3], e[1], e[3]);
            if (2 * k < kAcc) {
                mma_16816_first(sa[2 * k], a, qb[2 * k][0], qb[2 * k][1]);
                mma_16816_first(sa[2 * k + 1], e, qb[2 * k + 1][0], qb[2 * k + 1][1]);
            } else {
                mma_16816(sa[2 * k % kAcc], a, qb[2 * k][0], qb[2 * k][1]);
                mma_16816(sa[(2 * k + 1) % kAcc], e, qb[2 * k + 1][0], qb[2 * k + 1][1]);
            }
        }
    }
    float s[4];  // tokens g (0, 1) and g + 8 (2, 3) of heads 2c, 2c + 1
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        float v = sa[0][x] + sa[1][x];
        if constexpr (kAcc == 4) v += sa[2][x] + sa[3][x];
        s[x] = v * ks;
    }
    if (score0) {
        const uint64_t keep = keep_in_l2();
        if (g < nvalid) {
            store_kept(score0 + g, s[0], keep);
            if (two) store_kept(score0 + score_stride + g, s[1], keep);
        }
        if (g + 8 < nvalid) {
            store_kept(score0 + g + 8, s[2], keep);
            if (two) store_kept(score0 + score_stride + g + 8, s[3], keep);
        }
    }
    if (g >= nvalid) s[0] = s[1] = -INFINITY;  // tokens past the end are excluded
    if (g + 8 >= nvalid) s[2] = s[3] = -INFINITY;

    float bm0 = fmaxf(s[0], s[2]), bm1 = fmaxf(s[1], s[3]);
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
        bm0 = fmaxf(bm0, __shfl_xor_sync(kFull, bm0, off));
        bm1 = fmaxf(bm1, __shfl_xor_sync(kFull, bm1, off));
    }
    const float mn0 = fmaxf(st.m0, bm0), mn1 = fmaxf(st.m1, bm1);
    // (scores of -infinity alone leave m there: 0 then stands in as the reference)
    const float r0 = mn0 == -INFINITY ? 0.f : mn0, r1 = mn1 == -INFINITY ? 0.f : mn1;
    float al0 = pow2_of(st.m0 - r0), al1 = pow2_of(st.m1 - r1);
    st.m0 = mn0;
    st.m1 = mn1;
    const float e0 = r0 - kShift, e1 = r1 - kShift;
    float p0 = pow2_of(s[0] - e0), p1 = pow2_of(s[1] - e1), p2 = pow2_of(s[2] - e0), p3 = pow2_of(s[3] - e1);
    st.l0 = st.l0 * al0 + (p0 + p2);
    st.l1 = st.l1 * al1 + (p1 + p3);
    bool small = false;  // V's scale is far below the unit
    float ratio = 1.f;
    if constexpr (F != PA_KV_F16) {
        if (vs > st.vr && vs >= 0x1p-100f) {  // (448 times less than that is zero in the output)
            const float down = st.vr * (1.f / vs);  // 0 for the first block
            al0 *= down;
            al1 *= down;
            st.vr = vs;
            st.rvr = 1.f / vs;
        }
        ratio = vs * st.rvr;
        small = ratio < 0x1p-20f;
        if (!small) p0 *= ratio, p1 *= ratio, p2 *= ratio, p3 *= ratio;
    }
    if (__any_sync(kFull, al0 != 1.f || al1 != 1.f)) {
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt) {
            st.o[mt][0] *= al0;
            st.o[mt][1] *= al1;
            st.o[mt][2] *= al0;
            st.o[mt][3] *= al1;
        }
    }
    const uint32_t pb0 = movmatrix_trans(half2_bits(__floats2half2_rn(p0, p1)));  // tokens 0..7
    const uint32_t pb1 = movmatrix_trans(half2_bits(__floats2half2_rn(p2, p3)));  // tokens 8..15

    if (nvalid < kBlockSize) {
        // 0 * NaN would poison P.V: clear the V rows past the end
        constexpr int kUnits = kRow / 16;
        for (int u = lane; u < (kBlockSize - nvalid) * kUnits; u += 32)
            *reinterpret_cast<uint4*>(vgen + unit_at<F, D>(nvalid + u / kUnits, u % kUnits)) =
                make_uint4(0u, 0u, 0u, 0u);
        __syncwarp();
    }

    // O^T += V^T . P^T
    if constexpr (F == PA_KV_F16) {
        const int rv = r8 + ((mi >> 1) << 3);
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt) {
            uint32_t a[4];
            ldsm_x4_trans(a, vst + unit_at<F, D>(rv, 2 * mt + (mi & 1)));
            mma_16816(st.o[mt], a, pb0, pb1);
        }
    } else {
        auto product = [&](auto add) {
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
                uint32_t w[4];
                ldsm_x4_trans(w, vst + unit_at<F, D>(rq, 2 * k + (mi >> 1)));
#pragma unroll
                for (int x = 0; x < 4; ++x) w[x] = unsign<F>(__byte_perm(w[x], 0u, 0x3120));
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    uint32_t a[4];
                    to_halves<F>(w[2 * y], a[0], a[1]);
                    to_halves<F>(w[2 * y + 1], a[2], a[3]);
                    add(st.o[2 * k + y], a);
                }
            }
        };
        if (!small) {
            product([&](float(&o)[4], const uint32_t(&a)[4]) { mma_16816(o, a, pb0, pb1); });
        } else {
            product([&](float(&o)[4], const uint32_t(&a)[4]) {
                float x[4];
                mma_16816_first(x, a, pb0, pb1);
#pragma unroll
                for (int i = 0; i < 4; ++i) o[i] = fmaf(ratio, x[i], o[i]);
            });
        }
    }
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// Cluster: the cluster form (of its own, so that the others keep their code: in
// one kernel 64 x 128 tokens of 8 x 128 took 8.2 instead of 7.4 us).
template <int F, int D, int NS, bool Cluster>
__global__ void __launch_bounds__(kKvWarps * 32, ctas_of<F, D>())
    kv_partition_kernel(const KvDecodeParams prm) {
    using S = KvShape<F, D, NS>;
    constexpr int NW = S::kNW;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float2 part_ml[kMaxGroup];  // cluster form: the CTA's (reference, sum) by head
    float* sm_m = reinterpret_cast<float*>(smem + S::kArea);
    float* sm_l = sm_m + NW * kMaxGroup;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t* const my_stages = smem + warp * NS * S::kStage;
    const uint32_t stage0 = smem_addr(my_stages);

    // While the preceding kernel ends: the lengths and the block tables on
    // their way to L2 (a hint; they are read after the wait).
    {
        const size_t cta = ((size_t)blockIdx.z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x;
        const size_t line = (cta * blockDim.x + threadIdx.x) * 128;
        const size_t lens = (size_t)prm.num_seqs * 4, tables = lens * prm.max_blocks_per_seq;
        if (line < tables) prefetch_l2(reinterpret_cast<const char*>(prm.block_tables) + line);
        if (line < lens) prefetch_l2(reinterpret_cast<const char*>(prm.seq_lens) + line);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");

    const int G = prm.group, H = prm.num_heads;
    const int g = lane >> 2, c = lane & 3;
    auto length = [&](int b) {  // tokens of sequence b: 0 if out of range
        const int L = __ldg(prm.seq_lens + b);
        return L > 0 && L <= prm.max_seq_len ? L : 0;
    };
    auto blocks = [&](int b) { return (length(b) + kBlockSize - 1) / kBlockSize; };

    // The warp's first segment: `cnt` blocks of sequence b from block j0 on,
    // `stride` apart.  whole: the CTA's warps share the segment and merge.
    int kvh, b, j0, cnt, stride, cta, nseq;
    int units = 0, end = 0, first = 0;  // flat, by warp: the run's end and sequence b's first unit
    bool whole = true;
    bool joint = false;  // the CTAs of the cluster merge
    int ids_early = -1;  // grid form: ids read before the length is known
    if (!Cluster && prm.flat) {
        kvh = blockIdx.x % prm.num_kv_heads;
        cta = blockIdx.x / prm.num_kv_heads;
        // lane i has sequences [i per, (i + 1) per)
        const int per = (prm.num_seqs + 31) / 32;
        const int i0 = min(prm.num_seqs, lane * per), i1 = min(prm.num_seqs, i0 + per);
        int mine = 0;
        for (int i = i0; i < i1; ++i) {
            const int n = blocks(i);
            mine += n ? n + kLead : 0;
        }
        int incl = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int up = __shfl_up_sync(kFull, incl, off);
            if (lane >= off) incl += up;
        }
        units = __shfl_sync(kFull, incl, 31);
        const FlatRuns runs(units, prm.ctas_per_head);
        if (cta >= runs.ctas) return;
        // the sequence that unit u belongs to, and its first unit
        auto locate = [&](int u, int& seq, int& at) {
            const int owner = __ffs(__ballot_sync(kFull, u >= incl - mine && u < incl)) - 1;
            seq = __shfl_sync(kFull, i0, owner);
            at = __shfl_sync(kFull, incl - mine, owner);
            for (;; ++seq) {
                const int n = blocks(seq);
                const int size = n ? n + kLead : 0;
                if (u < at + size) return n;
                at += size;
            }
        };
        const int u0 = runs.begin(cta), u1 = runs.begin(cta + 1);
        nseq = locate(u0, b, first);
        whole = u1 <= first + kLead + nseq;
        if (whole) {
            const int lo = max(0, u0 - first - kLead), hi = u1 - first - kLead;  // blocks of the run
            j0 = lo + warp;
            stride = NW;
            cnt = hi - lo > warp ? (hi - lo - warp + NW - 1) / NW : 0;
        } else {
            const int v0 = FlatRuns::warp_begin(u0, u1, warp);
            end = FlatRuns::warp_begin(u0, u1, warp + 1);
            if (v0 >= first + kLead + nseq) nseq = locate(v0, b, first);
            j0 = max(0, v0 - first - kLead);
            stride = 1;
            cnt = max(0, min(nseq, end - first - kLead) - j0);
        }
    } else {
        kvh = blockIdx.y;
        b = blockIdx.z;
        cta = blockIdx.x;
        // a partition's blocks are its own; the CTAs of a cluster take turns
        stride = Cluster ? NW * prm.cluster : NW;
        const int each = prm.partition_size / kBlockSize, lo = cta * (Cluster ? NW : each);
        j0 = lo + warp;
        // bounded by the table's row
        if ((Cluster || lane * NW + warp < each) && j0 + lane * stride < prm.max_blocks_per_seq)
            ids_early = __ldg(prm.block_tables + (size_t)b * prm.max_blocks_per_seq + j0 + lane * stride);
        nseq = blocks(b);
        if (nseq == 0 && cta == 0) {  // (there may be no merge to do this)
            if (__ldg(prm.seq_lens + b) != 0) {
                if (kvh == 0 && threadIdx.x == 0) atomicOr(prm.status, PA_DEV_BAD_SEQ_LEN);
            } else {
                for (int i = threadIdx.x; i < G * D; i += blockDim.x)
                    prm.out[((size_t)b * H + kvh * G) * D + i] = __float2half_rn(0.f);
            }
        }
        if (nseq == 0) return;
        joint = Cluster && prm.cluster > 1 && nseq > NW;  // else the first CTA has it all
        const int n = Cluster ? nseq - lo : min(nseq - lo, each);
        if (n <= 0 && !joint) return;
        cnt = n > warp ? (n - warp + stride - 1) / stride : 0;
    }

    // Ids and scales of the segment's iterations, 32 at a time: lane k of batch
    // n holds iteration 32 n + k.  The copies run up to NS iterations ahead, so
    // at most one batch: ids, ks_i and vs_i belong to the batch of the latest
    // copy, ks_c and vs_c to that of the block at hand.
    int ids = -1;
    float ks_i = 1.f, vs_i = 1.f, ks_c = 1.f, vs_c = 1.f;
    auto load_ids = [&](int seq, int j, bool in, int early) {
        ids = !in ? -1 : early >= 0 ? early : __ldg(prm.block_tables + (size_t)seq * prm.max_blocks_per_seq + j);
        if constexpr (F != PA_KV_F16) {
            const bool ok = ids >= 0 && (long long)ids < prm.num_blocks;
            const size_t at = ok ? (size_t)ids * prm.num_kv_heads + kvh : 0;
            ks_i = ok ? __ldg(prm.k_scales + at) : 0.f;
            vs_i = ok ? __ldg(prm.v_scales + at) : 0.f;
        }
    };
    uint32_t valid_bits = 0;  // stage s holds a block with a legal id
    // Start copying the block of the batch's lane k into the stage of the
    // warp's n-th block.  Every block's copies are one group, and after the
    // first NS of a segment one group (it may be empty) follows each block
    // consumed, so the block at hand is in all but the latest NS - 1.
    auto copy = [&](int n, int k) {
        const int phys = __shfl_sync(kFull, ids, k);
        const int s = n % NS;
        const bool ok = phys >= 0 && (long long)phys < prm.num_blocks;
        valid_bits = ok ? (valid_bits | (1u << s)) : (valid_bits & ~(1u << s));
        if (ok) {
            const size_t at = ((size_t)phys * prm.num_kv_heads + kvh) * S::kTile;
            copy_tile<F, D>(stage0 + s * S::kStage, prm.k_cache + at);
            copy_tile<F, D>(stage0 + s * S::kStage + S::kTile, prm.v_cache + at);
        } else if (lane == 0) {
            atomicOr(prm.status, PA_DEV_BAD_BLOCK_ID);
        }
    };

    int done = 0;    // blocks this warp has consumed in earlier segments
    int issued = 0;  // blocks of this segment that are on their way
    load_ids(b, j0 + lane * stride, lane < cnt, ids_early);
    for (int k = 0; k < NS; ++k) {
        if (k < cnt) copy(k, k), ++issued;
        copies_commit();
    }

    uint32_t qb[D / 16][2];
    WarpState<D> st;
    for (;;) {
        const int L = length(b);
        if (!Cluster && prm.flat && j0 == 0 && kvh == 0 && lane == 0 && cnt > 0) {
            // where the merge finds the sequence's partials
            const FlatRuns runs(units, prm.ctas_per_head);
            const SeqParts parts(runs, first, nseq, b);
            int4* to = reinterpret_cast<int4*>(prm.seq_parts) + 2 * (size_t)b;
            to[0] = make_int4(parts.first[0], parts.count[0], parts.first[1], parts.count[1]);
            to[1] = make_int4(parts.first[2], parts.count[2], 0, 0);
        }
        // Q as the B operand, its k index in K's order: for fp16 the lane holds
        // dims 16 i + 2c (+1) and + 8, in 8 bits dims 16 i + 4c .. + 3
        {
            const uint32_t* qrow =
                reinterpret_cast<const uint32_t*>(prm.q + ((size_t)b * H + kvh * G + (g < G ? g : 0)) * D);
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                const int lo = F == PA_KV_F16 ? 8 * i + c : 8 * i + 2 * c;
                const int hi = F == PA_KV_F16 ? lo + 4 : lo + 1;
                qb[i][0] = g < G ? __ldg(qrow + lo) : 0u;
                qb[i][1] = g < G ? __ldg(qrow + hi) : 0u;
            }
        }
        st.clear();
        float* scores = nullptr;  // of head 2c
        if (prm.scores && 2 * c < G) scores = prm.scores + ((size_t)b * H + kvh * G + 2 * c) * prm.score_stride;
        const bool two = 2 * c + 1 < G;

        // a warp's next segment (runs of their own): the next sequence with tokens
        int b_next = b, n_next = 0, first_next = first, cnt_next = 0;
        if (!Cluster && !whole && first + kLead + nseq < end) {
            first_next = first + kLead + nseq;
            do n_next = blocks(++b_next);
            while (n_next == 0);  // the run goes on, so there is one
            cnt_next = max(0, min(n_next, end - first_next - kLead));
        }
        int issued_next = 0;

        for (int i = 0; i < cnt; ++i) {
            const int s = (done + i) % NS;
            copies_wait<NS - 1>();
            __syncwarp();
            // copy i has been issued, and none of the next batch or sequence
            if ((i & 31) == 0) ks_c = ks_i, vs_c = vs_i;
            if ((valid_bits >> s) & 1u) {
                const int tok0 = (j0 + i * stride) * kBlockSize;
                const uint32_t kst = stage0 + s * S::kStage;
                const float ks = F == PA_KV_F16 ? prm.scale_log2 : prm.scale_log2 * __shfl_sync(kFull, ks_c, i & 31);
                const float vs = F == PA_KV_F16 ? 1.f : __shfl_sync(kFull, vs_c, i & 31);
                block_update<F, D>(st, qb, kst, kst + S::kTile, my_stages + s * S::kStage + S::kTile,
                                   min(kBlockSize, L - tok0), ks, vs, scores ? scores + tok0 : nullptr,
                                   prm.score_stride, two);
            } else if (scores) {  // a block that is not there gets no weight
                const int tok0 = (j0 + i * stride) * kBlockSize;
                for (int t = g; t < min(kBlockSize, L - tok0); t += 8) {
                    scores[tok0 + t] = -INFINITY;
                    if (two) scores[prm.score_stride + tok0 + t] = -INFINITY;
                }
            }
            __syncwarp();
            if (issued < cnt) {
                if ((issued & 31) == 0) {
                    const int it = issued + lane;
                    load_ids(b, j0 + it * stride, it < cnt, -1);
                }
                copy(done + issued, issued & 31);
                ++issued;
            } else if (issued_next < cnt_next && (i >> 5) == ((cnt - 1) >> 5)) {
                // (the last batch's scales have been taken over)
                if (issued_next == 0) load_ids(b_next, lane, lane < cnt_next, -1);
                copy(done + cnt + issued_next, issued_next);
                ++issued_next;
            }
            copies_commit();
        }
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
            st.l0 += __shfl_xor_sync(kFull, st.l0, off);
            st.l1 += __shfl_xor_sync(kFull, st.l1, off);
        }
        if (F == PA_KV_F16) st.vr = 1.f;
        if (Cluster || whole) break;

        // the segment's partial, or the output, straight from the fragments
        if (cnt > 0) {
            const bool direct = j0 == 0 && cnt == nseq;
            // (a partial without weight is 0, a whole sequence without any NaN)
            const float f0 = st.l0 == 0.f && !direct ? 0.f : st.vr / st.l0;
            const float f1 = st.l1 == 0.f && !direct ? 0.f : st.vr / st.l1;
            const size_t head0 = (size_t)b * H + kvh * G + 2 * c;
            const size_t slot = (size_t)(prm.ctas_per_head + cta * NW + warp + b);
            const size_t pi = ((size_t)kvh * prm.slots + slot) * G + 2 * c;
            const bool one = 2 * c < G;
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt) {
                const float v[4] = {st.o[mt][0] * f0, st.o[mt][1] * f1, st.o[mt][2] * f0, st.o[mt][3] * f1};
                const int d0 = out_dim<F>(mt, g, 0), d1 = out_dim<F>(mt, g, 1);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (!(h ? two : one)) continue;
                    if (direct) {
                        __half* o = prm.out + (head0 + h) * D;
                        if (F == PA_KV_F16) {
                            o[d0] = __float2half_rn(v[h]);
                            o[d1] = __float2half_rn(v[2 + h]);
                        } else {
                            *reinterpret_cast<__half2*>(o + d0) = __floats2half2_rn(v[h], v[2 + h]);
                        }
                    } else {
                        float* o = prm.acc + (pi + h) * D;
                        if (F == PA_KV_F16) {
                            o[d0] = v[h];
                            o[d1] = v[2 + h];
                        } else {
                            *reinterpret_cast<float2*>(o + d0) = make_float2(v[h], v[2 + h]);
                        }
                    }
                }
            }
            // the sum is relative to 2^(m - kShift)
            if (g == 0 && one) prm.sums[pi] = make_float2(st.m0 - kShift, st.l0);
            if (g == 0 && two) prm.sums[pi + 1] = make_float2(st.m1 - kShift, st.l1);
        }
        if (n_next == 0) return;
        done += cnt;
        b = b_next;
        nseq = n_next;
        first = first_next;
        j0 = 0;
        cnt = cnt_next;
        issued = issued_next;
        if (issued == 0) load_ids(b, lane, lane < cnt, -1);
        for (int k = issued_next; k < NS; ++k) {
            if (k < cnt) copy(done + k, k), ++issued;
            copies_commit();
        }
    }

    __syncthreads();  // all stages consumed; the area is reused below

    // Merge the warps' states: every warp leaves (m, l, O) in shared memory,
    // then warp w merges dims [w D/NW, (w+1) D/NW) of every head, the sums in
    // warp order.
    float* red = reinterpret_cast<float*>(smem);
    {
        float* rw = red + warp * kMaxGroup * S::kRedStride;
#pragma unroll
        for (int mt = 0; mt < S::kTilesM; ++mt) {
            const int d0 = out_dim<F>(mt, g, 0), d1 = out_dim<F>(mt, g, 1);
            rw[(2 * c) * S::kRedStride + d0] = st.o[mt][0] * st.vr;
            rw[(2 * c + 1) * S::kRedStride + d0] = st.o[mt][1] * st.vr;
            rw[(2 * c) * S::kRedStride + d1] = st.o[mt][2] * st.vr;
            rw[(2 * c + 1) * S::kRedStride + d1] = st.o[mt][3] * st.vr;
        }
        if (g == 0) {
            sm_m[warp * kMaxGroup + 2 * c] = st.m0;
            sm_m[warp * kMaxGroup + 2 * c + 1] = st.m1;
            sm_l[warp * kMaxGroup + 2 * c] = st.l0;
            sm_l[warp * kMaxGroup + 2 * c + 1] = st.l1;
        }
    }
    __syncthreads();
    constexpr int kSlice = D / NW;
    const int h = lane >> 2, qd = lane & 3;
    if (!Cluster && h >= G) return;
    float Mh = sm_m[h];
#pragma unroll
    for (int w = 1; w < NW; ++w) Mh = fmaxf(Mh, sm_m[w * kMaxGroup + h]);
    float f[NW], Lh = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {  // a warp without blocks has m = -inf and counts for nothing
        const float mw = sm_m[w * kMaxGroup + h];
        f[w] = mw == -INFINITY ? 0.f : exp2f(mw - Mh);
        Lh += f[w] * sm_l[w * kMaxGroup + h];
    }
    const size_t head = (size_t)b * H + kvh * G + h;
    const size_t slot = !Cluster && prm.flat ? (size_t)cta : (size_t)b * prm.max_partitions + cta;
    const size_t pi = ((size_t)kvh * prm.slots + slot) * G + h;
    // the CTA has the whole sequence: its run begins in or before block 0 and ends with the last
    const bool direct = !joint && j0 == warp &&
                        (!Cluster && prm.flat ? FlatRuns(units, prm.ctas_per_head).begin(cta + 1) == first + kLead + nseq
                                  : Cluster || prm.partition_size / kBlockSize >= nseq);
    const float inv = Lh == 0.f && !direct ? 0.f : 1.f / Lh;
#pragma unroll
    for (int w = 0; w < NW; ++w) f[w] *= inv;
#pragma unroll
    for (int k = 0; k < kSlice / 8; ++k) {
        const int d = warp * kSlice + 8 * k + 2 * qd;
        float v0 = 0.f, v1 = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float* rw = red + (w * kMaxGroup + h) * S::kRedStride + d;
            v0 += f[w] * rw[0];
            v1 += f[w] * rw[1];
        }
        if (joint)  // over the first warp's, which only this lane reads
            *reinterpret_cast<float2*>(red + h * S::kRedStride + d) = make_float2(v0, v1);
        else if (direct && h < G)
            *reinterpret_cast<__half2*>(prm.out + head * D + d) = __floats2half2_rn(v0, v1);
        else if (!Cluster)
            *reinterpret_cast<float2*>(prm.acc + pi * D + d) = make_float2(v0, v1);
    }
    // the sum is relative to 2^(M - kShift): log2 of the whole is its reference plus log2 l
    if constexpr (!Cluster) {
        if (warp == 0 && qd == 0 && prm.sums) prm.sums[pi] = make_float2(Mh - kShift, Lh);
        return;
    }
    if (warp == 0 && qd == 0) part_ml[h] = make_float2(Mh, Lh);
    if (joint) {
        // The cluster's CTAs merge over distributed shared memory, each a share of
        // the G D / 4 columns of four, all reads of a column on their way at once.
        cg::cluster_group cluster = cg::this_cluster();
        cluster.sync();
        const int CS = prm.cluster;
        auto weights_of = [&](int head_, float (&w)[kKvMaxCluster]) {  // 2^(M_r - M) l_r of the CTAs; their sum's log2
            float2 ml[kKvMaxCluster];
            float M = -INFINITY, l = 0.f;
#pragma unroll
            for (int r = 0; r < kKvMaxCluster; ++r)
                ml[r] = r < CS ? *cluster.map_shared_rank(part_ml + head_, r) : make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int r = 0; r < kKvMaxCluster; ++r) M = fmaxf(M, ml[r].x);
#pragma unroll
            for (int r = 0; r < kKvMaxCluster; ++r) {
                w[r] = ml[r].x == -INFINITY ? 0.f : exp2f(ml[r].x - M) * ml[r].y;
                l += w[r];
            }
            return make_float2(M, l);
        };
        const int share = (G * (D / 4) + CS - 1) / CS;
        const int end_col = min(G * (D / 4), (cta + 1) * share);
        for (int col = cta * share + (int)threadIdx.x; col < end_col; col += NW * 32) {
            const int hh = col / (D / 4), d = col % (D / 4) * 4;
            float4 v[kKvMaxCluster];
            float w[kKvMaxCluster];
#pragma unroll
            for (int r = 0; r < kKvMaxCluster; ++r)
                v[r] = r < CS ? *reinterpret_cast<const float4*>(cluster.map_shared_rank(red + hh * S::kRedStride + d, r))
                              : make_float4(0.f, 0.f, 0.f, 0.f);
            const float inv_l = 1.f / weights_of(hh, w).y;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int r = 0; r < kKvMaxCluster; ++r) {
                a.x += w[r] * v[r].x;
                a.y += w[r] * v[r].y;
                a.z += w[r] * v[r].z;
                a.w += w[r] * v[r].w;
            }
            const __half2 o2[2] = {__floats2half2_rn(a.x * inv_l, a.y * inv_l),
                                   __floats2half2_rn(a.z * inv_l, a.w * inv_l)};
            *reinterpret_cast<uint2*>(prm.out + ((size_t)b * H + kvh * G + hh) * D + d) =
                *reinterpret_cast<const uint2*>(o2);
        }
        if (prm.weights_out && threadIdx.x < G) {
            float w[kKvMaxCluster];
            const float2 ml = weights_of(threadIdx.x, w);
            sm_m[threadIdx.x] = ml.x - kShift + log2f(ml.y);
        }
        cluster.sync();  // no CTA leaves while another may still read from it
    } else {
        __syncthreads();
        if (threadIdx.x < G) sm_m[threadIdx.x] = part_ml[threadIdx.x].x - kShift + log2f(part_ml[threadIdx.x].y);
        __syncthreads();
    }
    if (!prm.weights_out) return;
    // the weights of the warp's own tokens, from the scores that it left
    const size_t row = ((size_t)b * prm.num_kv_heads + kvh) * prm.weights_stride;
    const float* sc = prm.scores + ((size_t)b * H + kvh * G) * prm.score_stride;
    const int L = length(b);
    constexpr int kAtOnce = 2;  // pairs of blocks whose loads are in flight together
    for (int i = lane >> 4; i < cnt; i += 2 * kAtOnce) {
        float s[kAtOnce][kMaxGroup], w[kAtOnce];
        int tok[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const int t = (j0 + (i + 2 * k) * stride) * kBlockSize + (lane & 15);
            const bool in = i + 2 * k < cnt && t < L;
            tok[k] = in ? t : -1;
            w[k] = in && prm.weights_in ? prm.weights_in[row + t] : 0.f;
#pragma unroll
            for (int x = 0; x < kMaxGroup; ++x) s[k][x] = in && x < G ? sc[x * prm.score_stride + t] : 0.f;
        }
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            float sum = 0.f;
#pragma unroll
            for (int x = 0; x < kMaxGroup; ++x)
                if (x < G) sum += pow2_of(s[k][x] - sm_m[x]);
            if (tok[k] >= 0) prm.weights_out[row + tok[k]] = w[k] + sum;
        }
    }
}

// Blocks x < slices of a (sequence, kv head): `cols` float4 columns of the
// merge of its partials each; the rest: kKvWeightsTokens tokens of the weights
// each.  Both are chains of a few loads; each link loads all it can at once.
constexpr int kMergeThreads = 256;
constexpr int kPerThread = kKvWeightsTokens / kMergeThreads;

// Exponent reference, sum and weighted columns of some partials; empty: m = -inf.
struct MergeState {
    float m = -INFINITY, l = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    // with a partial's normalised columns t (beta: its weight) or another state's (beta: 2^(m - m'))
    __device__ __forceinline__ void add(float mo, float lo, const float4& t, float scale) {
        const float mn = fmaxf(m, mo);
        const float alpha = m == -INFINITY ? 0.f : exp2f(m - mn), f = mo == -INFINITY ? 0.f : exp2f(mo - mn);
        const float beta = f * scale;
        l = l * alpha + lo * f;
        a.x = a.x * alpha + beta * t.x;
        a.y = a.y * alpha + beta * t.y;
        a.z = a.z * alpha + beta * t.z;
        a.w = a.w * alpha + beta * t.w;
        m = mn;
    }
};

// GW: a bound on the heads of a kv head, for the weights' registers.
template <int D, int GW>
__global__ void __launch_bounds__(kMergeThreads, 4) kv_merge_kernel(const KvMergeParams prm) {
    __shared__ float4 red[kMergeThreads];
    __shared__ float2 red_ml[kMergeThreads];
    __shared__ float lse[kMaxGroup];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int kvh = blockIdx.y, b = blockIdx.z, G = prm.group;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int L = __ldg(prm.seq_lens + b);
    // Partial p of the sequence is slot at(p).  seq_parts is not written for an
    // empty sequence (and then not used).
    int n, n0 = 0, n1 = 0;
    long long s0 = 0, s1 = 0, s2 = 0;
    if (prm.flat) {
        const int4* parts = reinterpret_cast<const int4*>(prm.seq_parts) + 2 * (size_t)b;
        const int4 u = parts[0], v = parts[1];
        const long long most = prm.slots;
        auto clamp = [&](long long x, long long lo, long long hi) { return min(max(x, lo), hi); };
        n0 = (int)clamp(u.y, 0, kKvWarps);
        n1 = (int)clamp(u.w, 0, most);
        n = n0 + n1 + (int)clamp(v.y, 0, kKvWarps);
        s0 = clamp(u.x, 0, most - n0);
        s1 = clamp(u.z, 0, most - n1) - n0;
        s2 = clamp(v.x, 0, most - (n - n0 - n1)) - n0 - n1;
    } else {
        n = (L + prm.partition_size - 1) / prm.partition_size;
        n0 = n;
        s0 = (long long)b * prm.max_partitions;
    }
    const bool merge = (int)blockIdx.x < prm.slices;
    if (L < 0 || L > prm.max_seq_len) {
        if (blockIdx.x == 0 && kvh == 0 && tid == 0) atomicOr(prm.status, PA_DEV_BAD_SEQ_LEN);
        return;
    }
    const size_t head_slots = (size_t)(kvh * prm.slots);
    auto at = [&](int p) { return head_slots + (size_t)(p + (p < n0 ? s0 : p < n0 + n1 ? s1 : s2)); };
    constexpr int kAtOnce = 3;  // partials of a thread in flight
    if (merge) {
        // column `col` of the G D / 4, by `groups` groups of threads that take
        // every groups-th partial; cols is a power of two
        const int cols = prm.cols, groups = kMergeThreads / cols;
        const int col = blockIdx.x * cols + (tid & (cols - 1)), grp = tid / cols;
        const bool in = col < G * (D / 4);
        __half* out = prm.out + ((size_t)b * prm.num_heads + (size_t)kvh * G) * D;
        if (L == 0) {  // no tokens: zero
            if (grp == 0 && in) *reinterpret_cast<uint2*>(out + 4 * col) = make_uint2(0u, 0u);
            return;
        }
        if (n <= 1) return;  // written by the partition kernel
        const int h = in ? col / (D / 4) : 0;
        MergeState st;
        const float4* acc = reinterpret_cast<const float4*>(prm.acc) + (in ? col : 0);
        for (int p = grp; p < n; p += kAtOnce * groups) {
            float2 ml[kAtOnce];
            float4 t[kAtOnce];
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const int q = p + k * groups;
                ml[k] = make_float2(-INFINITY, 0.f);
                t[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (q < n) {
                    const size_t row = at(q) * G;
                    ml[k] = prm.sums[row + h];
                    t[k] = acc[row * (D / 4)];
                }
            }
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) st.add(ml[k].x, ml[k].y, t[k], ml[k].y);
        }
        // the groups of a warp, then the warps
        for (int off = cols; off < 32; off <<= 1) {
            const float mo = __shfl_xor_sync(kFull, st.m, off), lo = __shfl_xor_sync(kFull, st.l, off);
            const float4 t = make_float4(__shfl_xor_sync(kFull, st.a.x, off), __shfl_xor_sync(kFull, st.a.y, off),
                                         __shfl_xor_sync(kFull, st.a.z, off), __shfl_xor_sync(kFull, st.a.w, off));
            st.add(mo, lo, t, 1.f);
        }
        red[tid] = st.a;
        red_ml[tid] = make_float2(st.m, st.l);
        __syncthreads();
        if (grp == 0 && in) {
            const int step = max(cols, 32);  // the first group of every warp (or every group)
            for (int q = tid + step; q < kMergeThreads; q += step) st.add(red_ml[q].x, red_ml[q].y, red[q], 1.f);
            const float inv = 1.f / st.l;
            const __half2 v[2] = {__floats2half2_rn(st.a.x * inv, st.a.y * inv),
                                  __floats2half2_rn(st.a.z * inv, st.a.w * inv)};
            *reinterpret_cast<uint2*>(out + 4 * col) = *reinterpret_cast<const uint2*>(v);
        }
        return;
    }
    const int t0 = ((int)blockIdx.x - prm.slices) * kKvWeightsTokens + tid;
    if (t0 - tid >= L) return;
    // the tokens' scores and old weights are on their way while the sums are added up
    const float* sc = prm.scores + ((size_t)b * prm.num_heads + (size_t)kvh * G) * prm.score_stride + t0;
    const size_t row = ((size_t)b * prm.num_kv_heads + kvh) * prm.weights_stride + t0;
    float s[kPerThread][GW], w[kPerThread];
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
        const bool in = t0 + k * kMergeThreads < L;
        w[k] = in && prm.weights_in ? prm.weights_in[row + k * kMergeThreads] : 0.f;
        const float* from = sc + k * kMergeThreads;
#pragma unroll
        for (int h = 0; h < GW; ++h, from += prm.score_stride) s[k][h] = h < G && in ? *from : -INFINITY;
    }
    if (warp < G) {  // 8 warps, at most 8 heads
        MergeState st;
        const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int p = lane; p < n; p += 32 * kAtOnce) {
            float2 ml[kAtOnce];
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k)
                ml[k] = p + 32 * k < n ? prm.sums[at(p + 32 * k) * G + warp] : make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) st.add(ml[k].x, ml[k].y, none, 0.f);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            st.add(__shfl_xor_sync(kFull, st.m, off), __shfl_xor_sync(kFull, st.l, off), none, 0.f);
        if (lane == 0) lse[warp] = st.m + log2f(st.l);
    }
    __syncthreads();
    float by[GW];
#pragma unroll
    for (int h = 0; h < GW; ++h) by[h] = h < G ? lse[h] : 0.f;  // (absent heads: 2^-inf = 0)
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
        float sum = 0.f;
#pragma unroll
        for (int h = 0; h < GW; ++h) sum += pow2_of(s[k][h] - by[h]);
        if (t0 + k * kMergeThreads < L) prm.weights_out[row + k * kMergeThreads] = w[k] + sum;
    }
}

template <int F, int D, bool Cluster>
cudaError_t launch_fd(const KvDecodeParams& prm, dim3 grid, cudaStream_t stream) {
    constexpr int NS = stages_of<F, D>();
    using S = KvShape<F, D, NS>;
    static_assert(ctas_of<F, D>() * (S::kSmem + 1024 + 64) <= 228 * 1024, "shared memory of an SM");
    static std::atomic<unsigned long long> done{0};
    auto kern = kv_partition_kernel<F, D, NS, Cluster>;
    cudaError_t e = once_per_device(done, [&] {
        cudaError_t r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
        return r != cudaSuccess ? r : cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kKvWarps * 32);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2] = {pdl_attribute(), {}};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (prm.cluster > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = prm.cluster;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    return cudaLaunchKernelEx(&cfg, kern, prm);
}

}  // namespace

#define PA_KV_FOR_FD(X)                                                                                    \
    X(PA_KV_F16, 64) X(PA_KV_F16, 128) X(PA_KV_F16, 256) X(PA_KV_E4M3, 64) X(PA_KV_E4M3, 128)              \
    X(PA_KV_E4M3, 256) X(PA_KV_INT8, 64) X(PA_KV_INT8, 128) X(PA_KV_INT8, 256)

int kv_decode_ctas(int format, int head_dim) {
#define PA_CASE(F_, D_) \
    if (format == F_ && head_dim == D_) return ctas_of<F_, D_>();
    PA_KV_FOR_FD(PA_CASE)
#undef PA_CASE
    return -1;
}

cudaError_t launch_kv_decode(int format, int head_dim, const KvDecodeParams& prm, dim3 grid, cudaStream_t stream) {
#define PA_CASE(F_, D_) \
    if (format == F_ && head_dim == D_) \
        return prm.cluster ? launch_fd<F_, D_, true>(prm, grid, stream) : launch_fd<F_, D_, false>(prm, grid, stream);
    PA_KV_FOR_FD(PA_CASE)
#undef PA_CASE
    return cudaErrorInvalidValue;
}

// The merge asks for the decode kernel's division of an SM's memory although
// it needs little shared memory itself: while an SM is divided otherwise, fewer
// of the next decode's CTAs fit on it, and the rest would run as a second wave.
template <int D, int GW>
cudaError_t launch_merge_dg(const cudaLaunchConfig_t& cfg, const KvMergeParams& prm) {
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = once_per_device(done, [&] {
        return cudaFuncSetAttribute(kv_merge_kernel<D, GW>, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    });
    return e != cudaSuccess ? e : cudaLaunchKernelEx(&cfg, kv_merge_kernel<D, GW>, prm);
}

template <int D>
cudaError_t launch_merge_d(const cudaLaunchConfig_t& cfg, const KvMergeParams& prm) {
    if (prm.group == 1) return launch_merge_dg<D, 1>(cfg, prm);
    if (prm.group == 2) return launch_merge_dg<D, 2>(cfg, prm);
    if (prm.group <= 4) return launch_merge_dg<D, 4>(cfg, prm);
    return launch_merge_dg<D, 8>(cfg, prm);
}

cudaError_t launch_kv_merge(int head_dim, const KvMergeParams& prm, dim3 grid, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kMergeThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr = pdl_attribute();
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    switch (head_dim) {
        case 64: return launch_merge_d<64>(cfg, prm);
        case 128: return launch_merge_d<128>(cfg, prm);
        case 256: return launch_merge_d<256>(cfg, prm);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace pa
