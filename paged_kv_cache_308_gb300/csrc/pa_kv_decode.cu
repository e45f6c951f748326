// Decode attention over a cache in 8 bits (or fp16), and the accumulation of
// its attention weights.
//
// kv_partition_kernel<F, D, NS>: one CTA per (partition, kv head, sequence),
// the decomposition of pa_partition_kernel, over cache format F.  The math
// per 16-token block, for the <= 8 query heads of a kv head (log2 domain,
// c = scale * log2 e):
//     s[t, h] = c ks sum_d k8[t, d] q[h, d]             ks, vs: the block's scales
//     m'      = max(m, max_t s),  p = 2^(s - m' + kShift)
//     l       = l 2^(m - m') + sum_t p
//     o[d, h] = o 2^(m - m') + vs sum_t v8[t, d] p16[t, h]
// The scales stay outside the products, so K and V enter the tensor cores as
// exact halves (a code is at most 448) and a block's scale costs one multiply
// per score and one FMA per output instead of one per element.
// p is rounded to fp16 for the product (relative 2^-11; the shift keeps
// probabilities down to 2^-28 of the maximum normal and 2^-38 above zero);
// l adds the unrounded p, in 32 bits as m and o are, so that the weights of
// the accumulation are exact to 32-bit rounding.
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
// once, C per kv head.  The blocks of the batch's sequences form one list of
// T; CTA c takes blocks [f(c), f(c+1)), f(c) = floor(c T / C'), so every CTA
// reads the same amount whatever the lengths, and no CTA is launched for a
// partition that its sequence does not have.  A share that crosses sequences
// is processed sequence by sequence; each gives one partial (or, if it holds
// the whole sequence, the output).  Partial slots are c + b, b the sequence:
// along the list either c or b grows from one segment to the next, so slots
// never collide and C + B of them suffice.  Every CTA derives its share from
// seq_lens itself; the host never reads them.  Grid form (a partition size
// was given, or every sequence fits one CTA): one CTA per (partition, kv
// head, sequence).
//
// kv_merge_kernel: the log-sum-exp merge of the partials, and in further CTAs
// of the same launch weights_out = weights_in + sum_h 2^(s - lse) from the
// scores that the partition kernel left: 4 bytes per (token, head) written
// and read again, instead of K's D bytes a second time.
#include "pa_kv.h"

#include <cuda_fp8.h>
#include <math.h>

#include "pa_decode.h"
#include "pa_device.cuh"

namespace pa {
namespace {

constexpr float kShift = 14.f;
constexpr int kMinBlocks = kKvWarps;  // blocks of a share at least, while there are enough

template <int F, int D, int NS>
struct KvShape {
    static constexpr int kNW = kKvWarps;
    static constexpr int kElem = F == PA_KV_F16 ? 2 : 1;
    static constexpr int kRow = D * kElem;                       // bytes of a token's row
    static constexpr int kChunk = kRow < 128 ? kRow : 128;       // bytes of a row in one swizzled box
    static constexpr int kTile = kBlockSize * kRow;              // K (or V) of a block
    static constexpr int kStage = 2 * kTile;
    static constexpr int kStageArea = kNW * NS * kStage;
    static constexpr int kTilesM = D / 16;                       // m-tiles of P.V
    static constexpr int kRedStride = D + 4;
    static constexpr int kRedBytes = kNW * kMaxGroup * kRedStride * 4;
    static constexpr int kArea = kStageArea > kRedBytes ? kStageArea : kRedBytes;
    // barriers, (m, l) of the warps, abort flag
    static constexpr int kCtrl = kNW * NS * 8 + 2 * kNW * kMaxGroup * 4 + 16;
    static constexpr int kSmem = 1024 + kArea + kCtrl;
    static_assert(kSmem <= 227 * 1024, "shared memory budget of one CTA");
};

// Byte offset of 16-byte unit `unit` of row `row` in a staged tile.
template <int F, int D>
__device__ __forceinline__ uint32_t unit_at(int row, int unit) {
    if constexpr (F != PA_KV_F16 && D == 64)  // 64-byte rows, 64-byte swizzle
        return static_cast<uint32_t>(row * 64 + ((unit ^ ((row >> 1) & 3)) << 4));
    else
        return static_cast<uint32_t>((unit >> 3) * (kBlockSize * 128)) + swz(row, unit & 7);
}

__device__ __forceinline__ uint32_t cvt_e4m3x2(uint32_t two) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo;\n\tcvt.u16.u32 lo, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(two));
    return r;
}

// Two halves from bytes `sel` (a byte-permute selector of two bytes) of w.
template <int F>
__device__ __forceinline__ uint32_t halves_lo(uint32_t w) {  // bytes 0, 1
    if constexpr (F == PA_KV_E4M3) {
        return cvt_e4m3x2(w);
    } else {
        const uint32_t u = __byte_perm(w, 0x64646464u, 0x4140);
        const __half2 k = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152
        return half2_bits(__hsub2(*reinterpret_cast<const __half2*>(&u), k));
    }
}

template <int F>
__device__ __forceinline__ uint32_t halves_hi(uint32_t w) {  // bytes 2, 3
    if constexpr (F == PA_KV_E4M3) {
        return cvt_e4m3x2(w >> 16);
    } else {
        const uint32_t u = __byte_perm(w, 0x64646464u, 0x4342);
        const __half2 k = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
        return half2_bits(__hsub2(*reinterpret_cast<const __half2*>(&u), k));
    }
}

template <int F>
__device__ __forceinline__ uint32_t unsign(uint32_t w) {  // int8: bytes v + 128
    return F == PA_KV_INT8 ? w ^ 0x80808080u : w;
}

// (d of o[mt][0..1], d of o[mt][2..3]) of a lane with row group g.
template <int F>
__device__ __forceinline__ int out_dim(int mt, int g, int hi) {
    return F == PA_KV_F16 ? 16 * mt + g + 8 * hi : 16 * mt + 2 * g + hi;
}

// Stages per warp, and the CTAs an SM holds: 96 to 192 KB of copies in flight
// per SM, within its registers (an accumulator of 4 D / 16 and D / 8 of Q a
// thread) and 228 KB of shared memory.
template <int F, int D>
constexpr int stages_of() {
    return F == PA_KV_F16 ? (D == 256 ? 2 : D == 128 ? 3 : 4) : (D == 256 ? 3 : 4);
}
template <int F, int D>
constexpr int ctas_of() {
    return F == PA_KV_F16 ? (D == 256 ? 1 : D == 128 ? 2 : 3) : (D == 256 ? 2 : D == 128 ? 3 : 5);
}

template <int F, int D, int NS>
__global__ void __launch_bounds__(kKvWarps * 32, ctas_of<F, D>())
    kv_partition_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                        const KvDecodeParams prm) {
    using S = KvShape<F, D, NS>;
    constexpr int NW = S::kNW;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kArea);
    float* sm_m = reinterpret_cast<float*>(bars + NW * NS);
    float* sm_l = sm_m + NW * kMaxGroup;
    int* sm_abort = reinterpret_cast<int*>(sm_l + NW * kMaxGroup);
    __shared__ int sm_sum[NW], sm_start[2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t stage0 = smem_addr(smem) + warp * NS * S::kStage;
    const uint32_t bar0 = smem_addr(bars) + warp * NS * 8;

    if (threadIdx.x == 0) {
        *sm_abort = 0;
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_k)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_v)) : "memory");
    }
    if (lane == 0) {
        for (int s = 0; s < NS; ++s) mbar_init(bar0 + 8 * s, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");

    const int G = prm.group, H = prm.num_heads;
    const int g = lane >> 2, c = lane & 3;
    const int mi = lane >> 3, r8 = lane & 7;
    auto length = [&](int b) {  // tokens of sequence b: 0 if out of range
        const int L = __ldg(prm.seq_lens + b);
        return L > 0 && L <= prm.max_seq_len ? L : 0;
    };

    // The share [x, x1) of the list of blocks, from block `first` (list index)
    // of sequence b on; the list's T blocks are dealt to `ctas` CTAs, q each and
    // one more to the first r.
    int kvh, b, cta, x, x1, first, q = 0, r = 0;
    int ids_early = -1;  // grid form: ids read before the length is known
    if (prm.flat) {
        kvh = blockIdx.x % prm.num_kv_heads;
        cta = blockIdx.x / prm.num_kv_heads;
        // thread i sums the blocks of sequences [i per, (i + 1) per)
        const int per = (prm.num_seqs + NW * 32 - 1) / (NW * 32);
        const int i0 = threadIdx.x * per, i1 = min(prm.num_seqs, i0 + per);
        int mine = 0;
        for (int i = i0; i < i1; ++i) mine += (length(i) + kBlockSize - 1) / kBlockSize;
        int incl = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int up = __shfl_up_sync(kFull, incl, off);
            if (lane >= off) incl += up;
        }
        if (lane == 31) sm_sum[warp] = incl;
        __syncthreads();
        int T = 0;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            if (w < warp) incl += sm_sum[w];
            T += sm_sum[w];
        }
        const int ctas = min(prm.ctas_per_head, max(1, T / kMinBlocks));
        if (cta >= ctas || T == 0) return;
        q = T / ctas;
        r = T - q * ctas;
        x = cta * q + min(cta, r);
        x1 = x + q + (cta < r ? 1 : 0);
        if (x >= incl - mine && x < incl) {  // the thread whose sequences hold block x
            int at = incl - mine, i = i0;
            for (;; ++i) {
                const int n = (length(i) + kBlockSize - 1) / kBlockSize;
                if (x < at + n) break;
                at += n;
            }
            sm_start[0] = i;
            sm_start[1] = at;
        }
        __syncthreads();
        b = sm_start[0];
        first = sm_start[1];
    } else {
        kvh = blockIdx.y;
        b = blockIdx.z;
        cta = blockIdx.x;
        const int each = prm.partition_size / kBlockSize;
        first = 0;
        x = cta * each;
        const int j = warp + lane * NW;  // bounded by the table's row
        if (j < each && x + j < prm.max_blocks_per_seq)
            ids_early = __ldg(prm.block_tables + (size_t)b * prm.max_blocks_per_seq + x + j);
        const int n = (length(b) + kBlockSize - 1) / kBlockSize;
        if (n == 0 && cta == 0) {  // (there may be no merge to do this)
            if (__ldg(prm.seq_lens + b) != 0) {
                if (kvh == 0 && threadIdx.x == 0) atomicOr(prm.status, PA_DEV_BAD_SEQ_LEN);
            } else {
                for (int i = threadIdx.x; i < G * D; i += blockDim.x)
                    prm.out[((size_t)b * H + kvh * G) * D + i] = __float2half_rn(0.f);
            }
        }
        x1 = min(n, x + each);
        if (x >= x1) return;
    }

    // score rows, Q and the state are per sequence; the copy ring runs through
    int done = 0;  // blocks this warp has consumed in earlier segments
    for (;;) {
    const int L = length(b);
    const int nseq = (L + kBlockSize - 1) / kBlockSize;
    const int blk0 = x - first;
    const int nblk = min(x1, first + nseq) - x;
    const bool direct = blk0 == 0 && nblk == nseq;
    const size_t slot = prm.flat ? (size_t)(cta + b) : (size_t)b * prm.max_partitions + cta;
    if (prm.flat && blk0 == 0 && kvh == 0 && threadIdx.x == 0) {
        const int z = first + nseq - 1;  // the sequence's last block, and the CTA that has it
        const int last = z < r * (q + 1) ? z / (q + 1) : r + (z - r * (q + 1)) / q;
        prm.seq_parts[2 * b] = cta + b;
        prm.seq_parts[2 * b + 1] = last - cta + 1;
    }
    const int32_t* bt = prm.block_tables + (size_t)b * prm.max_blocks_per_seq + blk0;
    const int nmine = warp < nblk ? (nblk - warp + NW - 1) / NW : 0;

    // Ids and scales of this warp's iterations, 32 at a time: lane k of batch
    // n holds iteration 32 n + k, block warp + it * NW of the segment.  The
    // copies run up to NS iterations ahead, so at most one batch: ids, ks_i and
    // vs_i belong to the batch of the latest copy, ks_c and vs_c to that of the
    // block at hand.
    int ids = -1;
    float ks_i = 1.f, vs_i = 1.f, ks_c = 1.f, vs_c = 1.f;
    auto load_ids = [&](int j, int early) {
        ids = j < nblk ? (early >= 0 ? early : __ldg(bt + j)) : -1;
        if constexpr (F != PA_KV_F16) {
            const bool ok = ids >= 0 && (long long)ids < prm.num_blocks;
            const size_t at = ok ? (size_t)ids * prm.num_kv_heads + kvh : 0;
            ks_i = ok ? __ldg(prm.k_scales + at) : 0.f;
            vs_i = ok ? __ldg(prm.v_scales + at) : 0.f;
        }
    };
    load_ids(warp + lane * NW, ids_early);
    int batch = 0;
    uint32_t valid_bits = 0;  // stage s holds a block with a legal id
    auto issue = [&](int it) {
        if ((it >> 5) != batch) {
            batch = it >> 5;
            load_ids(warp + ((it & ~31) + lane) * NW, -1);
        }
        const int phys = __shfl_sync(kFull, ids, it & 31);
        const int s = (done + it) % NS;
        const uint32_t bar = bar0 + 8 * s;
        const bool ok = phys >= 0 && (long long)phys < prm.num_blocks;
        valid_bits = ok ? (valid_bits | (1u << s)) : (valid_bits & ~(1u << s));
        if (lane == 0) {
            if (ok) {
                mbar_arrive_expect_tx(bar, S::kStage);
                const int row = (phys * prm.num_kv_heads + kvh) * kBlockSize;
                const uint32_t kdst = stage0 + s * S::kStage;
                tma_load_3d(kdst, &tmap_k, 0, row, 0, bar);
                tma_load_3d(kdst + S::kTile, &tmap_v, 0, row, 0, bar);
            } else {
                atomicOr(prm.status, PA_DEV_BAD_BLOCK_ID);
                mbar_arrive(bar);  // complete the phase so the wait below stays in step
            }
        }
    };
    for (int it = 0; it < NS && it < nmine; ++it) issue(it);

    // Q as the B operand, its k index in K's order: for fp16 the lane holds
    // dims 16 i + 2c (+1) and + 8, in 8 bits dims 16 i' + 4c .. + 3, i' = the
    // i-th 16-byte unit of the row.
    uint32_t qb[D / 16][2];
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

    float o[S::kTilesM][4];
#pragma unroll
    for (int i = 0; i < S::kTilesM; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY;  // running maximum of heads 2c, 2c + 1
    float l0 = 0.f, l1 = 0.f;              // this lane's share of the exp sums
    // score rows of heads 2c and 2c + 1
    float* score0 = nullptr;
    if (prm.scores && 2 * c < G) score0 = prm.scores + ((size_t)b * H + kvh * G + 2 * c) * prm.score_stride;

    bool timed_out = false;
    int i = 0;
    for (; i < nmine; ++i) {
        const int s = (done + i) % NS;
        if (prm.force_timeout || !mbar_wait(bar0 + 8 * s, ((done + i) / NS) & 1, prm.wait_limit)) {
            timed_out = true;
            break;
        }
        if ((i & 31) == 0) ks_c = ks_i, vs_c = vs_i;  // copy i, and none of the next batch, has been issued
        if ((valid_bits >> s) & 1u) {
            const int tok0 = (blk0 + warp + i * NW) * kBlockSize;
            const int nvalid = min(kBlockSize, L - tok0);
            const uint32_t kst = stage0 + s * S::kStage, vst = kst + S::kTile;
            const float ks = F == PA_KV_F16 ? prm.scale_log2 : prm.scale_log2 * __shfl_sync(kFull, ks_c, i & 31);
            const float vs = F == PA_KV_F16 ? 1.f : __shfl_sync(kFull, vs_c, i & 31);

            // S^T = K . Q^T
            float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
            if constexpr (F == PA_KV_F16) {
                const int rq = r8 + ((mi & 1) << 3);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    uint32_t a[4];
                    ldsm_x4(a, kst + unit_at<F, D>(rq, 2 * k + (mi >> 1)));
                    if (k & 1)
                        mma_16816(sb, a, qb[k][0], qb[k][1]);
                    else
                        mma_16816(sa, a, qb[k][0], qb[k][1]);
                }
            } else {
                const int rq = r8 + ((mi & 1) << 3);
#pragma unroll
                for (int k = 0; k < D / 32; ++k) {  // two 16-byte units: units 2k and 2k + 1
                    uint32_t w[4];
                    ldsm_x4(w, kst + unit_at<F, D>(rq, 2 * k + (mi >> 1)));
#pragma unroll
                    for (int x = 0; x < 4; ++x) w[x] = unsign<F>(w[x]);
                    const uint32_t a[4] = {halves_lo<F>(w[0]), halves_lo<F>(w[1]), halves_hi<F>(w[0]),
                                           halves_hi<F>(w[1])};
                    mma_16816(sa, a, qb[2 * k][0], qb[2 * k][1]);
                    const uint32_t e[4] = {halves_lo<F>(w[2]), halves_lo<F>(w[3]), halves_hi<F>(w[2]),
                                           halves_hi<F>(w[3])};
                    mma_16816(sb, e, qb[2 * k + 1][0], qb[2 * k + 1][1]);
                }
            }
            // lane holds tokens g (s0, s1) and g + 8 (s2, s3) of heads 2c, 2c + 1
            float s0 = (sa[0] + sb[0]) * ks, s1 = (sa[1] + sb[1]) * ks;
            float s2 = (sa[2] + sb[2]) * ks, s3 = (sa[3] + sb[3]) * ks;
            if (score0) {
                float* r0 = score0 + tok0 + g;
                float* r1 = r0 + prm.score_stride;
                const bool two = 2 * c + 1 < G;
                if (g < nvalid) {
                    r0[0] = s0;
                    if (two) r1[0] = s1;
                }
                if (g + 8 < nvalid) {
                    r0[8] = s2;
                    if (two) r1[8] = s3;
                }
            }
            if (g >= nvalid) s0 = s1 = -INFINITY;  // tokens past the end are excluded
            if (g + 8 >= nvalid) s2 = s3 = -INFINITY;

            float bm0 = fmaxf(s0, s2), bm1 = fmaxf(s1, s3);
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
                bm0 = fmaxf(bm0, __shfl_xor_sync(kFull, bm0, off));
                bm1 = fmaxf(bm1, __shfl_xor_sync(kFull, bm1, off));
            }
            const float mn0 = fmaxf(m0, bm0), mn1 = fmaxf(m1, bm1);
            const float al0 = exp2f(m0 - mn0), al1 = exp2f(m1 - mn1);
            m0 = mn0;
            m1 = mn1;
            const float e0 = mn0 - kShift, e1 = mn1 - kShift;
            const float p0 = exp2f(s0 - e0), p1 = exp2f(s1 - e1), p2 = exp2f(s2 - e0), p3 = exp2f(s3 - e1);
            l0 = l0 * al0 + (p0 + p2);
            l1 = l1 * al1 + (p1 + p3);
            if (__any_sync(kFull, al0 != 1.f || al1 != 1.f)) {
#pragma unroll
                for (int mt = 0; mt < S::kTilesM; ++mt) {
                    o[mt][0] *= al0;
                    o[mt][1] *= al1;
                    o[mt][2] *= al0;
                    o[mt][3] *= al1;
                }
            }
            const uint32_t pb0 = movmatrix_trans(half2_bits(__floats2half2_rn(p0, p1)));  // tokens 0..7
            const uint32_t pb1 = movmatrix_trans(half2_bits(__floats2half2_rn(p2, p3)));  // tokens 8..15

            if (nvalid < kBlockSize) {
                // 0 * NaN would poison P.V: clear the V rows past the end
                constexpr int kUnits = S::kRow / 16;
                for (int u = lane; u < (kBlockSize - nvalid) * kUnits; u += 32) {
                    const uint32_t at = unit_at<F, D>(nvalid + u / kUnits, u % kUnits);
                    *reinterpret_cast<uint4*>(smem + (vst - smem_addr(smem)) + at) = make_uint4(0u, 0u, 0u, 0u);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
            }

            // O^T += V^T . P^T
            if constexpr (F == PA_KV_F16) {
                const int rv = r8 + ((mi >> 1) << 3);
#pragma unroll
                for (int mt = 0; mt < S::kTilesM; ++mt) {
                    uint32_t a[4];
                    ldsm_x4_trans(a, vst + unit_at<F, D>(rv, 2 * mt + (mi & 1)));
                    mma_16816(o[mt], a, pb0, pb1);
                }
            } else {
                const int rv = r8 + ((mi & 1) << 3);
#pragma unroll
                for (int k = 0; k < D / 32; ++k) {
                    uint32_t w[4];
                    ldsm_x4_trans(w, vst + unit_at<F, D>(rv, 2 * k + (mi >> 1)));
#pragma unroll
                    for (int x = 0; x < 4; ++x) w[x] = unsign<F>(__byte_perm(w[x], 0u, 0x3120));
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const uint32_t a[4] = {halves_lo<F>(w[2 * y]), halves_hi<F>(w[2 * y]),
                                               halves_lo<F>(w[2 * y + 1]), halves_hi<F>(w[2 * y + 1])};
                        float t[4] = {0.f, 0.f, 0.f, 0.f};
                        mma_16816(t, a, pb0, pb1);
#pragma unroll
                        for (int x = 0; x < 4; ++x) o[2 * k + y][x] = fmaf(vs, t[x], o[2 * k + y][x]);
                    }
                }
            }
        }
        __syncwarp();
        if (i + NS < nmine) issue(i + NS);
    }

    if (timed_out) {
        // wait for this warp's copies still in flight before the CTA may exit
        const int issued = min(nmine, i + NS);
        for (int k = done + i; k < done + issued; ++k)
            mbar_wait(bar0 + 8 * (k % NS), (k / NS) & 1, kDefaultWaitLimit);
        if (lane == 0) {
            atomicOr(prm.status, PA_DEV_TIMEOUT);
            atomicExch(sm_abort, 1);
        }
    }
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
        l0 += __shfl_xor_sync(kFull, l0, off);
        l1 += __shfl_xor_sync(kFull, l1, off);
    }
    __syncthreads();  // all stages consumed; the area is reused below
    if (*sm_abort) return;

    // Merge the warps' states: every warp leaves (m, l, O) in shared memory,
    // then warp w merges dims [w D/NW, (w+1) D/NW) of every head, the sums in
    // warp order.
    float* red = reinterpret_cast<float*>(smem);
    {
        float* rw = red + warp * kMaxGroup * S::kRedStride;
#pragma unroll
        for (int mt = 0; mt < S::kTilesM; ++mt) {
            const int d0 = out_dim<F>(mt, g, 0), d1 = out_dim<F>(mt, g, 1);
            rw[(2 * c) * S::kRedStride + d0] = o[mt][0];
            rw[(2 * c + 1) * S::kRedStride + d0] = o[mt][1];
            rw[(2 * c) * S::kRedStride + d1] = o[mt][2];
            rw[(2 * c + 1) * S::kRedStride + d1] = o[mt][3];
        }
        if (g == 0) {
            sm_m[warp * kMaxGroup + 2 * c] = m0;
            sm_m[warp * kMaxGroup + 2 * c + 1] = m1;
            sm_l[warp * kMaxGroup + 2 * c] = l0;
            sm_l[warp * kMaxGroup + 2 * c + 1] = l1;
        }
    }
    __syncthreads();
    constexpr int kSlice = D / NW;
    const int h = lane >> 2, qd = lane & 3;
    if (h < G) {
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
        const float inv = 1.f / Lh;
        const size_t head = (size_t)b * H + kvh * G + h;
        const size_t pi = ((size_t)kvh * prm.slots + slot) * G + h;
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
            if (direct)
                *reinterpret_cast<__half2*>(prm.out + head * D + d) = __floats2half2_rn(v0, v1);
            else
                *reinterpret_cast<float2*>(prm.acc + pi * D + d) = make_float2(v0, v1);
        }
        // the sum is relative to 2^(M - kShift): log2 of the whole is its reference plus log2 l
        if (warp == 0 && qd == 0 && prm.sums) prm.sums[pi] = make_float2(Mh - kShift, Lh);
    }
    // on to the next sequence of the share
    x += nblk;
    if (x >= x1) return;
    first += nseq;
    do ++b;
    while (length(b) == 0);  // x < x1 <= T: there is one
    done += nmine;
    ids_early = -1;
    // the next copies overwrite what the merge wrote and read through the generic proxy
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
    }
}

// Blocks x < slices of a (sequence, kv head): slice x of the merge of its
// partials; the rest: kWeightsTokens tokens of the weights each.
constexpr int kMergeThreads = 256;
constexpr int kPerThread = kKvWeightsTokens / kMergeThreads;

template <int D>
__global__ void __launch_bounds__(kMergeThreads) kv_merge_kernel(const KvMergeParams prm) {
    __shared__ float4 red[kMergeThreads];
    __shared__ float2 red_ml[kMergeThreads];
    __shared__ float lse[kMaxGroup];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int kvh = blockIdx.y, b = blockIdx.z, G = prm.group;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int L = __ldg(prm.seq_lens + b);
    long long slot0;
    int n;
    if (prm.flat) {
        // not written for an empty sequence (and then not used) nor after a
        // timeout: the clamps keep the reads inside the workspace
        slot0 = min(max((long long)prm.seq_parts[2 * b], 0ll), prm.slots - 1);
        n = (int)min(max((long long)prm.seq_parts[2 * b + 1], 1ll), prm.slots - slot0);
    } else {
        slot0 = (long long)b * prm.max_partitions;
        n = (L + prm.partition_size - 1) / prm.partition_size;
    }
    const bool merge = (int)blockIdx.x < prm.slices;
    if (L < 0 || L > prm.max_seq_len) {
        if (blockIdx.x == 0 && kvh == 0 && tid == 0) atomicOr(prm.status, PA_DEV_BAD_SEQ_LEN);
        return;
    }
    const size_t p0 = (size_t)(kvh * prm.slots + slot0);
    const float2* sums = prm.sums + p0 * G;
    if (merge) {
        // float4 column `col` of the G D outputs, by `groups` groups of threads
        // that take every groups-th partial
        const int cols = G * (D / 4) / prm.slices;
        const int groups = kMergeThreads / cols;
        const int col = blockIdx.x * cols + tid % cols, grp = tid / cols;
        __half* out = prm.out + ((size_t)b * prm.num_heads + (size_t)kvh * G) * D;
        if (L == 0) {  // no tokens: zero
            if (grp == 0) *reinterpret_cast<uint2*>(out + 4 * col) = make_uint2(0u, 0u);
            return;
        }
        if (n <= 1) return;  // written by the partition kernel
        const int h = col / (D / 4);
        float m = -INFINITY, l = 0.f;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        if (grp < groups) {
            const float4* acc = reinterpret_cast<const float4*>(prm.acc + p0 * G * D) + col;
#pragma unroll 4
            for (int p = grp; p < n; p += groups) {
                const float2 ml = sums[(size_t)p * G + h];
                const float4 t = acc[(size_t)p * G * (D / 4)];
                const float mn = fmaxf(m, ml.x);
                const float alpha = exp2f(m - mn), beta = ml.y * exp2f(ml.x - mn);
                l = l * alpha + beta;
                a.x = a.x * alpha + beta * t.x;
                a.y = a.y * alpha + beta * t.y;
                a.z = a.z * alpha + beta * t.z;
                a.w = a.w * alpha + beta * t.w;
                m = mn;
            }
        }
        red[tid] = a;
        red_ml[tid] = make_float2(m, l);
        __syncthreads();
        if (grp == 0) {
            float M = m;
            for (int q = 1; q < groups; ++q) M = fmaxf(M, red_ml[q * cols + tid].x);
            float w = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int q = 0; q < groups; ++q) {
                const float2 ml = red_ml[q * cols + tid];
                const float f = ml.x == -INFINITY ? 0.f : exp2f(ml.x - M);  // a group without partials
                const float4 t = red[q * cols + tid];
                w += f * ml.y;
                o.x += f * t.x;
                o.y += f * t.y;
                o.z += f * t.z;
                o.w += f * t.w;
            }
            const float inv = 1.f / w;
            const __half2 v[2] = {__floats2half2_rn(o.x * inv, o.y * inv), __floats2half2_rn(o.z * inv, o.w * inv)};
            *reinterpret_cast<uint2*>(out + 4 * col) = *reinterpret_cast<const uint2*>(v);
        }
        return;
    }
    const int t0 = ((int)blockIdx.x - prm.slices) * kKvWeightsTokens + tid;
    if (t0 - tid >= L) return;
    // the tokens' scores and old weights are on their way while the sums are added up
    const size_t head0 = (size_t)b * prm.num_heads + (size_t)kvh * G;
    const size_t row = ((size_t)b * prm.num_kv_heads + kvh) * prm.weights_stride;
    float s[kPerThread][kMaxGroup], w[kPerThread];
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
        const int t = t0 + k * kMergeThreads;
        w[k] = t < L && prm.weights_in ? prm.weights_in[row + t] : 0.f;
#pragma unroll
        for (int h = 0; h < kMaxGroup; ++h)
            s[k][h] = h < G && t < L ? prm.scores[(head0 + h) * prm.score_stride + t] : -INFINITY;
    }
    if (warp < G) {  // 8 warps, at most 8 heads
        float m = -INFINITY, l = 0.f;
        for (int p = lane; p < n; p += 32) {
            const float2 ml = sums[(size_t)p * G + warp];
            const float mn = fmaxf(m, ml.x);
            l = l * exp2f(m - mn) + ml.y * exp2f(ml.x - mn);
            m = mn;
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            const float mo = __shfl_xor_sync(kFull, m, off), lo = __shfl_xor_sync(kFull, l, off);
            const float mn = fmaxf(m, mo);
            l = (m == -INFINITY ? 0.f : l * exp2f(m - mn)) + (mo == -INFINITY ? 0.f : lo * exp2f(mo - mn));
            m = mn;
        }
        if (lane == 0) lse[warp] = m + log2f(l);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
        const int t = t0 + k * kMergeThreads;
        if (t >= L) break;
        float sum = 0.f;
#pragma unroll
        for (int h = 0; h < kMaxGroup; ++h)
            if (h < G) sum += exp2f(s[k][h] - lse[h]);
        prm.weights_out[row + t] = w[k] + sum;
    }
}

template <int F, int D>
cudaError_t launch_fd(const KvDecodeParams& prm, const CUtensorMap& tk, const CUtensorMap& tv, dim3 grid,
                      cudaStream_t stream) {
    constexpr int NS = stages_of<F, D>();
    using S = KvShape<F, D, NS>;
    static_assert(ctas_of<F, D>() * (S::kSmem + 1024 + 64) <= 228 * 1024, "shared memory of an SM");
    static std::atomic<unsigned long long> done{0};
    auto kern = kv_partition_kernel<F, D, NS>;
    cudaError_t e = once_per_device(
        done, [&] { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem); });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kKvWarps * 32);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr = pdl_attribute();
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, tk, tv, prm);
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

cudaError_t launch_kv_decode(int format, int head_dim, const KvDecodeParams& prm, const CUtensorMap& tk,
                             const CUtensorMap& tv, dim3 grid, cudaStream_t stream) {
#define PA_CASE(F_, D_) \
    if (format == F_ && head_dim == D_) return launch_fd<F_, D_>(prm, tk, tv, grid, stream);
    PA_KV_FOR_FD(PA_CASE)
#undef PA_CASE
    return cudaErrorInvalidValue;
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
        case 64: return cudaLaunchKernelEx(&cfg, kv_merge_kernel<64>, prm);
        case 128: return cudaLaunchKernelEx(&cfg, kv_merge_kernel<128>, prm);
        case 256: return cudaLaunchKernelEx(&cfg, kv_merge_kernel<256>, prm);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace pa
