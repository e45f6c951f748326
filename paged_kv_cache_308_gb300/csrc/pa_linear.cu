// Linear attention with a decay a kv head, token by token: the state in
// registers, from the pool and back (pa_linear_decode; pa_linear_prefix for few
// new tokens).
#include "pa_decode.h"

#include "pa_device.cuh"
#include "pa_linear.cuh"
#include "pa_step.h"

namespace pa {

namespace {

constexpr int kThreads = 256;

template <int D>
struct Slice {
    // of the state's columns (of V), of a block: 32 KB (16 at D = 64).  64 at D = 256 take 44.7 us for 64 sequences
    // of 24/4 heads, 32 take 30.6; 32 at D = 128 take 51.4 for 256 sequences of 32/8 heads, 64 take 45.4
    static constexpr int kCols = D == 256 ? 32 : 64;
    static constexpr int kLanes = kCols / 4;              // threads of a row
    static constexpr int kRows = kThreads / kLanes;       // rows at a time
    static constexpr int kPasses = D / kRows;
};

// Two 32-bit numbers a register pair, for the instructions that take two at a time.
typedef unsigned long long Two;
__device__ __forceinline__ Two two(float a, float b) {
    Two r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 parts(Two x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ Two mul2(Two a, Two b) {
    Two r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
    Two r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// Blocks an SM that the registers are shared out for: half a state a block at head_dim 64, a quarter and an eighth
// above (512 sequences of 24/4 x 64: 16.0 us with four, 14.8 with five; 256 of 32/8 x 128: 46.8 / 50.8, and 48.8
// with three).  More than four query heads are summed in two halves: six at once leave room for three blocks or spill
// (128 sequences of 24/4 x 256 57.0 us, in halves 52.9; 256 of 64/8 x 128 61.4 / 58.2).
template <int D>
constexpr int kBlocksPerSm = D == 64 ? 5 : 4;

// For each token S <- d S + k v^T and out = scale q S.  A block takes kCols columns of a
// (sequence, kv head)'s state through all of its tokens; each thread holds kPasses rows, next to
// each other, of four columns, so that the state is read and written once however many tokens
// there are.  A token's products with q are summed over the block's rows by shuffles and in
// shared memory.  One token a sequence is bound by the state's traffic, 8 D^2 bytes a kv head:
// 256 sequences of 32/8 x 128 (268 MB of states there and back) 46 us, 87 % of the measured
// bandwidth; 64 of 24/4 x 256 (134 MB) 29 us, 68 %, where the products with six heads are not all
// covered (23 us with one head; without the hint that states are not read again 41 us); a
// single sequence 4.2 us, a launch and two trips to memory.
// More tokens cost about 1.2 us each, the chain through shared memory.
template <int D, int G>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm<D>) linear_recurrent_kernel(const LinearParams prm) {
    using S = Slice<D>;
    constexpr int kHeads = G > 4 ? G / 2 : G;  // whose sums are in registers at a time
    __shared__ __align__(16) float ks[D];
    __shared__ __align__(16) float qs[G][D];
    __shared__ __align__(16) float red[kThreads / 32][G][S::kCols];
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int kvh = blockIdx.y, b = blockIdx.z;
    const int c0 = blockIdx.x * S::kCols + (t % S::kLanes) * 4, r0 = t / S::kLanes * S::kPasses;  // column, first row
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int slot = __ldg(prm.slots + b);
    if (slot < 0) return;
    if (slot >= prm.num_slots) {
        if (t == 0 && kvh == 0 && blockIdx.x == 0) atomicOr(prm.status, PA_DEV_BAD_BLOCK_ID);
        return;
    }
    int first = b, last = b + 1;
    bool fresh = false;
    if (prm.query_start_loc) {
        first = __ldg(prm.query_start_loc + b);
        last = __ldg(prm.query_start_loc + b + 1);
        const int context = __ldg(prm.context_lens + b);
        if (first < 0 || last < first || last > prm.num_tokens || last - first > prm.max_query_len || context < 0) {
            if (t == 0 && kvh == 0 && blockIdx.x == 0) atomicOr(prm.status, PA_DEV_BAD_SEQ_LEN);
            return;
        }
        fresh = context == 0;
    }
    if (first == last || (prm.few > 0 && last - first > prm.few)) return;
    const float g = __ldg(prm.log_decay + kvh);
    if (!(g <= 0.f) && t == 0 && blockIdx.x == 0) atomicOr(prm.status, PA_DEV_BAD_DECAY);
    const Decay dec = decay_of(g);

    ulonglong2* state = reinterpret_cast<ulonglong2*>(prm.states + (((size_t)slot * prm.num_kv_heads + kvh) * D + r0) * D + c0);
    ulonglong2 s[S::kPasses];
#pragma unroll
    for (int i = 0; i < S::kPasses; ++i) s[i] = fresh ? make_ulonglong2(0, 0) : __ldcs(state + i * D / 4);
    const Two whole = two(dec.whole, dec.whole), rest = two(dec.rest, dec.rest);

    for (int row = first; row < last; ++row) {
        const __half* k = prm.k + ((size_t)row * prm.num_kv_heads + kvh) * D;
        const __half* q = prm.q + ((size_t)row * prm.num_heads + kvh * prm.group) * D;
        const uint2 vr = __ldg(reinterpret_cast<const uint2*>(prm.v + ((size_t)row * prm.num_kv_heads + kvh) * D + c0));
        for (int i = t; i < D; i += kThreads) ks[i] = __half2float(k[i]);
        for (int i = t; i < G * D; i += kThreads) qs[i / D][i % D] = i < prm.group * D ? __half2float(q[i]) : 0.f;
        const float2 v01 = __half22float2(*reinterpret_cast<const __half2*>(&vr.x));
        const float2 v23 = __half22float2(*reinterpret_cast<const __half2*>(&vr.y));
        const Two va = two(v01.x, v01.y), vb = two(v23.x, v23.y);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < S::kPasses; i += 4) {
            const float4 k4 = *reinterpret_cast<const float4*>(ks + r0 + i);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float kk = j == 0 ? k4.x : j == 1 ? k4.y : j == 2 ? k4.z : k4.w;
                ulonglong2& x = s[i + j];
                x.x = fma2(two(kk, kk), va, fma2(x.x, whole, mul2(x.x, rest)));
                x.y = fma2(two(kk, kk), vb, fma2(x.y, whole, mul2(x.y, rest)));
            }
        }
#pragma unroll
        for (int h0 = 0; h0 < G; h0 += kHeads) {
            Two sum[kHeads][2];
#pragma unroll
            for (int h = 0; h < kHeads; ++h) sum[h][0] = sum[h][1] = 0;
#pragma unroll
            for (int i = 0; i < S::kPasses; i += 4) {
#pragma unroll
                for (int h = 0; h < kHeads; ++h) {
                    const float4 q4 = *reinterpret_cast<const float4*>(&qs[h0 + h][r0 + i]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float qq = j == 0 ? q4.x : j == 1 ? q4.y : j == 2 ? q4.z : q4.w;
                        sum[h][0] = fma2(two(qq, qq), s[i + j].x, sum[h][0]);
                        sum[h][1] = fma2(two(qq, qq), s[i + j].y, sum[h][1]);
                    }
                }
            }
            // each lane of a column's four (at head_dim 256, else two) ends with a share of the columns
#pragma unroll
            for (int h = 0; h < kHeads; ++h) {
                const bool upper = lane & S::kLanes;
                const float2 mine = parts(upper ? sum[h][1] : sum[h][0]), other = parts(upper ? sum[h][0] : sum[h][1]);
                float2 o = make_float2(mine.x + __shfl_xor_sync(kFull, other.x, S::kLanes),
                                       mine.y + __shfl_xor_sync(kFull, other.y, S::kLanes));
                float* at = &red[warp][h0 + h][lane % S::kLanes * 4 + (upper ? 2 : 0)];
                if (S::kLanes == 8) {
                    const bool odd = lane & 16;
                    const float x = (odd ? o.y : o.x) + __shfl_xor_sync(kFull, odd ? o.x : o.y, 16);
                    at[odd] = x;
                } else {
                    *reinterpret_cast<float2*>(at) = o;
                }
            }
        }
        __syncthreads();
        for (int i = t; i < prm.group * S::kCols; i += kThreads) {
            const int h = i / S::kCols, c = i % S::kCols;
            float o = 0.f;
#pragma unroll
            for (int w = 0; w < kThreads / 32; ++w) o += red[w][h][c];
            prm.out[((size_t)row * prm.num_heads + kvh * prm.group + h) * D + blockIdx.x * S::kCols + c] =
                __float2half_rn(o * prm.scale);
        }
    }
#pragma unroll
    for (int i = 0; i < S::kPasses; ++i) __stcs(state + i * D / 4, s[i]);
}

template <int D, int G>
cudaError_t launch(const LinearParams& prm, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(D / Slice<D>::kCols, prm.num_kv_heads, prm.num_seqs);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, linear_recurrent_kernel<D, G>, prm);
}

template <int D>
cudaError_t by_group(const LinearParams& prm, cudaStream_t stream) {
    if (prm.group == 1) return launch<D, 1>(prm, stream);
    if (prm.group == 2) return launch<D, 2>(prm, stream);
    if (prm.group <= 4) return launch<D, 4>(prm, stream);
    if (prm.group <= 6) return launch<D, 6>(prm, stream);
    return launch<D, 8>(prm, stream);
}

}  // namespace

cudaError_t launch_linear_recurrent(int head_dim, const LinearParams& prm, cudaStream_t stream) {
    switch (head_dim) {
        case 64: return by_group<64>(prm, stream);
        case 128: return by_group<128>(prm, stream);
        case 256: return by_group<256>(prm, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace pa
