// Linear attention with a decay a kv head, token by token: the state in
// registers, from the pool and back (pa_linear_decode; pa_linear_prefix for few
// new tokens).
#include "pa_decode.h"

#include "pa_device.cuh"
#include "pa_step.h"

namespace pa {

namespace {

constexpr int kThreads = 256;

template <int D>
struct Slice {
    static constexpr int kCols = D == 256 ? 32 : 64;      // of the state's columns (of V), of a block: 32 KB (16 at D = 64)
    static constexpr int kLanes = kCols / 4;              // threads of a row
    static constexpr int kRows = kThreads / kLanes;       // rows at a time
    static constexpr int kPasses = D / kRows;
};

// What a state is multiplied by for one token: S -> S * whole + S * rest, where
// exp(g) - 1 in 32 bits has what exp(g) loses next to 1.
struct Decay {
    float whole, rest;
};
__device__ __forceinline__ Decay decay_of(float g) {
    if (g > -0.5f) return {1.f, expm1f(g)};
    return {0.f, expf(g)};
}

// A block takes kCols columns of a (sequence, kv head)'s state through all of its
// tokens; each thread holds kPasses rows of four columns.  A token's products with
// q are summed over the block's rows by shuffles and in shared memory.
template <int D, int G>
__global__ void __launch_bounds__(kThreads) linear_recurrent_kernel(const LinearParams prm) {
    using S = Slice<D>;
    __shared__ float ks[D];
    __shared__ float qs[G][D];
    __shared__ float red[kThreads / 32][G][S::kCols];
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int kvh = blockIdx.y, b = blockIdx.z, c0 = blockIdx.x * S::kCols + (t % S::kLanes) * 4, r0 = t / S::kLanes;
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
    if (first == last) return;
    const float g = __ldg(prm.log_decay + kvh);
    if (!(g <= 0.f) && t == 0 && blockIdx.x == 0) atomicOr(prm.status, PA_DEV_BAD_DECAY);
    const Decay dec = decay_of(g);

    float4* state = reinterpret_cast<float4*>(prm.states + (((size_t)slot * prm.num_kv_heads + kvh) * D + r0) * D + c0);
    float4 s[S::kPasses];
#pragma unroll
    for (int i = 0; i < S::kPasses; ++i)
        s[i] = fresh ? make_float4(0.f, 0.f, 0.f, 0.f) : __ldcs(state + (size_t)i * S::kRows * D / 4);

    for (int row = first; row < last; ++row) {
        const __half* k = prm.k + ((size_t)row * prm.num_kv_heads + kvh) * D;
        const __half* q = prm.q + ((size_t)row * prm.num_heads + kvh * prm.group) * D;
        const uint2 vr = __ldg(reinterpret_cast<const uint2*>(prm.v + ((size_t)row * prm.num_kv_heads + kvh) * D + c0));
        for (int i = t; i < D; i += kThreads) ks[i] = __half2float(k[i]);
        for (int i = t; i < G * D; i += kThreads) qs[i / D][i % D] = i < prm.group * D ? __half2float(q[i]) : 0.f;
        const float2 v01 = __half22float2(*reinterpret_cast<const __half2*>(&vr.x));
        const float2 v23 = __half22float2(*reinterpret_cast<const __half2*>(&vr.y));
        __syncthreads();
        float4 acc[G];
#pragma unroll
        for (int h = 0; h < G; ++h) acc[h] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < S::kPasses; ++i) {
            const float kk = ks[r0 + i * S::kRows];
            auto step = [&](float x, float v) { return fmaf(kk, v, fmaf(x, dec.rest, x * dec.whole)); };
            s[i] = make_float4(step(s[i].x, v01.x), step(s[i].y, v01.y), step(s[i].z, v23.x), step(s[i].w, v23.y));
#pragma unroll
            for (int h = 0; h < G; ++h) {
                const float qq = qs[h][r0 + i * S::kRows];
                acc[h].x = fmaf(qq, s[i].x, acc[h].x);
                acc[h].y = fmaf(qq, s[i].y, acc[h].y);
                acc[h].z = fmaf(qq, s[i].z, acc[h].z);
                acc[h].w = fmaf(qq, s[i].w, acc[h].w);
            }
        }
#pragma unroll
        for (int h = 0; h < G; ++h) {
#pragma unroll
            for (int d = S::kLanes; d < 32; d *= 2) {
                acc[h].x += __shfl_xor_sync(kFull, acc[h].x, d);
                acc[h].y += __shfl_xor_sync(kFull, acc[h].y, d);
                acc[h].z += __shfl_xor_sync(kFull, acc[h].z, d);
                acc[h].w += __shfl_xor_sync(kFull, acc[h].w, d);
            }
            if (lane < S::kLanes) *reinterpret_cast<float4*>(&red[warp][h][lane * 4]) = acc[h];
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
    for (int i = 0; i < S::kPasses; ++i) __stcs(state + (size_t)i * S::kRows * D / 4, s[i]);
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
