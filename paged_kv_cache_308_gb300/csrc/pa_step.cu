// Kernels of a serving step around the cache: block tables and slot maps from
// request lengths (pa_kv_alloc), the rotary embedding with the write into the
// cache (pa_kv_put).
#include "pa_step.h"

#include <cooperative_groups.h>

#include "pa_decode.h"

#include "pa_device.cuh"

namespace pa {

namespace {

constexpr int kWarps = kAllocThreads / 32;

// Counts that are summed over the sequences, in 64 bits: lengths of a batch may
// add up to more than an int even where each is in range.
struct Sums {
    long long query, back, need;  // new tokens, blocks given back, blocks wanted
};

__device__ __forceinline__ Sums plus(Sums a, Sums b) { return {a.query + b.query, a.back + b.back, a.need + b.need}; }

__device__ __forceinline__ Sums shfl_up(Sums v, int d) {
    return {__shfl_up_sync(kFull, v.query, d), __shfl_up_sync(kFull, v.back, d), __shfl_up_sync(kFull, v.need, d)};
}

// Exclusive sums over the block's threads, and the total.
__device__ Sums block_scan(Sums v, Sums* sm, Sums& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Sums inc = v;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const Sums o = shfl_up(inc, d);
        if (lane >= d) inc = plus(inc, o);
    }
    if (lane == 31) sm[warp] = inc;
    __syncthreads();
    Sums before{0, 0, 0};
    total = before;
    for (int w = 0; w < kWarps; ++w) {
        if (w == warp) before = total;
        total = plus(total, sm[w]);
    }
    return {before.query + inc.query - v.query, before.back + inc.back - v.back, before.need + inc.need - v.need};
}

// A sequence's lengths; blocks held and wanted are equal where they are bad.
struct Seq {
    int context, query, n0, n1;
    bool bad;
};

__device__ __forceinline__ Seq seq_of(const KvAllocParams& prm, int b) {
    Seq s;
    s.context = __ldg(prm.context + b);
    s.query = __ldg(prm.query + b);
    const int held = __ldg(prm.held + b);
    const long long room = min((long long)prm.cols * kBlockSize, 1ll << 30);
    s.bad = s.context < 0 || s.query < 0 || held < s.context || held > room || (long long)s.context + s.query > room;
    s.n0 = s.bad ? 0 : (held + kBlockSize - 1) / kBlockSize;
    s.n1 = s.bad ? 0 : (s.context + s.query + kBlockSize - 1) / kBlockSize;
    return s;
}

__device__ __forceinline__ Sums sums_of(const Seq& s) {
    return {max(s.query, 0), max(s.n0 - s.n1, 0), max(s.n1 - s.n0, 0)};
}

// One cluster does everything: its blocks meet at the cluster's barrier, which
// needs no counter in memory that two calls could share.  Every block sums over
// all sequences (a thread over consecutive ones), keeps the running sums of its
// own share of them in shared memory, and its warps then move their blocks; the
// tokens are dealt to the threads of the whole cluster, each of which finds its
// sequence by bisection.
__global__ void __launch_bounds__(kAllocThreads) kv_alloc_kernel(const KvAllocParams prm) {
    namespace cg = cooperative_groups;
    extern __shared__ int2 offsets[];  // of the own sequences: blocks given back and wanted before them
    __shared__ Sums sm[kWarps];
    __shared__ unsigned long long taken_sm;
    const cg::cluster_group cluster = cg::this_cluster();
    const int rank = cluster.block_rank(), ctas = cluster.num_blocks();
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31, B = prm.num_seqs;
    if (t == 0) taken_sm = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");

    const int share = (B + ctas - 1) / ctas, b0 = min(B, rank * share), b1 = min(B, b0 + share);
    const int each = (B + kAllocThreads - 1) / kAllocThreads;
    const int s0 = min(B, t * each), s1 = min(B, s0 + each);
    const int count = __ldg(prm.count);
    Sums mine{0, 0, 0}, total;
    bool bad = false;
    for (int b = s0; b < s1; ++b) {
        const Seq s = seq_of(prm, b);
        bad |= s.bad;
        mine = plus(mine, sums_of(s));
    }
    Sums at = block_scan(mine, sm, total);
    const bool bad_pool = count < 0 || count > prm.num_blocks || count + total.back > prm.num_blocks;
    const long long top = bad_pool ? 0 : count + total.back;
    unsigned status = bad || total.query > prm.num_tokens ? PA_DEV_BAD_SEQ_LEN : 0;
    if (bad_pool) status |= PA_DEV_NO_BLOCKS;
    long long taken = 0;
    for (int b = s0; b < s1; ++b) {
        const Seq s = seq_of(prm, b);
        const Sums one = sums_of(s);
        const bool served = one.need == 0 || (!bad_pool && at.need + one.need <= top);
        if (served)
            taken = max(taken, one.need ? at.need + one.need : 0);
        else
            status |= PA_DEV_NO_BLOCKS;
        if (b >= b0 && b < b1) {
            // (both below 2^31 where they are used: the stack has no more blocks)
            offsets[b - b0] = make_int2((int)min(at.back, 1ll << 30), served ? (int)min(at.need, 1ll << 30) : -1);
            prm.lens[b] = s.bad ? 0 : served ? s.context + s.query : s.context;
            prm.loc[b] = (int)min(at.query, (long long)prm.num_tokens);
        }
        at = plus(at, one);
    }
    if (taken) atomicMax(&taken_sm, (unsigned long long)taken);
    if (status && rank == 0) atomicOr(prm.status, status);
    const int end = (int)min(total.query, (long long)prm.num_tokens);
    if (rank == 0 && t == 0) prm.loc[B] = end;
    cluster.sync();  // every block has read the count

    if (rank == 0 && t == 0) *prm.new_count = bad_pool ? count : (int)(top - (long long)taken_sm);
    if (!bad_pool && total.back > 0) {
        for (int b = b0 + warp; b < b1; b += kWarps) {
            const Seq s = seq_of(prm, b);
            int32_t* row = prm.tables + (size_t)b * prm.cols;
            for (int i = s.n1 + lane; i < s.n0; i += 32)
                prm.free_blocks[count + offsets[b - b0].x + i - s.n1] = row[i];
        }
        cluster.sync();  // the stack is whole
    }
    if (!bad_pool && total.need > 0) {
        for (int b = b0 + warp; b < b1; b += kWarps) {
            const Seq s = seq_of(prm, b);
            const int before = offsets[b - b0].y;
            if (before < 0) continue;
            int32_t* row = prm.tables + (size_t)b * prm.cols;
            for (int i = s.n0 + lane; i < s.n1; i += 32) row[i] = __ldcg(prm.free_blocks + (top - 1 - before - (i - s.n0)));
        }
        cluster.sync();  // the tables are whole
    }
    for (int i = rank * kAllocThreads + t; i < prm.num_tokens; i += ctas * kAllocThreads) {
        int slot = -1, pos = -1;
        if (i < end) {
            int lo = 0, hi = B;  // the sequence: the last one that starts at or before i
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                (__ldcg(prm.loc + mid) <= i ? lo : hi) = mid;
            }
            const int context = __ldg(prm.context + lo), query = __ldg(prm.query + lo);
            pos = context + i - __ldcg(prm.loc + lo);
            const int blk = pos / kBlockSize;
            if (pos >= 0 && blk < prm.cols && __ldcg(prm.lens + lo) == context + query) {
                const int id = __ldcg(prm.tables + (size_t)lo * prm.cols + blk);
                if (id < 0 || id >= prm.num_blocks)
                    atomicOr(prm.status, PA_DEV_BAD_BLOCK_ID);
                else
                    slot = id * kBlockSize + pos % kBlockSize;
            }
        }
        prm.slots[i] = slot;
        prm.positions[i] = pos;
    }
}

// Eight halves.
struct alignas(16) Piece {
    __half2 h[4];
    __device__ __forceinline__ uint4& raw() { return *reinterpret_cast<uint4*>(h); }
};

// A warp takes rows_per_warp heads of one token, of Q, K and V in this order.  A
// row is D / 8 pieces of 16 bytes, a lane has the same piece of every row it
// meets and keeps that piece's cosines and sines in registers; 32 / (D / 8) rows
// at a time.  What is rotated lies in the lane's own piece (pairs) or in that of
// another lane of the row (halves); where half the rotated dims is not a whole
// number of pieces, partners are read one by one.
template <int D>
__global__ void __launch_bounds__(kPutThreads) kv_put_kernel(const KvPutParams prm) {
    constexpr int kPieces = D / 8, kRows = 32 / kPieces;
    const int lane = threadIdx.x & 31, token = blockIdx.x * (kPutThreads / 32) + (threadIdx.x >> 5);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    if (token >= prm.num_tokens) return;
    const int pos = __ldg(prm.positions + token);
    if (pos < 0) return;
    if (pos >= prm.max_positions && prm.rot > 0) {
        if (lane == 0) atomicOr(prm.status, PA_DEV_BAD_SEQ_LEN);
        return;
    }
    const bool caching = prm.cache[0] != nullptr;
    int slot = caching ? __ldg(prm.slots + token) : -1;
    if (slot >= prm.num_blocks * kBlockSize) {
        if (lane == 0) atomicOr(prm.status, PA_DEV_BAD_BLOCK_ID);
        slot = -1;
    }
    const int piece = lane % kPieces, d0 = piece * 8, r = prm.rot, half_r = r / 2;
    const bool whole = prm.pairs || half_r % 8 == 0;  // a piece's partners are one piece
    // the dims' factors: y = x * c + partner * s
    float c[8], s[8];
    int partner[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int d = d0 + e;
        c[e] = 1.f;
        s[e] = 0.f;
        partner[e] = d;
        if (d < r) {
            const bool second = prm.pairs ? d & 1 : d >= half_r;
            const int i = prm.pairs ? d / 2 : second ? d - half_r : d;
            c[e] = __ldg(prm.cos_sin + (size_t)pos * r + i);
            s[e] = __ldg(prm.cos_sin + (size_t)pos * r + half_r + i);
            if (!second) s[e] = -s[e];
            partner[e] = prm.pairs ? d ^ 1 : second ? d - half_r : d + half_r;
        }
    }
    const int src_lane = (lane & ~(kPieces - 1)) + (d0 >= r ? piece : d0 < half_r ? piece + half_r / 8 : piece - half_r / 8);
    const int H = prm.num_heads, K = prm.num_kv_heads, all = H + K + (caching ? K : 0);
    const int first = blockIdx.y * prm.rows_per_warp, last = min(all, first + prm.rows_per_warp);
    for (int base = first; base < last; base += kRows) {
        const int row = base + lane / kPieces;
        const bool real = row < last;
        const bool is_q = row < H, is_v = row >= H + K;
        const int head = is_q ? row : is_v ? row - H - K : row - H;
        const __half* src = is_q ? prm.q + token * prm.q_stride : is_v ? prm.v + token * prm.v_stride : prm.k + token * prm.k_stride;
        src += (size_t)head * D;
        Piece x, y;
        x.raw() = make_uint4(0u, 0u, 0u, 0u);
        if (real) x.raw() = *reinterpret_cast<const uint4*>(src + d0);
        y = x;
        if (whole) {
            Piece o;
            if (prm.pairs) {
#pragma unroll
                for (int e = 0; e < 4; ++e) o.h[e] = __lowhigh2highlow(x.h[e]);
            } else {
                o.raw().x = __shfl_sync(kFull, x.raw().x, src_lane);
                o.raw().y = __shfl_sync(kFull, x.raw().y, src_lane);
                o.raw().z = __shfl_sync(kFull, x.raw().z, src_lane);
                o.raw().w = __shfl_sync(kFull, x.raw().w, src_lane);
            }
            if (!is_v && d0 < r) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 a = __half22float2(x.h[e]), b = __half22float2(o.h[e]);
                    y.h[e] = __floats2half2_rn(fmaf(a.x, c[2 * e], b.x * s[2 * e]), fmaf(a.y, c[2 * e + 1], b.y * s[2 * e + 1]));
                    // (a dim past the rotated ones is copied: NaN payloads and signed zeros too)
                    if (d0 + 2 * e >= r) y.h[e] = x.h[e];
                }
            }
        } else if (real && !is_v && d0 < r) {
            __half* ye = reinterpret_cast<__half*>(y.h);
            const __half* xe = reinterpret_cast<const __half*>(x.h);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (d0 + e < r)
                    ye[e] = __float2half_rn(fmaf(__half2float(xe[e]), c[e], __half2float(src[partner[e]]) * s[e]));
        }
        __syncwarp();  // (in place: the row has been read)
        if (!real) continue;
        __half* dst = is_q ? prm.q_out : is_v ? nullptr : prm.k_out;
        if (dst) *reinterpret_cast<uint4*>(dst + ((size_t)token * (is_q ? H : K) + head) * D + d0) = y.raw();
        if (!is_q && slot >= 0) {
            __half* cache = prm.cache[is_v ? 1 : 0] +
                            (((size_t)(slot / kBlockSize) * K + head) * kBlockSize + slot % kBlockSize) * D;
            *reinterpret_cast<uint4*>(cache + d0) = y.raw();
        }
    }
}

}  // namespace

cudaError_t launch_kv_alloc(const KvAllocParams& prm, int cluster, cudaStream_t stream) {
    const int share = (prm.num_seqs + cluster - 1) / cluster;
    const int smem = 8 * (share > 0 ? share : 1);
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = once_per_device(done, [] {
        return cudaFuncSetAttribute(kv_alloc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 8 * 8192);
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(cluster);
    cfg.blockDim = dim3(kAllocThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2] = {pdl_attribute(), {}};
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kv_alloc_kernel, prm);
}

template <int D>
static cudaError_t launch_put(const KvPutParams& prm, dim3 grid, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kPutThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv_put_kernel<D>, prm);
}

cudaError_t launch_kv_put(int head_dim, const KvPutParams& prm, dim3 grid, cudaStream_t stream) {
    switch (head_dim) {
        case 64: return launch_put<64>(prm, grid, stream);
        case 128: return launch_put<128>(prm, grid, stream);
        case 256: return launch_put<256>(prm, grid, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace pa
