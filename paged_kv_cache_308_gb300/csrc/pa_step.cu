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
    const int held = prm.held[b];  // (which may become new_held)
    const long long room = min((long long)prm.cols * kBlockSize, 1ll << 30);
    s.bad = s.context < 0 || s.query < 0 || held < s.context || held > room || (long long)s.context + s.query > room;
    s.n0 = s.bad ? 0 : (held + kBlockSize - 1) / kBlockSize;
    s.n1 = s.bad ? 0 : (s.context + s.query + kBlockSize - 1) / kBlockSize;
    return s;
}

__device__ __forceinline__ Sums sums_of(const Seq& s) {
    return {max(s.query, 0), max(s.n0 - s.n1, 0), max(s.n1 - s.n0, 0)};
}

// What the placing of tokens needs to know of a sequence: where its tokens start, its
// context length, and of its blocks how many it held and how many were wanted before
// those it takes; -1 where it is not served, or its lengths are bad.
struct alignas(16) Taken {
    int loc, context, held, before;
};

// Slot and position of token i of sequence b, whose blocks are in its row up to those it
// takes and then on the stack, whose top (with what came back) is `top`.
__device__ __forceinline__ void place_token(const KvAllocParams& prm, int i, int b, const Taken& s, long long top) {
    const int pos = s.context + i - s.loc, blk = pos / kBlockSize;
    int slot = -1;
    if (pos >= 0 && blk < prm.cols && s.before >= 0) {
        const int id = blk < s.held ? __ldcg(prm.tables + (size_t)b * prm.cols + blk)
                                    : __ldcg(prm.free_blocks + (top - 1 - s.before - (blk - s.held)));
        if (id < 0 || id >= prm.num_blocks)
            atomicOr(prm.status, PA_DEV_BAD_BLOCK_ID);
        else
            slot = id * kBlockSize + pos % kBlockSize;
    }
    prm.slots[i] = slot;
    prm.positions[i] = pos;
}

// The last of n ascending starts (the first is 0) that is at most i.
template <typename F>
__device__ __forceinline__ int bisect(int n, int i, F&& start) {
    int lo = 0;
    while (n > 1) {
        const int half = n >> 1;
        if (start(lo + half) <= i) lo += half;
        n -= half;
    }
    return lo;
}

// The tokens of a call with many: a thread each, over the whole device.  The starts of up
// to kStarts sequences are looked up in shared memory.
constexpr int kStarts = 2048;
__global__ void __launch_bounds__(256) kv_alloc_place_kernel(const KvAllocParams prm) {
    __shared__ int starts[kStarts];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int B = prm.num_seqs, i = blockIdx.x * 256 + threadIdx.x;
    if (B <= kStarts) {
        for (int b = threadIdx.x; b < B; b += 256) starts[b] = __ldcg(prm.loc + b);
        __syncthreads();
    }
    if (i >= prm.num_tokens) return;
    if (i >= __ldcg(prm.loc + B)) {
        prm.slots[i] = prm.positions[i] = -1;
        return;
    }
    const int b = bisect(B, i, [&](int x) { return B <= kStarts ? starts[x] : __ldcg(prm.loc + x); });
    const int context = __ldg(prm.context + b), query = __ldg(prm.query + b);
    // (the tables are whole: every block is in its row)
    place_token(prm, i, b, {__ldcg(prm.loc + b), context, prm.cols, __ldcg(prm.lens + b) == context + query ? 0 : -1}, 0);
}

// One cluster does everything but, where there are many, the tokens: its blocks meet at
// the cluster's barrier, which needs no counter in memory that two calls could share.
// Every block sums over all sequences (a thread over consecutive ones) and keeps what it
// finds in shared memory: of all sequences where they are few enough (`All`), so that
// tokens can be placed next to the blocks' moves, else of its own share of them.  Its warps
// then move the blocks of its share, a sequence a warp at a time.
// What bounds it is the chain of trips to memory (lengths; sums; blocks given back; blocks
// taken; slots), not its bytes, a few hundred KB at most: 2.8 us for one sequence, 6.8 for a step of 64
// of which four end or shrink, 12.3 for 512 sequences' 130000 new tokens, 2 of them the second launch.
template <bool All>
__global__ void __launch_bounds__(kAllocThreads) kv_alloc_kernel(const KvAllocParams prm) {
    namespace cg = cooperative_groups;
    extern __shared__ Taken kept[];  // then as many blocks given back before a sequence, and wanted by it
    __shared__ Sums sm[kWarps];
    __shared__ unsigned long long taken_sm;
    const cg::cluster_group cluster = cg::this_cluster();
    const int rank = cluster.block_rank(), ctas = cluster.num_blocks();
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31, B = prm.num_seqs;
    if (t == 0) taken_sm = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");

    const int share = (B + ctas - 1) / ctas, b0 = min(B, rank * share), b1 = min(B, b0 + share);
    const int k0 = All ? 0 : b0, k1 = All ? B : b1;  // those kept
    int2* moves = reinterpret_cast<int2*>(kept + (All ? B : share));
    const int each = (B + kAllocThreads - 1) / kAllocThreads;
    const int s0 = min(B, t * each), s1 = min(B, s0 + each);
    const int count = __ldg(prm.count);
    Sums mine{0, 0, 0}, total;
    bool bad = false;
    Seq first{};
    for (int b = s0; b < s1; ++b) {
        const Seq s = seq_of(prm, b);
        if (b == s0) first = s;
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
        const Seq s = b == s0 ? first : seq_of(prm, b);
        const Sums one = sums_of(s);
        const bool served = one.need == 0 || (!bad_pool && at.need + one.need <= top);
        if (served)
            taken = max(taken, one.need ? at.need + one.need : 0);
        else
            status |= PA_DEV_NO_BLOCKS;
        const int loc = (int)min(at.query, (long long)prm.num_tokens);
        if (b >= k0 && b < k1) {
            // (sums are below 2^31 where they are used: the stack has no more blocks)
            kept[b - k0] = {loc, s.context, s.n0, served && !s.bad ? (int)min(at.need, 1ll << 30) : -1};
            moves[b - k0] = make_int2((int)min(at.back, 1ll << 30), s.n1);
        }
        if (b >= b0 && b < b1) {
            prm.lens[b] = s.bad ? 0 : served ? s.context + s.query : s.context;
            prm.loc[b] = loc;
        }
        at = plus(at, one);
    }
    if (taken) atomicMax(&taken_sm, (unsigned long long)taken);
    if (status && rank == 0) atomicOr(prm.status, status);
    const int end = (int)min(total.query, (long long)prm.num_tokens);
    if (rank == 0 && t == 0) prm.loc[B] = end;
    cluster.sync();  // every block has read the count and the lengths

    if (rank == 0 && t == 0) *prm.new_count = bad_pool ? count : (int)(top - (long long)taken_sm);
    if (prm.new_held) {
        for (int b = b0 + t; b < b1; b += kAllocThreads) {
            const Seq s = seq_of(prm, b);
            const bool moved = kept[b - k0].before >= 0 && (!bad_pool || s.n0 == s.n1);
            prm.new_held[b] = moved ? s.context + s.query : prm.held[b];
        }
    }
    if (!bad_pool && total.back > 0) {
        for (int b = b0 + warp; b < b1; b += kWarps) {
            const int held = kept[b - k0].held;
            const int2 m = moves[b - k0];
            const int32_t* row = prm.tables + (size_t)b * prm.cols;
            for (int i = m.y + lane; i < held; i += 32) prm.free_blocks[count + m.x + i - m.y] = row[i];
        }
        cluster.sync();  // the stack is whole
    }
    if (!bad_pool && total.need > 0) {
        for (int b = b0 + warp; b < b1; b += kWarps) {
            const Taken s = kept[b - k0];
            if (s.before < 0) continue;
            int32_t* row = prm.tables + (size_t)b * prm.cols;
            for (int i = s.held + lane; i < moves[b - k0].y; i += 32)
                row[i] = __ldcg(prm.free_blocks + (top - 1 - s.before - (i - s.held)));
        }
    }
    if (All && prm.place) {
        for (int i = rank * kAllocThreads + t; i < prm.num_tokens; i += ctas * kAllocThreads) {
            if (i < end) {
                const int b = bisect(B, i, [&](int x) { return kept[x].loc; });
                place_token(prm, i, b, kept[b], top);
            } else {
                prm.slots[i] = prm.positions[i] = -1;
            }
        }
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
// Bound by memory: 16384 tokens of 32/8 x 128 (436 MB) 80 us, 80 % of the measured
// bandwidth, the slots in no order; 64 tokens of 24/4 x 256 3.2 us, of 32/8 x 128 2.5, a launch and the chain
// position -> factors -> row.
template <int D, int Ahead>
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
    const float* row = prm.cos_sin + (size_t)pos * r;
    if (!prm.pairs && half_r % 8 == 0) {
        // eight factors in a row, a multiple of 32 bytes from the row's start (itself one of 64)
        const bool second = d0 >= half_r, turned = d0 < r;
        const float4* at = reinterpret_cast<const float4*>(row + (second ? d0 - half_r : d0));
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float4 x = turned ? __ldg(at + e) : make_float4(1.f, 1.f, 1.f, 1.f);
            float4 y = turned ? __ldg(at + half_r / 4 + e) : make_float4(0.f, 0.f, 0.f, 0.f);
            if (!second) y = make_float4(-y.x, -y.y, -y.z, -y.w);
            c[4 * e] = x.x, c[4 * e + 1] = x.y, c[4 * e + 2] = x.z, c[4 * e + 3] = x.w;
            s[4 * e] = y.x, s[4 * e + 1] = y.y, s[4 * e + 2] = y.z, s[4 * e + 3] = y.w;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int d = d0 + e;
            c[e] = 1.f;
            s[e] = 0.f;
            if (d < r) {
                const bool second = prm.pairs ? d & 1 : d >= half_r;
                const int i = prm.pairs ? d / 2 : second ? d - half_r : d;
                c[e] = __ldg(row + i);
                s[e] = __ldg(row + half_r + i);
                if (!second) s[e] = -s[e];
            }
        }
    }
    const int src_lane = (lane & ~(kPieces - 1)) + (d0 >= r ? piece : d0 < half_r ? piece + half_r / 8 : piece - half_r / 8);
    const int H = prm.num_heads, K = prm.num_kv_heads, all = H + K + (caching ? K : 0);
    const int first = blockIdx.y * prm.rows_per_warp, last = min(all, first + prm.rows_per_warp);
    // the lane's next Ahead rows are on their way while it works on as many (in place: a row is read whole before
    // any of it is written)
    const int mine = lane / kPieces;
    auto source = [&](int row) {
        const bool is_q = row < H, is_v = row >= H + K;
        return is_q   ? prm.q + token * prm.q_stride + (size_t)row * D
               : is_v ? prm.v + token * prm.v_stride + (size_t)(row - H - K) * D
                      : prm.k + token * prm.k_stride + (size_t)(row - H) * D;
    };
    Piece x[Ahead], next[Ahead];
    auto fetch = [&](int base) {
#pragma unroll
        for (int a = 0; a < Ahead; ++a) {
            const int row = base + a * kRows + mine;
            next[a].raw() = make_uint4(0u, 0u, 0u, 0u);
            if (row < last) next[a].raw() = __ldcs(reinterpret_cast<const uint4*>(source(row) + d0));
        }
    };
    fetch(first);
    for (int base = first; base < last; base += kRows * Ahead) {
#pragma unroll
        for (int a = 0; a < Ahead; ++a) x[a] = next[a];
        fetch(base + kRows * Ahead);
#pragma unroll
        for (int a = 0; a < Ahead; ++a) {
            const int row = base + a * kRows + mine;
            const bool real = row < last, is_q = row < H, is_v = row >= H + K;
            const int head = is_q ? row : is_v ? row - H - K : row - H;
            Piece y = x[a];
            if (whole) {
                Piece o;
                if (prm.pairs) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) o.h[e] = __lowhigh2highlow(x[a].h[e]);
                } else {
                    o.raw().x = __shfl_sync(kFull, x[a].raw().x, src_lane);
                    o.raw().y = __shfl_sync(kFull, x[a].raw().y, src_lane);
                    o.raw().z = __shfl_sync(kFull, x[a].raw().z, src_lane);
                    o.raw().w = __shfl_sync(kFull, x[a].raw().w, src_lane);
                }
                if (!is_v && d0 < r) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 u = __half22float2(x[a].h[e]), v = __half22float2(o.h[e]);
                        y.h[e] = __floats2half2_rn(fmaf(u.x, c[2 * e], v.x * s[2 * e]),
                                                   fmaf(u.y, c[2 * e + 1], v.y * s[2 * e + 1]));
                        // (a dim past the rotated ones is copied: NaN payloads and signed zeros too)
                        if (d0 + 2 * e >= r) y.h[e] = x[a].h[e];
                    }
                }
            } else if (real && !is_v && d0 < r) {
                __half* ye = reinterpret_cast<__half*>(y.h);
                const __half* xe = reinterpret_cast<const __half*>(x[a].h);
                const __half* src = source(row);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int d = d0 + e;
                    if (d < r) {
                        const float partner = __half2float(src[d < half_r ? d + half_r : d - half_r]);
                        ye[e] = __float2half_rn(fmaf(__half2float(xe[e]), c[e], partner * s[e]));
                    }
                }
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
}

}  // namespace

template <bool All>
static cudaError_t launch_alloc(const KvAllocParams& prm, int cluster, cudaStream_t stream) {
    constexpr int kMost = All ? kAllocAllSeqs : (65535 + kAllocMaxCluster - 1) / kAllocMaxCluster;
    constexpr int kEach = sizeof(Taken) + sizeof(int2);
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = once_per_device(done, [] {
        return cudaFuncSetAttribute(kv_alloc_kernel<All>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost * kEach);
    });
    if (e != cudaSuccess) return e;
    const int seqs = All ? prm.num_seqs : (prm.num_seqs + cluster - 1) / cluster;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(cluster);
    cfg.blockDim = dim3(kAllocThreads);
    cfg.dynamicSmemBytes = (seqs > 0 ? seqs : 1) * kEach;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2] = {pdl_attribute(), {}};
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, kv_alloc_kernel<All>, prm);
    if (e != cudaSuccess || (All && prm.place) || prm.num_tokens == 0) return e;
    cfg.gridDim = dim3((prm.num_tokens + 255) / 256);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv_alloc_place_kernel, prm);
}

cudaError_t launch_kv_alloc(const KvAllocParams& prm, int cluster, cudaStream_t stream) {
    return prm.num_seqs <= kAllocAllSeqs ? launch_alloc<true>(prm, cluster, stream)
                                         : launch_alloc<false>(prm, cluster, stream);
}

// Rows ahead of a lane: two where that is all of a warp's rows, or rows are so many at a time that four would
// leave the last ones of a token's heads mostly empty (head_dim 64); else four, which cover more of the trips to
// memory.  With two and four: 64 tokens of 32/8 x 128 2.5 / 3.0 us, 8192 of them 45.9 / 42.1; 64 of 12/12 x 64
// 2.2 / 2.7, 4096 of them 11.3 / 12.3, 8192 of them 23.7 / 23.5; 8192 of 24/4 x 256 58.4 / 51.8 (eight: 57.7).
template <int D>
static cudaError_t launch_put(const KvPutParams& prm, dim3 grid, cudaStream_t stream) {
    constexpr int kRows = 256 / D;  // at a time
    const bool two = D == 64 || prm.rows_per_warp <= 2 * kRows;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kPutThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return two ? cudaLaunchKernelEx(&cfg, kv_put_kernel<D, 2>, prm)
               : cudaLaunchKernelEx(&cfg, kv_put_kernel<D, D == 64 ? 2 : 4>, prm);
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
