// gq_group.cu -- what stands between a router and grouped products: the token-expert pairs in order of
// their expert, and the weighted sum of the experts' results back to tokens.
//
// gq_moe_group is a counting sort: offsets[e] = pairs of experts below e; a pair's place is
// offsets[e] + the pairs of e before it. One launch of one cluster: every warp counts a run of pairs in a
// table of its own, CTAs exchange their sums through distributed shared memory, and a second pass over
// the same pairs, 32 at a time, gives each its place. Integer counts: the same bits on every call. Bound
// by the chain of these steps, and by the second pass where there are many pairs: 8 pairs 3.3 us, 65528 pairs
// of 128 experts 9.5 us (in graphs of calls; one by one from Python 12 and 16 us: the host).
//
// gq_moe_combine reads each result row once: bound by memory. 8191 tokens of 4 results, 2048 wide: 48 us,
// 6.4 TB/s; 16 tokens of 8: 2.2 us.
#include <algorithm>
#include <atomic>

#include "gq_few.cuh"
#include "gq_umma.cuh"

namespace gq {
namespace {

constexpr int kMaxCluster = 8;
constexpr int kMaxThreads = 1024;

__device__ __forceinline__ uint32_t ld_shared_cluster_u32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

struct GroupParams {
    const int32_t* ids;
    int32_t *offsets, *pairs, *places;
    int R, E;
    int run;   // pairs of a warp, a multiple of 32
    int bits;  // of a number up to E
};

// Eight rounds of a warp at a time: their ids are read together.
constexpr int kRounds = 8;

__global__ void __launch_bounds__(kMaxThreads, 1) group_kernel(const __grid_constant__ GroupParams p) {
    extern __shared__ int table[];   // [warp][E | 1], then the CTA's sums [E] and each expert's first place [E]
    __shared__ int warp_sum[kMaxThreads / 32];
    const int threads = blockDim.x, warps = threads >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_ctarank()), ctas = gridDim.x, stride = p.E | 1;
    int* sums = table + warps * stride;
    int* base = sums + p.E;
    int* mine = table + warp * stride;
    for (int i = threadIdx.x; i < warps * stride; i += threads) table[i] = 0;
    griddep_wait();
    griddep_launch_dependents();
    const int64_t first = (static_cast<int64_t>(rank) * warps + warp) * p.run;
    const int begin = static_cast<int>(min(first, static_cast<int64_t>(p.R)));
    const int end = static_cast<int>(min(first + p.run, static_cast<int64_t>(p.R)));
    int id[kRounds];
    const auto read = [&](int q0) {
#pragma unroll
        for (int i = 0; i < kRounds; ++i) {
            const int q = q0 + 32 * i + lane;
            id[i] = q < end ? p.ids[q] : -1;
        }
#pragma unroll
        for (int i = 0; i < kRounds; ++i)
            if (id[i] < 0 || id[i] >= p.E) id[i] = p.E;   // none
    };
    const unsigned below = (1u << lane) - 1u;
    read(begin);
    __syncthreads();
    for (int q0 = begin;;) {
#pragma unroll
        for (int i = 0; i < kRounds; ++i) {
            if (q0 + 32 * i >= end) break;
            if (id[i] < p.E) atomicAdd(&mine[id[i]], 1);
        }
        q0 += 32 * kRounds;
        if (q0 >= end) break;
        read(q0);
    }
    __syncthreads();
    // over the warps of the CTA: a lane for each
    for (int e = warp; e < p.E; e += warps) {
        const int c = lane < warps ? table[lane * stride + e] : 0;
        int incl = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xFFFFFFFFu, incl, o);
            if (lane >= o) incl += up;
        }
        if (lane < warps) table[lane * stride + e] = incl - c;
        if (lane == 31) sums[e] = incl;
    }
    cluster_sync();
    // each expert's pairs in all CTAs, in those before, and in the experts below it
    int carry = 0;
    for (int e0 = 0; e0 < p.E; e0 += threads) {
        const int e = e0 + threadIdx.x;
        int all = 0, before = 0;
        if (e < p.E) {
            const uint32_t at = smem_addr(&sums[e]);
            int c[kMaxCluster];
#pragma unroll
            for (int i = 0; i < kMaxCluster; ++i)
                c[i] = i < ctas ? static_cast<int>(ld_shared_cluster_u32(map_shared_rank(at, i))) : 0;
#pragma unroll
            for (int i = 0; i < kMaxCluster; ++i) {
                if (i < rank) before += c[i];
                all += c[i];
            }
        }
        int incl = all;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xFFFFFFFFu, incl, o);
            if (lane >= o) incl += up;
        }
        __syncthreads();   // warp_sum of the round before has been read
        if (lane == 31) warp_sum[warp] = incl;
        __syncthreads();
        int total = 0, start = carry + incl - all;
        for (int w = 0; w < warps; ++w) {
            if (w < warp) start += warp_sum[w];
            total += warp_sum[w];
        }
        carry += total;
        if (e < p.E) {
            if (rank == 0) {
                p.offsets[e] = start;
                if (e == p.E - 1) p.offsets[p.E] = start + all;
            }
            base[e] = start + before;
        }
    }
    __syncthreads();
    if (p.run > 32 * kRounds) read(begin);   // else the ids are still here
    for (int q0 = begin;;) {
#pragma unroll
        for (int i = 0; i < kRounds; ++i) {
            if (q0 + 32 * i >= end) break;
            const int q = q0 + 32 * i + lane;
            unsigned same = 0xFFFFFFFFu;   // lanes with this lane's expert
            for (int b = 0; b < p.bits; ++b) {
                const unsigned set = __ballot_sync(0xFFFFFFFFu, id[i] >> b & 1);
                same &= id[i] >> b & 1 ? set : ~set;
            }
            int place = -1;
            if (id[i] < p.E) {
                place = base[id[i]] + mine[id[i]] + __popc(same & below);
                p.pairs[place] = q;
            }
            __syncwarp();
            if (id[i] < p.E && (same & below) == 0) mine[id[i]] += __popc(same);
            __syncwarp();
            if (q < end) p.places[q] = place;
        }
        q0 += 32 * kRounds;
        if (q0 >= end) break;
        read(q0);
    }
    for (int64_t i = carry + static_cast<int64_t>(rank) * threads + threadIdx.x; i < p.R; i += int64_t(ctas) * threads)
        p.pairs[i] = -1;
    cluster_sync();   // no CTA leaves while another reads its sums
}

// A thread has V consecutive columns of one token; results are added in the order of the token's
// experts, four rows on their way at a time.
template <int V>
__global__ void __launch_bounds__(256)
combine_kernel(const float* __restrict__ O, int64_t R, int64_t D, const int32_t* __restrict__ places,
               const float* __restrict__ weights, int64_t N, int top_k, float* __restrict__ Y) {
    griddep_wait();
    griddep_launch_dependents();
    const int64_t cols = D / V;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= N * cols) return;
    const int64_t n = i / cols, d = (i - n * cols) * V;
    float y[V] = {};
    for (int j0 = 0; j0 < top_k; j0 += 4) {
        float v[4][V], w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int at = j0 + j < top_k ? places[n * top_k + j0 + j] : -1;
            const bool real = at >= 0 && at < R;
            w[j] = real ? weights[n * top_k + j0 + j] : 0.0f;
            if constexpr (V == 4) {
                const float4 o = real ? __ldcs(reinterpret_cast<const float4*>(O + at * D + d)) : float4{};
                v[j][0] = o.x; v[j][1] = o.y; v[j][2] = o.z; v[j][3] = o.w;
            } else {
                v[j][0] = real ? __ldcs(O + at * D + d) : 0.0f;
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int k = 0; k < V; ++k) y[k] = fmaf(w[j], v[j][k], y[k]);
    }
    if constexpr (V == 4) *reinterpret_cast<float4*>(Y + n * D + d) = make_float4(y[0], y[1], y[2], y[3]);
    else Y[n * D + d] = y[0];
}

}  // namespace

cudaError_t launch_moe_group(const int32_t* ids, int64_t R, int E, int32_t* offsets, int32_t* pairs,
                             int32_t* places, cudaStream_t s) {
    DeviceInfo* info = nullptr;
    cudaError_t e = current_device_info(&info);
    if (e != cudaSuccess) return e;
    static std::atomic<uint64_t> ready{0};   // devices whose attribute is set
    const uint64_t bit = uint64_t(1) << info->device;
    constexpr int kMost = (kMaxThreads / 32 + 2) * (kMoeMaxExperts + 1) * 4;
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(group_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    // A CTA for each 1024 pairs, up to eight. Its threads, 256, 512 or 1024, in us: 8 pairs of 64 experts 3.1,
    // 3.3, 3.4; 2048 4.9, 3.8, 4.8; 32768 -, 5.9, 6.5; 65528 of 128 experts -, 10.5, 9.5; 128 pairs of 1000 experts,
    // whose sums a warp each takes in turn, 18, 10.7, 8.7.
    const int threads = E > 256 || R > 32768 ? kMaxThreads : R <= 1024 ? 256 : 512;
    int ctas = 1;
    while (ctas < kMaxCluster && R > int64_t(ctas) * 1024) ctas *= 2;
    GroupParams p{ids, offsets, pairs, places, static_cast<int>(R), E, 0, 1};
    while (E >> p.bits) ++p.bits;
    const int64_t warps = int64_t(ctas) * (threads / 32);
    p.run = static_cast<int>(((R + warps - 1) / warps + 31) & ~int64_t(31));
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = (static_cast<size_t>(threads / 32) * (E | 1) + 2 * static_cast<size_t>(E)) * 4;
    cfg.stream = s;
    cudaLaunchAttribute attr[2]{};
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, group_kernel, p);
}

cudaError_t launch_moe_combine(const float* O, int64_t R, int64_t D, const int32_t* places, const float* weights,
                               int64_t N, int top_k, float* Y, cudaStream_t s) {
    const bool vec = D % 4 == 0 && ((reinterpret_cast<uintptr_t>(O) | reinterpret_cast<uintptr_t>(Y)) & 15) == 0;
    const int64_t threads = N * (vec ? D / 4 : D), ctas = (threads + 255) / 256;
    if (ctas > INT32_MAX) return cudaErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>(ctas));
    return vec ? launch_after(combine_kernel<4>, grid, 256, 0, s, O, R, D, places, weights, N, top_k, Y)
               : launch_after(combine_kernel<1>, grid, 256, 0, s, O, R, D, places, weights, N, top_k, Y);
}

}  // namespace gq
