// gq_moe.cu -- the router of a mixture-of-experts layer: per token, the top_k of E logits and
// their softmax weights. The layer itself is in gq_few.cu.
//
// One warp per token keeps the token's logits in registers (expert lane + 32 i) as integers in
// the order of the floats, so a round of the selection is one maximum over the lane's values,
// one warp maximum and one warp minimum over the lanes that hold it (the lowest index of equal
// logits). It reads 4 E bytes a token and is bound by those rounds, two warp reductions and the search
// for the holder for each of the top_k: a chain for one token, instructions for many (issue slots
// are 71 % busy). One token over 64 experts takes 1.8 us (a launch), 8191 over 128 with top_k = 8
// 7.5 us (0.7 us of bytes).
#include <algorithm>

#include "gq_few.cuh"

namespace gq {
namespace {

constexpr int kRouteThreads = 128;

// Order-preserving bits: larger float, larger unsigned. NaN counts as -infinity, and -0 as +0.
__device__ __forceinline__ uint32_t ordered(float z) {
    if (isnan(z)) z = -INFINITY;
    const uint32_t u = __float_as_uint(z + 0.0f);
    return u ^ (u >> 31 ? 0xFFFFFFFFu : 0x80000000u);
}

__device__ __forceinline__ float unordered(uint32_t o) {
    return __uint_as_float(o ^ (o >> 31 ? 0x80000000u : 0xFFFFFFFFu));
}

// e^(z - top), 1 where both are the same infinity.
__device__ __forceinline__ float share(float z, float top) { return z == top ? 1.0f : expf(z - top); }

template <int Per>   // values per lane: E <= 32 Per
__global__ void __launch_bounds__(kRouteThreads)
route_kernel(const float* __restrict__ logits, int64_t N, int E, int top_k, bool renorm,
             int32_t* __restrict__ ids, float* __restrict__ weights) {
    const int lane = threadIdx.x & 31;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (kRouteThreads / 32);
    for (int64_t n = static_cast<int64_t>(blockIdx.x) * (kRouteThreads / 32) + (threadIdx.x >> 5);
         n < N; n += warps) {
        const float* row = logits + n * E;
        uint32_t v[Per];   // 0: no expert, or one already taken (every logit's order is above 0)
        float all = 0.0f;
#pragma unroll
        for (int i = 0; i < Per; ++i) v[i] = lane + 32 * i < E ? ordered(row[lane + 32 * i]) : 0u;
        uint32_t best = v[0];
#pragma unroll
        for (int i = 1; i < Per; ++i) best = max(best, v[i]);
        const float top = unordered(__reduce_max_sync(0xFFFFFFFFu, best));
        if (!renorm) {
#pragma unroll
            for (int i = 0; i < Per; ++i)
                if (v[i]) all += share(unordered(v[i]), top);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xFFFFFFFFu, all, o);
        }
        int my_id[2] = {0, 0};
        float my_z[2] = {0.0f, 0.0f};
        float chosen = 0.0f;
        for (int j = 0; j < top_k; ++j) {
            uint32_t b = v[0];
#pragma unroll
            for (int i = 1; i < Per; ++i) b = max(b, v[i]);
            const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, b);
            unsigned at = 0xFFFFFFFFu;
            if (b == m) {
#pragma unroll
                for (int i = Per - 1; i >= 0; --i)
                    if (v[i] == m) at = lane + 32 * i;
            }
            const unsigned id = __reduce_min_sync(0xFFFFFFFFu, at);
#pragma unroll
            for (int i = 0; i < Per; ++i)
                if (id == static_cast<unsigned>(lane + 32 * i)) v[i] = 0u;
            const float z = unordered(m);
            chosen += share(z, top);
            if (lane == (j & 31)) {
                my_id[j >> 5] = static_cast<int>(id);
                my_z[j >> 5] = z;
            }
        }
        const float total = renorm ? chosen : all;
        const bool none = top == -INFINITY;   // every expert masked: no weights
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int j = lane + 32 * h;
            if (j < top_k) {
                ids[n * top_k + j] = my_id[h];
                weights[n * top_k + j] = none ? 0.0f : share(my_z[h], top) / total;
            }
        }
    }
}

}  // namespace

cudaError_t launch_moe_route(const float* logits, int64_t N, int E, int top_k, bool renorm,
                             int32_t* ids, float* weights, cudaStream_t s) {
    DeviceInfo* info = nullptr;
    cudaError_t e = current_device_info(&info);
    if (e != cudaSuccess) return e;
    const int64_t want = (N + kRouteThreads / 32 - 1) / (kRouteThreads / 32);
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(want, int64_t(info->sm_count) * 16));
    const auto run = [&](auto kernel) {
        kernel<<<grid, kRouteThreads, 0, s>>>(logits, N, E, top_k, renorm, ids, weights);
    };
    if (E <= 32) run(route_kernel<1>);
    else if (E <= 64) run(route_kernel<2>);
    else if (E <= 128) run(route_kernel<4>);
    else if (E <= 256) run(route_kernel<8>);
    else if (E <= 512) run(route_kernel<16>);
    else run(route_kernel<32>);
    return cudaGetLastError();
}

}  // namespace gq
