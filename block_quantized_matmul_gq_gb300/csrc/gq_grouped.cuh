// gq_grouped.cuh -- the product kernel of grouped rows (its mathematics and design: gq_grouped.cu) and its
// launch. One translation unit for each weight type includes it, so that they compile in parallel.
#pragma once

#include <algorithm>
#include <atomic>
#include <cuda.h>   // CUtensorMap and its enums (header only; no libcuda link)
#include <type_traits>

#include "gq_few.cuh"
#include "gq_umma.cuh"

namespace gq {

constexpr int kBM = 128;         // weight rows of a tile
constexpr int kThreads = 640;    // warps: copying, issuing, two idle, eight unpacking, eight adding up
constexpr int kChunk = 256;      // k of a row's chunk of raw bytes: two stages of 128
constexpr int kSlots = 2;        // stages in TMEM: codes, and accumulators
constexpr int kScaleRing = 4;    // stages whose scales are kept

// Raw bytes of a chunk in shared memory: 16-byte words copied a row, pitch (an odd number of words:
// a warp's 16-byte reads of 32 rows do not collide), chunks in flight. Aligned: a row's chunks start
// on 16-byte boundaries (K % 256 == 0; MXFP4, K % 512 == 0: 8-byte ones), and come by tensor map; else
// anywhere.
template <int T, bool Aligned>
struct Raw;
template <>
struct Raw<GQ_TYPE_Q4_0, true> {
    static constexpr int bytes = 144, words = 9, pitch = 144, bufs = 4;
};
template <>
struct Raw<GQ_TYPE_Q4_0, false> {
    static constexpr int bytes = 144, words = 10, pitch = 176, bufs = 3;
};
template <>
struct Raw<GQ_TYPE_Q8_0, true> {
    static constexpr int bytes = 272, words = 17, pitch = 272, bufs = 2;
};
template <>
struct Raw<GQ_TYPE_Q8_0, false> {
    static constexpr int bytes = 272, words = 18, pitch = 304, bufs = 2;
};
template <>
struct Raw<GQ_TYPE_Q4_K, true> {
    static constexpr int bytes = 144, words = 9, pitch = 144, bufs = 4;
};
template <>
struct Raw<GQ_TYPE_MXFP4, true> {
    static constexpr int bytes = 136, words = 9, pitch = 144, bufs = 4;
};
template <>
struct Raw<GQ_TYPE_MXFP4, false> {
    static constexpr int bytes = 136, words = 10, pitch = 176, bufs = 3;
};

// Forms of the kernel, by the rows an expert has: tiles of up to 32 rows with a sum for each 32 k, or of 64 or
// 128 (Q4_K 96) with one for 128 k.
enum Form { kFewRows, kSomeRows, kManyRows };

template <int T, bool Aligned, int F>
struct Cfg {
    using R = Raw<T, Aligned>;
    static_assert(F != kFewRows || T != GQ_TYPE_MXFP4, "its weights are one exact term");
    static constexpr bool kMins = T == GQ_TYPE_Q4_K;
    static constexpr bool kFew = F == kFewRows;
    static constexpr bool kTwo = !kFew && T != GQ_TYPE_MXFP4;   // terms of a weight
    static constexpr int kBN = kFew ? 32 : F == kSomeRows ? 64 : kMins ? 96 : 128;   // most tokens of a tile
    static constexpr int kUnits = kFew ? 4 + kMins : 1;         // accumulators (and scales) of a stage
    static constexpr int kACols = (kTwo ? 128 : 64) + (kMins ? 16 : 0);   // TMEM columns of a stage's weights
    static constexpr int kDCols = kUnits * kBN;
    static constexpr int kMinA = kTwo ? 128 : 64;              // Q4_K: the mins' columns
    static constexpr int kBufs = !kFew ? R::bufs : R::pitch == 144 ? 6 : R::pitch == 176 ? 5 : 3;   // of raw chunks
    static constexpr int kHalf = kBN * 256;              // 64 k of the tokens, two terms
    // (few rows, 16 tokens over 64 Q8_0 experts: with two stages 39.4 us, four 34.1, six 34.7)
    static constexpr int kXStages = F == kManyRows ? 2 : kMins && !kFew ? 3 : 4, kMinBytes = kBN * 128;
    static constexpr int kMin = kXStages * 2 * kHalf;
    static constexpr int kRaw = kMin + (kMins ? 2 * kMinBytes : 0);
    static constexpr int kRawBytes = kBM * R::pitch;     // of one chunk
    static constexpr int kScales = kRaw + kBufs * kRawBytes;
    static constexpr int kLists = kScales + kScaleRing * kUnits * kBM * 4;
    static constexpr int kSwap = kLists + 2 * (kGroupedMaxExperts + 1 + 512) * 4;   // few rows: partial sums
    static constexpr int kSmem = kSwap + (kFew ? 8 * 16 * 32 * 4 : 0) + 1024;
    static constexpr int kA = kSlots * kDCols;           // TMEM: accumulators, then weights
    static_assert(kA + kSlots * kACols <= 512, "TMEM");
    static_assert(kSmem <= 227 * 1024 - 2560, "shared memory, beside 2304 bytes of fixed size");
};

// A group's first row in the split activations: groups are padded to 16 rows, so that a tile is
// whole atoms of 8 rows, and every group that is not empty starts behind the last one's padding.
__host__ __device__ __forceinline__ int64_t padded_start(int64_t off, int64_t e) {
    return ((off + 15) & ~int64_t(15)) + 16 * (e < off ? e : off);
}

struct GroupedParams {
    CUtensorMap map, map2;    // aligned: the weights' bytes, boxes of 64 rows and one chunk
    const uint8_t* W;
    const uint8_t* W2;        // SwiGLU: the up matrices (W: gate); else nullptr
    int64_t total_bytes;      // of W (and of W2)
    int64_t row_bytes;
    const int32_t* offsets;
    int64_t R;
    int E, M, kb, m_tiles;
    unsigned inverse;         // 2^32 / m_tiles, rounded down, below 2^32
    int64_t atoms;
    const uint8_t* xw;
    const uint8_t* mins;
    const float* xs;
    float* Y;
    unsigned* status;
};

// What the host side of gq_grouped.cu has decided.
struct GroupedLaunch {
    int64_t tiles;   // at most
    Form form;
    bool aligned, swiglu;
};
cudaError_t launch_grouped_q4_0(GroupedParams& g, const GroupedLaunch& l, const DeviceInfo* info, cudaStream_t s);
cudaError_t launch_grouped_q8_0(GroupedParams& g, const GroupedLaunch& l, const DeviceInfo* info, cudaStream_t s);
cudaError_t launch_grouped_q4_k(GroupedParams& g, const GroupedLaunch& l, const DeviceInfo* info, cudaStream_t s);
cudaError_t launch_grouped_mxfp4(GroupedParams& g, const GroupedLaunch& l, const DeviceInfo* info, cudaStream_t s);

namespace {

// kind::f16 with fp16 operands and fp32 accumulators, 128 rows, n columns.
__device__ __forceinline__ uint32_t f16_idesc(int n) {
    return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(kBM >> 4) << 24);
}

// K-major operand in the 128-byte swizzle, groups of 8 rows `stride` bytes apart.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr, uint32_t stride) {
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(1) << 16) |
           (static_cast<uint64_t>(stride >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
           (static_cast<uint64_t>(2) << 61);
}

__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}

// acc += s * v, two fp32 lanes each.
__device__ __forceinline__ void fma2(uint64_t& acc, uint64_t v, uint64_t s) {
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(v), "l"(s));
}

// Ends the loads of 16 columns: nothing may use them before.
__device__ __forceinline__ void tmem_wait16(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15])::"memory");
}

// Whether a phase is complete; and the wait that ends with it. A test of a barrier takes 110 cycles from
// the instruction to the first use of its answer, so every warp tests its next barrier before the work at
// hand and uses the answer after it. (One lane alone waiting takes two to five times as long to notice.)
__device__ __forceinline__ uint32_t peek(const uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return ok;
}
// A try sleeps up to 1.4 us (measured), so a wait ends after about 1.5 s; a loop with the timer in it, or a
// call of one, costs up to 8 %: the code of all roles has to come from one instruction cache.
__device__ __forceinline__ bool finish(uint32_t seen, const uint64_t* bar, uint32_t parity) {
    bool ok = __all_sync(0xFFFFFFFFu, seen);
#pragma unroll 1
    for (int i = 0; i < 1 << 20 && !ok; ++i) ok = __all_sync(0xFFFFFFFFu, mbar_try_wait(smem_addr(bar), parity));
    return ok;
}

__device__ __forceinline__ void sts32(uint32_t a, float v) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}
__device__ __forceinline__ float lds_f32(uint32_t a) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
    return v;
}

// g / (1 + e^-g), by e^-|g|, which stays in range. The reciprocal (1 ulp) of a number in [1, 2] instead of
// a division: the whole is off by at most 12 2^-24.
__device__ __forceinline__ float swish(float g) {
    const float e = expf(-fabsf(g));
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return (g < 0.0f ? g * e : g) * r;
}

// The launch's tiles, the same in every CTA: a unit is a tile of tokens of one expert, each with the
// expert's m_tiles tiles of weight rows. Units beyond the list are searched for by the number of units
// before each expert: a search and its divisions cost a role 500 cycles a tile, the list 100.
constexpr int kUnitList = 512;
struct Lists {
    int off[kGroupedMaxExperts + 1];      // first row of each group, inside [0, R]
    int units[kGroupedMaxExperts + 1];    // of the experts before
    int row[kUnitList];                   // of the first units: first row,
    uint32_t expert[kUnitList];           // expert, number of rows << 16
};

struct Tile {
    int e, mt;      // expert, tile of weight rows
    int row, n;     // first row of Y and number of rows (1..BN)
    int64_t x_row;  // first row of the split activations
};

// Rows of the units of a group of n: even, whole MMA columns (the last may have fewer).
template <int BN>
__device__ __forceinline__ int unit_rows(int n, int units) {
    return ((n + units - 1) / units + 15) & ~15;
}

template <int BN>
__device__ __forceinline__ Tile locate(const Lists& L, const GroupedParams& p, int t) {
    Tile o;
    int unit = static_cast<int>(__umulhi(static_cast<unsigned>(t), p.inverse));   // t / m_tiles, or one less
    o.mt = t - unit * p.m_tiles;
    if (o.mt >= p.m_tiles) {
        ++unit;
        o.mt -= p.m_tiles;
    }
    if (unit < kUnitList) {
        const uint32_t en = L.expert[unit];
        o.row = L.row[unit];
        o.e = static_cast<int>(en & 0xFFFFu);
        o.n = static_cast<int>(en >> 16);
        const int off = L.off[o.e];
        o.x_row = padded_start(off, o.e) + (o.row - off);
        return o;
    }
    int lo = 0, hi = p.E - 1;   // the last expert with at most `unit` units before it
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (L.units[mid] <= unit) lo = mid;
        else hi = mid - 1;
    }
    o.e = lo;
    const int off = L.off[lo], n = L.off[lo + 1] - off, per = unit_rows<BN>(n, L.units[lo + 1] - L.units[lo]);
    const int first = (unit - L.units[lo]) * per;
    o.row = off + first;
    o.n = min(per, n - first);
    o.x_row = padded_start(off, lo) + first;
    return o;
}

// SwiGLU tiles are 64 gate rows and the 64 up rows of the same numbers, in shared memory one after the
// other, in TMEM (rows r) 16 of each in turn: the shared row of r, and where a shared row's weights begin.
__device__ __forceinline__ int shared_row(bool swiglu, int r) {
    return swiglu ? (r >> 5) * 16 + (r & 15) + ((r & 16) << 2) : r;
}
template <bool Swiglu>
__device__ __forceinline__ int64_t place_of(const GroupedParams& p, const Tile& at, int row) {
    const int m = Swiglu ? at.mt * (kBM / 2) + (row & 63) : at.mt * kBM + row;
    return (static_cast<int64_t>(at.e) * p.M + min(m, p.M - 1)) * p.row_bytes;
}

// One stage (64 k, two blocks) of a weight row: its words in order, the first block at byte 0.
template <int T, bool Aligned>
struct StageWords;
template <>
struct StageWords<GQ_TYPE_Q4_0, true> {
    uint32_t w[9];
    template <int S>
    __device__ __forceinline__ void load(uint32_t row, int) {
        uint32_t u[12];
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const uint4 v = lds128(row + 16 * (2 * S + i));
            u[4 * i] = v.x; u[4 * i + 1] = v.y; u[4 * i + 2] = v.z; u[4 * i + 3] = v.w;
        }
#pragma unroll
        for (int i = 0; i < 9; ++i) w[i] = u[i + S];
    }
};
template <>
struct StageWords<GQ_TYPE_Q8_0, true> {
    uint32_t w[17];
    template <int S>
    __device__ __forceinline__ void load(uint32_t row, int) {
        uint32_t u[20];
#pragma unroll
        for (int i = 0; i < 5; ++i) {
            const uint4 v = lds128(row + 16 * (4 * S + i));
            u[4 * i] = v.x; u[4 * i + 1] = v.y; u[4 * i + 2] = v.z; u[4 * i + 3] = v.w;
        }
#pragma unroll
        for (int i = 0; i < 17; ++i) w[i] = u[i + S];
    }
};
template <>
struct StageWords<GQ_TYPE_MXFP4, true> {   // lead: 0 or 8
    uint32_t w[9];
    template <int S>
    __device__ __forceinline__ void load(uint32_t row, int lead) {
        uint32_t u[10];
#pragma unroll
        for (int i = 0; i < 5; ++i) {
            const uint2 v = lds64(row + lead + 8 * (4 * S + i));
            u[2 * i] = v.x; u[2 * i + 1] = v.y;
        }
#pragma unroll
        for (int i = 0; i < 9; ++i) {
            constexpr int at = S >> 1;   // 2 S bytes in
            const uint32_t next = i + at + 1 < 10 ? u[i + at + 1 < 10 ? i + at + 1 : 9] : 0u;
            w[i] = S & 1 ? __funnelshift_r(u[i + at], next, 16) : u[i + at];
        }
    }
};
template <int T>
struct StageWords<T, false> {
    static constexpr int kBytes = Raw<T, false>::bytes / 4, kWords = (kBytes + 3) / 4;
    uint32_t w[kWords];
    template <int S>
    __device__ __forceinline__ void load(uint32_t row, int lead) {
        const int at = lead + S * kBytes;
        const uint32_t a = row + (at & ~3), sh = 8 * (at & 3);
        uint32_t before = lds32(a);
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            const uint32_t next = lds32(a + 4 * i + 4);
            w[i] = __funnelshift_r(before, next, sh);
            before = next;
        }
    }
};

// fp16 words with the same value in both halves.
__device__ __forceinline__ uint32_t dup_half(float v) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %1;" : "=r"(r) : "f"(v));
    return r;
}
// a b - c.
__device__ __forceinline__ uint32_t h2_fms(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("{\n\t.reg .b32 t;\n\tneg.f16x2 t, %3;\n\tfma.rn.f16x2 %0, %1, %2, t;\n\t}" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}

// Floor of log2 of a positive normal float; for zero and subnormal ones -127.
__device__ __forceinline__ int exponent_of(float v) { return static_cast<int>(__float_as_uint(v) >> 23) - 127; }

// Where a weight is two terms its code comes times 2^-kLift, into [-1, 1], and its scale with the rest of the 15 bits
// that a term has: scales that are small beside the largest then stay out of fp16's subnormals, where they would lose
// bits that the code multiplies again (Q8_0: 2^-25 of the largest scale instead of 2^-31, Q4_0 2^-33 and 2^-35, Q4_K
// 2^-29 and 2^-32).
template <int T>
constexpr int kLift = T == GQ_TYPE_Q8_0 ? 7 : T == GQ_TYPE_Q4_0 ? 3 : T == GQ_TYPE_Q4_K ? 4 : 0;

// The codes of block b (0, 1) of two, times 2^-Lift, as fp16, 16 words in the order of few_place.
template <int T, int Lift, int N>
__device__ __forceinline__ void codes_of(const uint32_t (&w)[N], int b, uint32_t (&h)[16]) {
    uint32_t q[4];
    if constexpr (T == GQ_TYPE_Q4_0) {   // 18 bytes: codes start 2 (20) bytes in
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            nibbles_to_f16<8, Lift>(b == 0 ? __funnelshift_r(w[t], w[t + 1], 16) : w[5 + t], q);
#pragma unroll
            for (int j = 0; j < 4; ++j) h[4 * t + j] = q[j];
        }
    } else if constexpr (T == GQ_TYPE_MXFP4) {   // 17 bytes: codes start 1 (18) bytes in
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            e2m1_to_f16(__funnelshift_r(w[4 * b + t], w[4 * b + t + 1], b == 0 ? 8 : 16), q);
#pragma unroll
            for (int j = 0; j < 4; ++j) h[4 * t + j] = q[j];
        }
    } else {   // Q8_0, 34 bytes: codes start 2 (36) bytes in
        constexpr uint32_t kOne = 0x64006400u - 0x00010001u * (Lift << 10), kZero = kOne + 0x00800080u;   // 1024, + 128
        constexpr uint32_t kHigh = kOne >> 8 & 0xFFu, kBytes = kHigh * 0x01010101u;
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            const uint32_t v = (b == 0 ? __funnelshift_r(w[t], w[t + 1], 16) : w[9 + t]) ^ 0x80808080u;
            h[2 * t] = h2_sub(__byte_perm(v, kBytes, 0x4140), kZero);
            h[2 * t + 1] = h2_sub(__byte_perm(v, kBytes, 0x4342), kZero);
        }
    }
}

template <int T, bool Aligned, bool Swiglu, int F>
__global__ void __launch_bounds__(kThreads, 1) grouped_kernel(const __grid_constant__ GroupedParams p) {
    using C = Cfg<T, Aligned, F>;
    constexpr bool Few = C::kFew;
    using R = Raw<T, Aligned>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t x_full[C::kXStages], x_empty[C::kXStages], a_full[kSlots], done[kSlots], d_empty[kSlots],
        raw_full[C::kBufs], raw_empty[C::kBufs], drained;
    __shared__ __align__(16) float x_scale[8][64];
    __shared__ uint32_t tmem_at;
    __shared__ int warp_sum[kThreads / 32];
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // warp: uniform
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    Lists& L = *reinterpret_cast<Lists*>(smem_raw + (base - smem_addr(smem_raw)) + C::kLists);
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kXStages; ++i) {
            mbar_init(smem_addr(&x_full[i]), 1);
            mbar_init(smem_addr(&x_empty[i]), 1);
        }
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(smem_addr(&a_full[i]), 8);
            mbar_init(smem_addr(&done[i]), 1);
            mbar_init(smem_addr(&d_empty[i]), 8);
        }
        for (int i = 0; i < C::kBufs; ++i) {
            mbar_init(smem_addr(&raw_full[i]), Aligned ? 1 : 64);
            mbar_init(smem_addr(&raw_empty[i]), 8);
        }
        mbar_init(smem_addr(&drained), 1);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_addr(&tmem_at), 512);
        tmem_relinquish();
    }
    // The groups (they come from before the preparation, which let this kernel start): a group's first
    // row is the largest offset up to its own, inside [0, R]; units by a sum over the experts, two to a
    // thread (more threads than pairs of experts).
    {
        const int e = 2 * threadIdx.x;
        const auto offset = [&](int i) {
            return i <= p.E ? static_cast<int>(min(static_cast<int64_t>(max(p.offsets[i], 0)), p.R)) : 0;
        };
        const int o0 = offset(e), o1 = max(o0, offset(e + 1));
        int top = o1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) top = max(top, __shfl_up_sync(0xFFFFFFFFu, top, o));   // own value below
        if (lane == 31) warp_sum[warp] = top;
        __syncthreads();
        int prev = __shfl_up_sync(0xFFFFFFFFu, top, 1);
        if (lane == 0) prev = 0;
        for (int i = 0; i < warp; ++i) prev = max(prev, warp_sum[i]);
        if (e <= p.E) L.off[e] = max(prev, o0);
        if (e + 1 <= p.E) L.off[e + 1] = max(prev, o1);
        __syncthreads();
        int n[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            n[i] = e + i < p.E ? (L.off[e + i + 1] - L.off[e + i] + C::kBN - 1) / C::kBN : 0;
        int incl = n[0] + n[1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xFFFFFFFFu, incl, o);
            if (lane >= o) incl += up;
        }
        if (lane == 31) warp_sum[warp] = incl;
        __syncthreads();
        int before = incl - n[0] - n[1];
        for (int i = 0; i < warp; ++i) before += warp_sum[i];
        if (e <= p.E) L.units[e] = before;
        if (e + 1 <= p.E) L.units[e + 1] = before + n[0];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (n[i] == 0) continue;
            const int off = L.off[e + i], rows = L.off[e + i + 1] - off, per = unit_rows<C::kBN>(rows, n[i]);
            const int first = i ? before + n[0] : before;
            for (int u = 0; u < n[i] && first + u < kUnitList; ++u) {
                L.row[first + u] = off + u * per;
                L.expert[first + u] = static_cast<uint32_t>(e + i) | static_cast<uint32_t>(min(per, rows - u * per)) << 16;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_launch_dependents();
    const uint32_t tmem = tmem_at;
    const int tiles = L.units[p.E] * p.m_tiles;
    const int stages = (p.kb + 3) / 4;

    if (warp == 0) {
        griddep_wait();   // the split activations
        int slot = 0, used = 0, sb = 0;
        uint32_t phase = 1;   // of `x_empty`: the first round passes at once
        uint32_t seen = 1;
        bool ok = true;
        for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
            const Tile at = locate<C::kBN>(L, p, t);
            const uint32_t atoms = static_cast<uint32_t>((at.n + 15) & ~15) >> 3;
            const uint8_t* from = p.xw + ((at.x_row >> 3) << 11);
            const uint8_t* mins = p.mins + ((at.x_row >> 3) << 10);
            for (int s = 0; s < stages; ++s) {
                ok = finish(seen, &x_empty[slot], phase);
                if (!ok) break;
                const uint32_t bar = smem_addr(&x_full[slot]), to = base + slot * 2 * C::kHalf;
                const bool both = 4 * s + 2 < p.kb, last = C::kMins && (s & 1);
                if (elect_one()) {
                    mbar_arrive_expect_tx(bar, atoms * (last ? 5120u : both ? 4096u : 2048u));
                    bulk_g2s(to, from, atoms * 2048u, bar);
                    if (both) bulk_g2s(to + C::kHalf, from + (p.atoms << 11), atoms * 2048u, bar);
                    if (last) bulk_g2s(base + C::kMin + sb * C::kMinBytes, mins, atoms * 1024u, bar);
                }
                __syncwarp();
                from += p.atoms << 12;
                if (last) {
                    mins += p.atoms << 10;
                    sb ^= 1;
                }
                ++used;
                if (++slot == C::kXStages) {
                    slot = 0;
                    phase ^= 1;
                }
                seen = peek(&x_empty[slot], phase);
            }
        }
        if (!ok && lane == 0) report_status(p.status, kStatusTimeout);
        // no copy may be in flight when the CTA leaves
        for (int i = 0; i < min(used, C::kXStages); ++i) {
            if (--slot < 0) {
                slot = C::kXStages - 1;
                phase ^= 1;
            }
            finish(0, &x_full[slot], phase ^ 1);
        }
    } else if (warp == 1) {
        griddep_wait();   // no wait below is for another kernel
        int slot = 0, xslot = 0, sb = 0;
        uint32_t phase = 0, x_phase = 0, seen_a = 0, seen_x = 0, seen_d = 1;
        bool ok = true;
        for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
            const uint32_t idesc = f16_idesc((locate<C::kBN>(L, p, t).n + 15) & ~15);
            for (int s = 0; s < stages; ++s) {
                ok = finish(seen_x, &x_full[xslot], x_phase) && finish(seen_a, &a_full[slot], phase) &&
                     finish(seen_d, &d_empty[slot], phase ^ 1);
                if (!ok) break;
                tc_fence_after();
                const uint32_t d = tmem + slot * C::kDCols, a = tmem + C::kA + slot * C::kACols;
                const uint64_t hi = sw128_desc(base + xslot * 2 * C::kHalf, 2048);
                const uint32_t full = smem_addr(&done[slot]), empty = smem_addr(&x_empty[xslot]);
                slot ^= 1;
                phase ^= slot == 0;
                if (++xslot == C::kXStages) {
                    xslot = 0;
                    x_phase ^= 1;
                }
                seen_a = peek(&a_full[slot], phase);
                seen_x = peek(&x_full[xslot], x_phase);
                seen_d = peek(&d_empty[slot], phase ^ 1);
                const int steps = min(8, 2 * (p.kb - 4 * s));   // of 16 k: 32 bytes of a row, 8 columns of A
                const bool last = C::kMins && (s & 1);
                if (elect_one()) {
                    const auto at = [&](int q) { return hi + (q >> 2) * (C::kHalf >> 4) + 2 * (q & 3); };
                    const auto products = [&](int n) {
                        if constexpr (Few) {   // a sum for each block
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                if (2 * u >= n) break;
                                const uint32_t du = d + u * C::kBN, au = a + 16 * u;
                                umma_bf16_tmem_a(du, au, at(2 * u) + (1024 >> 4), idesc, 0);
                                umma_bf16_tmem_a(du, au + 8, at(2 * u + 1) + (1024 >> 4), idesc, 1);
                                umma_bf16_tmem_a(du, au, at(2 * u), idesc, 1);
                                umma_bf16_tmem_a(du, au + 8, at(2 * u + 1), idesc, 1);
                            }
                            if (last) {
                                const uint64_t m = sw128_desc(base + C::kMin + sb * C::kMinBytes, 1024);
                                umma_bf16_tmem_a(d + 4 * C::kBN, a + C::kMinA, m + 2, idesc, 0);
                                umma_bf16_tmem_a(d + 4 * C::kBN, a + C::kMinA, m, idesc, 1);
                            }
                            return;
                        }
                        if (C::kTwo)
#pragma unroll
                            for (int q = 0; q < 8; ++q)
                                if (q < n) umma_bf16_tmem_a(d, a + 64 + 8 * q, at(q), idesc, q > 0);
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            if (q < n) umma_bf16_tmem_a(d, a + 8 * q, at(q) + (1024 >> 4), idesc, C::kTwo || q > 0);
                        if (last) {
                            const uint64_t m = sw128_desc(base + C::kMin + sb * C::kMinBytes, 1024);
                            umma_bf16_tmem_a(d, a + C::kMinA, m, idesc, 1);
                            umma_bf16_tmem_a(d, a + C::kMinA + 8, m + 2, idesc, 1);
                        }
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            if (q < n) umma_bf16_tmem_a(d, a + 8 * q, at(q), idesc, 1);
                    };
                    if (steps == 8) products(8);
                    else products(steps);
                    umma_commit(full);
                    umma_commit(empty);
                }
                __syncwarp();
                if (last) sb ^= 1;
            }
        }
        if (!ok && lane == 0) report_status(p.status, kStatusTimeout);
        if (elect_one()) umma_commit(smem_addr(&drained));   // nothing may run when TMEM is given back
        __syncwarp();
        finish(0, &drained, 0);
    } else if (Aligned && warp == 2) {
        // The weights' raw bytes, a chunk of 256 k of the tile's 128 rows at a time, two boxes of 64 rows
        // (SwiGLU: gate, up). They do not depend on the kernel before. Rows past an expert's last are the next
        // expert's, past the last matrix zeros: their results are not stored.
        const int chunks = (p.kb + 7) / 8;
        const CUtensorMap* second = Swiglu ? &p.map2 : &p.map;
        constexpr int kUnit = R::words > 16 ? 2 : 1;   // bytes of an element: a box has at most 256
        int buf = 0, used = 0;
        uint32_t phase = 1, seen = 1;
        bool ok = true;
        for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
            const Tile at = locate<C::kBN>(L, p, t);
            const int row = at.e * p.M + at.mt * (Swiglu ? kBM / 2 : kBM), row2 = Swiglu ? row : row + kBM / 2;
            for (int c = 0; c < chunks; ++c) {
                ok = finish(seen, &raw_empty[buf], phase);
                if (!ok) break;
                const uint32_t bar = smem_addr(&raw_full[buf]), to = base + C::kRaw + buf * C::kRawBytes;
                const int x = c * R::bytes / 16 * 16 / kUnit;
                if (elect_one()) {
                    mbar_arrive_expect_tx(bar, C::kRawBytes);
                    tma_load_2d(to, &p.map, x, row, bar);
                    tma_load_2d(to + C::kRawBytes / 2, second, x, row2, bar);
                }
                __syncwarp();
                ++used;
                if (++buf == C::kBufs) {
                    buf = 0;
                    phase ^= 1;
                }
                seen = peek(&raw_empty[buf], phase);
            }
        }
        if (!ok && lane == 0) report_status(p.status, kStatusTimeout);
        for (int i = 0; i < min(used, C::kBufs); ++i) {
            if (--buf < 0) {
                buf = C::kBufs - 1;
                phase ^= 1;
            }
            finish(0, &raw_full[buf], phase ^ 1);
        }
    } else if (!Aligned && (warp == 2 || warp == 3)) {
        // The same where rows begin anywhere: 64 rows by each of two warps, four lanes to a row, 16-byte
        // words from the one that holds the chunk's first byte. (A bulk copy a row took 64 cycles each.)
        const int chunks = (p.kb + 7) / 8, first = 64 * (warp - 2) + (lane >> 2);
        const uint8_t* W = Swiglu && warp == 3 ? p.W2 : p.W;
        int buf = 0;
        uint32_t phase = 1, seen = 1;
        bool ok = true;
        for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
            const Tile at = locate<C::kBN>(L, p, t);
            int64_t from[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) from[j] = place_of<Swiglu>(p, at, first + 8 * j) + 16 * (lane & 3);
            for (int c = 0; c < chunks; ++c) {
                ok = finish(seen, &raw_empty[buf], phase);
                if (!ok) break;
                const uint32_t dst = base + C::kRaw + buf * C::kRawBytes + first * R::pitch + 16 * (lane & 3);
                if (from[7] + R::words * 16 <= p.total_bytes) {   // the lane's last row: all of them
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint8_t* src = W + (from[j] & ~int64_t(15));
#pragma unroll
                        for (int i = 0; i < R::words; i += 4)
                            if (i + 4 <= R::words || i + (lane & 3) < R::words)
                                copy16(dst + j * 8 * R::pitch + 16 * i, src + 16 * i);
                    }
                } else {   // the matrix may end inside a word, or before it
#pragma unroll 1
                    for (int j = 0; j < 8; ++j) {
                        const int64_t begin = (place_of<Swiglu>(p, at, first + 8 * j) + 16 * (lane & 3) +
                                               static_cast<int64_t>(c) * R::bytes) & ~int64_t(15);
#pragma unroll 1
                        for (int i = 0; i + (lane & 3) < R::words; i += 4) {
                            const int64_t left = p.total_bytes - (begin + 16 * i);
                            if (left > 0)
                                copy16(dst + j * 8 * R::pitch + 16 * i, W + begin + 16 * i,
                                       static_cast<int>(min(left, int64_t(16))));
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) from[j] += R::bytes;
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(&raw_full[buf]))
                             : "memory");
                if (++buf == C::kBufs) {
                    buf = 0;
                    phase ^= 1;
                }
                seen = peek(&raw_empty[buf], phase);
            }
        }
        if (!ok && lane == 0) report_status(p.status, kStatusTimeout);
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp >= 4 && warp < 12) {
        // Unpacking: 32 rows of each tile (the TMEM lanes that the warp may write); four warps have the
        // first 64 k of every stage, four the second.
        const int quarter = warp & 3, my_row = shared_row(Swiglu, quarter * 32 + lane);
        const int chunks = (p.kb + 7) / 8;
        const auto run = [&](auto which) {
            constexpr int H = decltype(which)::value;
            int buf = 0, it = 0;
            uint32_t phase = 1;   // of `done`: the first round passes at once
            uint32_t raw_phase = 0, seen_raw = 0;
            bool ok = true;
            for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
                [[maybe_unused]] int lead0 = 0;
                if (!Aligned) lead0 = static_cast<int>(place_of<Swiglu>(p, locate<C::kBN>(L, p, t), my_row) & 15);
                for (int c = 0; ok && c < chunks; ++c) {
                    ok = finish(seen_raw, &raw_full[buf], raw_phase);
                    if (!ok) break;
                    const uint32_t row = base + C::kRaw + buf * C::kRawBytes + my_row * R::pitch;
                    const uint32_t empty = smem_addr(&raw_empty[buf]);
                    if (++buf == C::kBufs) {
                        buf = 0;
                        raw_phase ^= 1;
                    }
                    seen_raw = peek(&raw_full[buf], raw_phase);
                    [[maybe_unused]] const int lead = (lead0 + c * R::bytes) & 15;
                    [[maybe_unused]] uint32_t sc[2], m[2];   // Q4_K: scales and mins of the super-block
                    [[maybe_unused]] float dd, dm, up_k;
                    float scale;
                    if constexpr (T == GQ_TYPE_Q4_K) {
                        const uint4 head = lds128(row);
                        // of sub-blocks 0..3 and 4..7, a byte each; their largest up to a factor of two by an OR
                        sc[0] = head.y & 0x3F3F3F3Fu;
                        sc[1] = (head.w & 0x0F0F0F0Fu) | ((head.y >> 2) & 0x30303030u);
                        m[0] = head.z & 0x3F3F3F3Fu;
                        m[1] = ((head.w >> 4) & 0x0F0F0F0Fu) | ((head.z >> 2) & 0x30303030u);
                        uint32_t sm = sc[0] | sc[1], mm = m[0] | m[1];
                        sm |= sm >> 16;
                        mm |= mm >> 16;
                        dd = half_bits_to_float(head.x);
                        dm = half_bits_to_float(head.x >> 16);
                        // codes times scales below 2^15, mins below 2^10
                        const float most = fmaxf(fabsf(dd) * static_cast<float>(((sm | sm >> 8) & 0xFFu) * 16),
                                                 fabsf(dm) * static_cast<float>(((mm | mm >> 8) & 0xFFu) * 32));
                        const int e = most > 0.0f ? exponent_of(most) : 14;
                        up_k = pow2f(14 - e);
                        scale = pow2f(e - 14);
                        if (!Few) dd *= pow2f(kLift<T>);
                    }
                    const auto stage = [&](auto half) {
                        constexpr int St = decltype(half)::value, S = 2 * St + H;   // S: 64 k of the chunk
                        const int blocks = p.kb - 8 * c - 4 * St;   // of this stage, from here on
                        if (blocks <= 0 || !ok) return;
                        const int slot = it & 1;
                        const uint32_t seen = peek(&done[slot], phase);
                        uint32_t h[2][16], l[2][16], mins[16];
                        [[maybe_unused]] float scales[2] = {}, least = 0.0f;   // Few: of the blocks, of Q4_K's mins
                        if constexpr (T == GQ_TYPE_Q4_K) {
                            const uint4 a = lds128(row + 16 + 32 * S), b = lds128(row + 32 + 32 * S);
                            const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
                            uint32_t sh[2], sl[2];
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const float sub = dd * static_cast<float>((sc[S >> 1] >> (16 * (S & 1) + 8 * i)) & 0xFFu);
                                if (Few) {
                                    scales[i] = sub;
                                    continue;
                                }
                                const float v = sub * up_k;
                                sh[i] = dup_half(v);
                                sl[i] = dup_half(v - half_bits_to_float(sh[i]));
                            }
#pragma unroll
                            for (int t8 = 0; t8 < 8; ++t8) {   // word 4 hi + t of both sub-blocks
                                uint32_t q[4];   // low nibbles of bytes 0, 2; high; low of 1, 3; high
                                nibbles_to_f16<0, Few ? 0 : kLift<T>>(w[t8], q);
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    const int i = j & 1, at = 4 * (t8 & 3) + 2 * (t8 >> 2) + (j >> 1);
                                    if (Few) {
                                        h[i][at] = q[j];
                                        continue;
                                    }
                                    h[i][at] = h2_mul(q[j], sh[i]);
                                    l[i][at] = h2_fma(q[j], sl[i], h2_fms(q[j], sh[i], h[i][at]));
                                }
                            }
                            if constexpr (S == 3 && Few) {   // the sums come times 2^-5, in two terms: the mins as they are
                                least = -32.0f * dm;
#pragma unroll
                                for (int g = 0; g < 4; ++g) {
                                    const uint32_t both = m[g >> 1] >> (16 * (g & 1));
                                    mins[g] = h2_sub((both & 0xFFu) | (both & 0xFF00u) << 8 | kMagic, kMagic);
                                    mins[4 + g] = 0;
                                }
                            } else if constexpr (S == 3) {   // the sums come times 2^-5
                                const float um = -32.0f * dm * up_k;
#pragma unroll
                                for (int g = 0; g < 4; ++g) {
                                    const float v0 = um * static_cast<float>((m[g >> 1] >> (16 * (g & 1))) & 0xFFu);
                                    const float v1 = um * static_cast<float>((m[g >> 1] >> (16 * (g & 1) + 8)) & 0xFFu);
                                    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(mins[g]) : "f"(v1), "f"(v0));
                                    const float r0 = v0 - half_bits_to_float(mins[g]);
                                    const float r1 = v1 - half_bits_to_float(mins[g] >> 16);
                                    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(mins[4 + g]) : "f"(r1), "f"(r0));
                                    mins[8 + g] = mins[g];
                                    mins[12 + g] = 0;
                                }
                            }
                        } else if constexpr (Few) {
                            StageWords<T, Aligned> words{};
                            words.template load<S>(row, lead);
                            codes_of<T, 0>(words.w, 0, h[0]);
                            codes_of<T, 0>(words.w, 1, h[1]);
                            scales[0] = half_bits_to_float(words.w[0]);
                            scales[1] = half_bits_to_float(words.w[R::bytes / 32] >> 16);
                        } else {
                            // the stage's other two scales stand beside this warp's; past the row's end: 0
                            StageWords<T, Aligned> words{};
                            words.template load<S>(row, lead);
                            constexpr int kPair = R::bytes / 4, kBlock = kPair / 2;
                            const uint32_t other = row + (Aligned && T != GQ_TYPE_MXFP4 ? 0 : lead) + (S ^ 1) * kPair;
                            float up[2];
                            if constexpr (T == GQ_TYPE_MXFP4) {
                                uint32_t s4[4] = {words.w[0] & 0xFFu, (words.w[4] >> 8) & 0xFFu, lds8(other),
                                                  lds8(other + kBlock)};
                                uint32_t top = 0;
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const int block = i < 2 ? 2 * H + i : 2 * (H ^ 1) + i - 2;
                                    if (s4[i] != 255u && block < blocks) top = max(top, s4[i]);
                                }
#pragma unroll
                                for (int i = 0; i < 2; ++i)
                                    up[i] = s4[i] == 255u ? __uint_as_float(0x7FC00000u)
                                                          : pow2f(max(static_cast<int>(s4[i] - top) + 12, -126));
                                scale = mx_scale(top) * pow2f(-12);
                            } else {
                                constexpr int kP = T == GQ_TYPE_Q4_0 ? 11 : 7;   // |c| <= 2^3, 2^7
                                const float d4[4] = {half_bits_to_float(words.w[0]),
                                                     half_bits_to_float(words.w[kBlock / 4] >> 16),
                                                     half_bits_to_float(lds16(other)),
                                                     half_bits_to_float(lds16(other + kBlock))};
                                float most = 0.0f;
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const int block = i < 2 ? 2 * H + i : 2 * (H ^ 1) + i - 2;
                                    if (block < blocks) most = fmaxf(most, fabsf(d4[i]));
                                }
                                const int e = most > 0.0f ? exponent_of(most) : kP;
                                up[0] = d4[0] * pow2f(kP + kLift<T> - e);
                                up[1] = d4[1] * pow2f(kP + kLift<T> - e);
                                scale = pow2f(e - kP);
                            }
#pragma unroll
                            for (int b = 0; b < 2; ++b) {
                                uint32_t q[16];
                                codes_of<T, kLift<T>>(words.w, b, q);
                                const uint32_t d = dup_half(up[b]);
#pragma unroll
                                for (int i = 0; i < 16; ++i) {
                                    h[b][i] = h2_mul(q[i], d);
                                    if (C::kTwo) l[b][i] = h2_fms(q[i], d, h[b][i]);
                                }
                            }
                        }
                        ok = finish(seen, &done[slot], phase);
                        if (!ok) return;
                        tc_fence_after();
                        const uint32_t to =
                            tmem + C::kA + slot * C::kACols + (static_cast<uint32_t>(quarter) << 21) + 32 * H;
                        tmem_st16(to, h[0]);
                        tmem_st16(to + 16, h[1]);
                        if (C::kTwo) {
                            tmem_st16(to + 64, l[0]);
                            tmem_st16(to + 80, l[1]);
                        }
                        if constexpr (T == GQ_TYPE_Q4_K && S == 3) tmem_st16(to + C::kMinA - 32, mins);   // from column kMinA on
                        const uint32_t ring =
                            base + C::kScales + ((it & (kScaleRing - 1)) * C::kUnits * kBM + quarter * 32 + lane) * 4;
                        if (Few) {
                            sts32(ring + 2 * H * kBM * 4, scales[0]);
                            sts32(ring + (2 * H + 1) * kBM * 4, scales[1]);
                            if (T == GQ_TYPE_Q4_K && S == 3) sts32(ring + 4 * kBM * 4, least);
                        } else if (H == 0) {
                            sts32(ring, scale);
                        }
                        tmem_st_wait();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_addr(&a_full[slot]));
                        ++it;
                        phase ^= slot;
                    };
                    stage(std::integral_constant<int, 0>());
                    stage(std::integral_constant<int, 1>());
                    if (Aligned) release_warp_to_async_proxy(0);   // every lane has used its words
                    else __syncwarp();
                    if (lane == 0) mbar_arrive(empty);
                }
            }
            if (!ok && lane == 0) report_status(p.status, kStatusTimeout);
        };
        if (warp < 8) run(std::integral_constant<int, 0>());
        else run(std::integral_constant<int, 1>());
    } else if (warp >= 12) {
        // Adding up: 32 rows, every second group of 16 columns. Few: all columns of every second pair of
        // blocks; at a tile's end the two warps of the same rows give each other what they have of the
        // other's columns.
        constexpr int kGroups = C::kBN / 32, kSums = Few ? 2 : kGroups;   // of 16 columns
        const int quarter = warp & 3, half = (warp - 12) >> 2;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter) << 21) + (Few ? 0 : 16 * half);
        const uint32_t scales = base + C::kScales + (quarter * 32 + lane) * 4;
        griddep_wait();   // the activations' scales
        int it = 0;
        uint32_t phase = 0, seen = 0;
        bool ok = true;   // Few: if not, the loops go on without waiting, for the two warps meet every tile
        for (int t = blockIdx.x; (Few || ok) && t < tiles; t += gridDim.x) {
            const Tile at = locate<C::kBN>(L, p, t);
            const int all = (at.n + 15) >> 4, groups = (all + 1 - half) >> 1;   // of 16 columns; this warp's
            __syncwarp();
#pragma unroll
            for (int i = lane; i < 64; i += 32)   // the tokens' scales, for the end
                if (i >> 4 < groups) x_scale[warp - 12][i] = p.xs[at.x_row + 16 * half + 32 * (i >> 4) + (i & 15)];
            uint64_t sum[kSums][8];
#pragma unroll
            for (int c = 0; c < kSums; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) sum[c][i] = 0;
            for (int s = 0; ok && s < stages; ++s) {
                const int slot = it & 1;
                ok = finish(seen, &done[slot], phase);
                if (!ok) break;
                tc_fence_after();
                const uint32_t ring = scales + (it & (kScaleRing - 1)) * (C::kUnits * kBM * 4);
                ++it;
                phase ^= slot;
                seen = peek(&done[slot ^ 1], phase);
                const uint32_t src = lanes + slot * C::kDCols;
                const auto add = [&](uint32_t (&r)[16], uint64_t (&to)[8], float d) {
                    const uint64_t dd = pack2(d, d);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        fma2(to[i], pack2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), dd);
                };
                if constexpr (Few) {
                    const int units = C::kMins ? 4 + (s & 1) : min(4, p.kb - 4 * s);
                    constexpr int kMine = 2 + C::kMins;   // blocks 2 half, 2 half + 1; Q4_K's mins (unit 4): half 1
                    float d[kMine];
#pragma unroll
                    for (int j = 0; j < kMine; ++j)
                        d[j] = lds_f32(ring + (j < 2 ? 2 * half + j : 4) * (kBM * 4));
#pragma unroll
                    for (int j = 0; j < kMine; ++j) {
                        const int u = j < 2 ? 2 * half + j : 4;
                        if (u >= units || (j == 2 && half == 0)) break;
                        uint32_t r[2][16];
                        tmem_ld16_async(src + u * C::kBN, r[0]);
                        if (all > 1) tmem_ld16_async(src + u * C::kBN + 16, r[1]);
                        tmem_wait16(r[0]);
                        add(r[0], sum[0], d[j]);
                        if (all > 1) {
                            tmem_wait16(r[1]);
                            add(r[1], sum[1], d[j]);
                        }
                    }
                } else {
                    const float d = lds_f32(ring);
#pragma unroll
                    for (int c = 0; c < kGroups; ++c) {
                        if (c < groups) {
                            uint32_t r[16];
                            tmem_ld16_async(src + 32 * c, r);
                            tmem_wait16(r);
                            add(r, sum[c], d);
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&d_empty[slot]));
            }
            if (!Few && !ok) break;
            if constexpr (Few) {
                // [warp][column][lane]; this warp's columns are sum[half]
                const uint32_t give = base + C::kSwap + ((warp - 12) * 16 * 32 + lane) * 4;
                const uint32_t take = base + C::kSwap + (((warp - 12) ^ 4) * 16 * 32 + lane) * 4;
                const auto both = [&](uint64_t (&mine)[8], uint64_t (&theirs)[8]) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float a, b;
                        asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(theirs[i]));
                        sts32(give + 2 * i * 128, a);
                        sts32(give + (2 * i + 1) * 128, b);
                    }
                    asm volatile("bar.sync %0, 64;" ::"r"(1 + quarter) : "memory");
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float a, b;
                        asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(mine[i]));
                        mine[i] = pack2(a + lds_f32(take + 2 * i * 128), b + lds_f32(take + (2 * i + 1) * 128));
                    }
                    asm volatile("bar.sync %0, 64;" ::"r"(1 + quarter) : "memory");
                };
                if (half == 0) {
                    both(sum[0], sum[1]);
                } else {
                    both(sum[1], sum[0]);
#pragma unroll
                    for (int i = 0; i < 8; ++i) sum[0][i] = sum[1][i];
                }
                if (!ok) continue;
            }
            __syncwarp();
            const int r = quarter * 32 + lane;
            const int m = Swiglu ? at.mt * (kBM / 2) + quarter * 16 + (lane & 15) : at.mt * kBM + r;
            const int mine = Swiglu ? lane >> 4 : 0;   // of two columns
            float* out = p.Y + (static_cast<int64_t>(at.row) + 16 * half + mine) * p.M + m;
            const int left = m < p.M ? at.n - 16 * half - mine : 0;   // columns from here on
            const int64_t next = 2 * static_cast<int64_t>(p.M);
            const auto columns = [&](const uint64_t (&v)[8], int c) {   // 16 of them
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float v0, v1;
                    asm("mov.b64 {%0, %1}, %2;" : "=f"(v0), "=f"(v1) : "l"(v[i]));
                    const float2 sc = *reinterpret_cast<const float2*>(&x_scale[warp - 12][16 * c + 2 * i]);
                    v0 *= sc.x;
                    v1 *= sc.y;
                    if (Swiglu) {   // lanes 0..15 hold gate rows, the others the up rows of the same numbers
                        const float other = __shfl_xor_sync(0xFFFFFFFFu, mine ? v0 : v1, 16);
                        const float h = swish(mine ? other : v0) * (mine ? v1 : other);
                        if (32 * c + 2 * i < left) out[0] = h;
                    } else {
                        if (32 * c + 2 * i < left) out[0] = v0;
                        if (32 * c + 2 * i + 1 < left) out[p.M] = v1;
                    }
                    out += next;
                }
                out += 8 * next;   // the other warp's 16
            };
#pragma unroll
            for (int c = 0; c < kGroups; ++c)
                if (c < groups) columns(sum[c], c);
        }
        if (!ok && lane == 0) report_status(p.status, kStatusTimeout);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

// ---- Launch --------------------------------------------------------------------------------

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled from the driver (nullptr if it has none).
EncodeTiledFn encode_fn() {
    static const EncodeTiledFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q{};
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                                               cudaEnableDefault, &q);
        return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? reinterpret_cast<EncodeTiledFn>(p) : nullptr;
    }();
    return fn;
}

// Rows of row_bytes bytes, boxes of 64 rows x `words` 16-byte words.
cudaError_t weight_map(const uint8_t* W, int64_t rows, int64_t row_bytes, int words, CUtensorMap* out) {
    const EncodeTiledFn enc = encode_fn();
    if (!enc) return cudaErrorNotSupported;
    const int unit = words > 16 ? 2 : 1;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(row_bytes / unit), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(row_bytes)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(words * 16 / unit), kBM / 2};
    const cuuint32_t steps[2] = {1, 1};
    const CUresult r = enc(out, unit == 2 ? CU_TENSOR_MAP_DATA_TYPE_UINT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
                           const_cast<uint8_t*>(W), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int T, bool Aligned, bool Swiglu, int F>
cudaError_t launch_product(GroupedParams& g, int64_t tiles, const DeviceInfo* info, cudaStream_t s) {
    auto kernel = grouped_kernel<T, Aligned, Swiglu, F>;
    constexpr int smem = Cfg<T, Aligned, F>::kSmem;
    if (Aligned) {
        const int64_t rows = static_cast<int64_t>(g.E) * g.M;
        cudaError_t e = weight_map(g.W, rows, g.row_bytes, Raw<T, Aligned>::words, &g.map);
        if (e == cudaSuccess && Swiglu) e = weight_map(g.W2, rows, g.row_bytes, Raw<T, Aligned>::words, &g.map2);
        if (e != cudaSuccess) return e;
    }
    static std::atomic<uint64_t> ready{0};   // devices whose attribute is set
    const uint64_t bit = uint64_t(1) << info->device;
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    return launch_after(kernel, dim3(static_cast<unsigned>(std::min<int64_t>(tiles, info->sm_count))), kThreads, smem, s,
                        g);
}

// The instances of one type.
template <int T>
cudaError_t launch_type(GroupedParams& g, const GroupedLaunch& l, const DeviceInfo* info, cudaStream_t s) {
    const auto form = [&](auto aligned, auto swiglu) {
        constexpr bool A = decltype(aligned)::value, S = decltype(swiglu)::value;
        if constexpr (T != GQ_TYPE_MXFP4)
            if (l.form == kFewRows) return launch_product<T, A, S, kFewRows>(g, l.tiles, info, s);
        return l.form == kManyRows ? launch_product<T, A, S, kManyRows>(g, l.tiles, info, s)
                                   : launch_product<T, A, S, kSomeRows>(g, l.tiles, info, s);
    };
    if constexpr (T != GQ_TYPE_Q4_K)
        if (!l.aligned)
            return l.swiglu ? form(std::false_type(), std::true_type()) : form(std::false_type(), std::false_type());
    return l.swiglu ? form(std::true_type(), std::true_type()) : form(std::true_type(), std::false_type());
}

}  // namespace
}  // namespace gq
