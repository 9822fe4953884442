// gq_few.cu -- block-quantized weights times a few fp32 tokens, to fp32 accuracy: the MXFP4
// mul_mat and the two weight passes of the mixture-of-experts layer.
//
// Mathematics. A weight row's block is d (q - z) with small integers q (or E2M1 values), so
//     sum_k What[m][k] x[k] = sum_b d_b s_b sum_{k in b} (q_k - z) xs_k
// with xs = x / s split in two fp16 terms (gq_few.cuh). The inner sum runs on the tensor
// cores: mma.m16n8k16 with 16 weight rows as exact fp16 codes and 8 tokens as columns, four
// instructions a block (two halves of k, hi and lo into the same fp32 accumulators); the outer
// sum is one fp32 multiply-add per block, row and token (Q4_K: per super-block, see super_block).
// Nothing is rounded below 22 bits but the fp32 sums.
//
// What bounds it. One pass over the weights: 17 to 34 bytes per 32 weights from DRAM, 35 to 55
// instructions per 16 rows x 32 weights x 8 tokens. At 6.8 TB/s an SM takes in 512 4-bit weights
// every 12 cycles, 48 issue slots, so with issue slots half filled instructions and the latencies
// between them come before memory as the limit: 304 CTAs of 8 warps (128 registers) issue in 38 %
// (Q8_0: the shared-memory queue) to 53 % (Q4_K) of the cycles, tensor cores are at 12 to 18 %,
// DRAM at 20 to 35 %. Measured, as a graph on a GB300: 32000 x 2048 MXFP4 times 13 tokens is
// 23.0 us (5.4 us of bytes), an expert layer of 16 tokens over 64 Q8_0 experts 98 us (38), of 61
// tokens over 64 Q4_K experts 148 us (33), of 4 tokens over 16 of 32 MXFP4 experts 39 us (9).
// Next to it the instruction cache: forms of this kernel with all loops unrolled (70 to 150 KB of
// code) lost 4 to 10 us a launch, so loops stay rolled, what is rare is not inlined, and the number
// of column tiles is the kernel's, not a branch's. tcgen05 is not used: its operands would have to
// pass through shared memory once more, fp16 scales would have to be applied outside, and its
// 128-row tiles leave most SMs without work here. (The microscaled product, whose scales the
// tensor cores apply, does use it: gq_mx.cu.)
// More tokens than one group: every group unpacks the weights again (from L2), so prompts cost in
// proportion, far from their bytes: 32000 x 2048 MXFP4 times 512 tokens 479 us (35 of operations and
// bytes), 512 tokens over 64 Q4_K experts, 8 each, in 8 passes 1220 us.
//
// Layout of the work. A unit is (a group of up to 8 NT tokens, 32 result rows); a row warp has a
// run of consecutive units, so that those of one group follow each other and share activations
// through L1. Where there are too few units, 2, 4 or 8 warps split a unit's K and join through
// shared memory in a fixed order; they wait for each other, nobody else does. Every warp runs
// its own ring of 16-byte asynchronous copies, four lanes to a weight row: a row's chunk from
// the word that holds its first byte, because rows of 17- and 18-byte blocks start anywhere; the
// words are aligned in registers. The ring runs on across units, and weights do not depend on
// the kernel before, so they start to stream before griddepcontrol.wait. (They, and ids, come
// from before the call: the split kernel, which every call begins with, waits for all that came
// before it on the stream, and only then lets this kernel start.)
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstddef>

#include "gq_few.cuh"

namespace gq {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kStages = 2;

constexpr int64_t kFewMaxTokens = 4096;   // of one launch: bounds the workspace

enum Mode { kDense = 0, kGateUp = 1, kDown = 2 };

template <int T>
struct Fmt;   // bytes of 32 weights, blocks per chunk, shared-memory pitch of a row's chunk
template <>
struct Fmt<GQ_TYPE_Q4_0> {
    static constexpr int bb = kQ4Bytes, cb = 8, pitch = 176;
};
template <>
struct Fmt<GQ_TYPE_Q8_0> {
    static constexpr int bb = kQ8Bytes, cb = 4, pitch = 160;
};
template <>
struct Fmt<GQ_TYPE_Q4_K> {   // a super-block's bytes over its 8 sub-blocks
    static constexpr int bb = kQ4KBytes / 8, cb = 8, pitch = 144;
};
template <>
struct Fmt<GQ_TYPE_MXFP4> {
    static constexpr int bb = kMxfp4Bytes, cb = 8, pitch = 176;
};
// Pitches: a chunk is 136 or 144 bytes and starts up to 15 bytes into its first 16-byte word;
// 176 = 44 words puts the eight rows that a warp reads at once on eight distinct groups of four
// banks, as 144 = 36 words does where rows are always aligned (Q4_K).

struct Params {
    const uint8_t* W;
    const uint8_t* W2;        // kGateUp: the up matrices
    int64_t total_bytes;      // of W (and of W2)
    int64_t row_bytes;
    int rows;                 // weight rows (of one expert)
    int kb;                   // 32-weight blocks per row
    int chunks;
    int tiles;                // 32-row tiles: ceil(rows / 32)
    int kshift;               // log2 of the warps that split a unit's K
    const uint4* xb;          // split activations, 64 bytes per (row, block, term)
    const float* xs;          // their scales: per row (two terms but for kDown), else per block
    const float* xsum;        // Q4_K: their sums per block
    int N;                    // tokens
    int E, top_k, pairs;
    const int* ids;
    float* out;               // kDense: Y; kDown: [pair][rows]
    __half* hb;               // kGateUp: split activations of the result,
    float* hs;                //          scales and sums per block
    float* hsum;
    int h_type;               //          in the order of the down matrices' type
};

// 16 bytes global -> shared, of which the first n (1..16) are read and the others zero.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int n) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
    unsigned short v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(a));
    return v;
}

// 32 bytes at once: the two terms of a lane's eight activations. A warp's eight tokens are eight
// cache lines, and 16-byte loads of hi and lo would visit each twice.
__device__ __forceinline__ void load32(uint4 (&v)[2], const uint4* at) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v[0].x), "=r"(v[0].y), "=r"(v[0].z), "=r"(v[0].w), "=r"(v[1].x), "=r"(v[1].y),
                   "=r"(v[1].z), "=r"(v[1].w)
                 : "l"(at));
}

// c = A (16 weight rows x 16) . B (16 x 8 columns), then c += for the block's second half.
__device__ __forceinline__ void mma_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void mma_next(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two E8M0 scale bytes to fp32 (255: NaN; 0: the subnormal 2^-127).
__device__ __forceinline__ void e8m0_to_f32(uint32_t lo, uint32_t hi, float& dlo, float& dhi) {
    uint32_t r;
    const unsigned short both = static_cast<unsigned short>(lo | (hi << 8));
    asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(r) : "h"(both));
    dlo = __uint_as_float(r << 16);
    dhi = __uint_as_float(r & 0xFFFF0000u);
}

// fp16 arithmetic on pairs: 1024 + u lies in an fp16 word as 0x6400 | u, so integers become
// fp16 by a mask and one exact subtraction. (Integers left as subnormal fp16 would save the
// subtraction, but the tensor cores align products by their nominal exponents: sums then lose
// the subnormals' leading zeros, measured as 6e-6 of the result instead of 3e-7.)
__device__ __forceinline__ uint32_t h2_sub(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t h2_fma(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
__device__ __forceinline__ uint32_t h2_mul(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
constexpr uint32_t kMagic = 0x64006400u;       // 1024
constexpr uint32_t kSixteenth = 0x2C002C00u;   // 1/16

// The eight 4-bit codes of a word minus Z (0 or 8), as fp16 pairs (bits 0 and 16), (4 and 20),
// (8 and 24), (12 and 28).
template <int Z>
__device__ __forceinline__ void nibbles_to_f16(uint32_t w, uint32_t (&h)[4]) {
    constexpr uint32_t kLow = Z == 8 ? 0x64086408u : 0x64006400u;     // 1024 + Z
    constexpr uint32_t kHigh = Z == 8 ? 0xD480D480u : 0xD400D400u;    // -(64 + Z)
    const uint32_t v = w >> 8;
    h[0] = h2_sub((w & 0x000F000Fu) | kMagic, kLow);
    h[1] = h2_fma((w & 0x00F000F0u) | kMagic, kSixteenth, kHigh);
    h[2] = h2_sub((v & 0x000F000Fu) | kMagic, kLow);
    h[3] = h2_fma((v & 0x00F000F0u) | kMagic, kSixteenth, kHigh);
}

// Four E2M1 pairs (one byte each: low nibble, high nibble) to four fp16 pairs, exact.
__device__ __forceinline__ void e2m1_to_f16(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

// One block's activations in this lane.
template <int NT, int Terms>
struct Columns {
    uint4 b[NT][Terms];        // eight fp16 of column g, hi and lo
    float2 s[NT];              // scales of tokens 2t, 2t + 1, where there are any per block
};

// c (+)= products of one 16-row tile with one term of one block's activations, for NT tiles of 8
// tokens: rows g, g + 8 x tokens 2t, 2t + 1.
template <bool First, int Terms, int NT>
__device__ __forceinline__ void term_products(const uint32_t (&q)[2][4], const Columns<NT, Terms>& col, int term,
                                              float (&c)[NT][4]) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        if (First)
            mma_first(c[n], q[0][0], q[1][0], q[0][1], q[1][1], col.b[n][term].x, col.b[n][term].y);
        else
            mma_next(c[n], q[0][0], q[1][0], q[0][1], q[1][1], col.b[n][term].x, col.b[n][term].y);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
        mma_next(c[n], q[0][2], q[1][2], q[0][3], q[1][3], col.b[n][term].z, col.b[n][term].w);
}

// Both terms, the small one first: the tensor cores cut a sum off below the last bit of its
// largest part (they do not round it), which costs the more the more often a sum of full size
// passes through them.
template <int Terms, int NT>
__device__ __forceinline__ void block_products(const uint32_t (&q)[2][4], const Columns<NT, Terms>& col,
                                               float (&c)[NT][4]) {
    if constexpr (Terms == 2) {
        term_products<true>(q, col, 1, c);
        term_products<false>(q, col, 0, c);
    } else {
        term_products<true>(q, col, 0, c);
    }
}

// The shared lists of a launch over experts: pairs sorted by expert, and groups of pairs of one
// expert.
struct Lists {
    uint16_t pair[kMoeMaxPairs], token[kMoeMaxPairs];
    uint16_t expert[kMoeMaxPairs], start[kMoeMaxPairs];
    uint8_t count[kMoeMaxPairs];
    int groups;
};

// Sorts the pairs by expert, in their own order inside an expert: every CTA has to find the
// same groups. ids outside [0, E) are in no group. `scratch`: kMoeMaxExperts + kMoeMaxPairs
// ints. One warp ranks 32 pairs at a time by matching their ids; 512 pairs are 16 steps.
__device__ __noinline__ void build_lists(const int* __restrict__ all_ids, int E, int top_k, int pairs, int group,
                                         Lists& L, int* scratch) {
    int* count = scratch;
    int* ids = scratch + kMoeMaxExperts;
#pragma unroll 1
    for (int e = threadIdx.x; e < E; e += kThreads) count[e] = 0;
#pragma unroll 1
    for (int q = threadIdx.x; q < pairs; q += kThreads) {
        const int id = all_ids[q];
        ids[q] = id >= 0 && id < E ? id : -1;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        const unsigned below = (1u << threadIdx.x) - 1u;
#pragma unroll 1
        for (int q0 = 0; q0 < pairs; q0 += 32) {
            const int q = q0 + threadIdx.x;
            const int id = q < pairs ? ids[q] : -1;
            const unsigned same = __match_any_sync(0xFFFFFFFFu, id);
            const int before = id >= 0 ? count[id] : 0;
            __syncwarp();
            if (id >= 0) {
                if ((same & below) == 0) count[id] = before + __popc(same);
                ids[q] = id | ((before + __popc(same & below)) << 16);   // id < 1024, rank < 512
            }
            __syncwarp();
        }
        // exclusive sums over the experts: pairs (low half) and groups (high half)
        int base = 0;
#pragma unroll 1
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + threadIdx.x;
            const int c = e < E ? count[e] : 0;
            const int g = (c + group - 1) / group;
            int incl = c | (g << 16);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(0xFFFFFFFFu, incl, o);
                if (static_cast<int>(threadIdx.x) >= o) incl += up;
            }
            const int excl = base + incl - (c | (g << 16));
            const int pair0 = excl & 0xFFFF, group0 = excl >> 16;
#pragma unroll 1
            for (int i = 0; i < g; ++i) {
                L.expert[group0 + i] = static_cast<uint16_t>(e);
                L.start[group0 + i] = static_cast<uint16_t>(pair0 + i * group);
                L.count[group0 + i] = static_cast<uint8_t>(min(group, c - i * group));
            }
            if (e < E) count[e] = pair0;
            base += __shfl_sync(0xFFFFFFFFu, incl, 31);
        }
        if (threadIdx.x == 0) L.groups = base >> 16;
    }
    __syncthreads();
#pragma unroll 1
    for (int q = threadIdx.x; q < pairs; q += kThreads)
        if (ids[q] >= 0) {
            const int at = count[ids[q] & 0xFFFF] + (ids[q] >> 16);
            L.pair[at] = static_cast<uint16_t>(q);
            L.token[at] = static_cast<uint16_t>(q / top_k);
        }
    __syncthreads();
}

// The split of one block of an activation row, held by a warp or by 8 lanes of it: scale
// exponent of a maximum over them, and an element's two terms.
struct Split {
    __half hi, lo;
    __device__ __forceinline__ Split(float x, int e) {
        const float xs = x * pow2f(14 - e);
        hi = __float2half_rn(xs);
        lo = __float2half_rn(xs - __half2float(hi));
    }
    __device__ __forceinline__ float sum() const { return __half2float(hi) + __half2float(lo); }
};

template <int T, int M, int Terms, int NT>
struct Worker {
    static constexpr int kBB = Fmt<T>::bb, kCB = Fmt<T>::cb, kPitch = Fmt<T>::pitch;
    static constexpr int kStageBytes = 32 * kPitch + 16;      // the last word's second half
    static constexpr int kWords = T == GQ_TYPE_Q4_K ? 9 : 10;   // 16-byte words of a row's chunk
    static constexpr int kGroup = 8 * NT;
    static constexpr bool kScaled = M == kDown || Terms == 1;   // scales per block, not per row
    static constexpr bool kSums = T == GQ_TYPE_Q4_K;
    static constexpr int kSub = M == kGateUp ? 2 : 1;   // a unit's passes: 16 gate and 16 up rows each
    static constexpr int kTotals = 2 * NT * 4;   // a lane's, of one pass
    // Blocks whose activations are in registers ahead of their use: they come from L1 or L2, and a
    // warp, one of four on its scheduler, is at a block for some 130 to 250 cycles. Four fit the
    // registers with one column tile, two with two.
    static constexpr int kDepth = NT == 1 ? 4 : 2;
    static constexpr int kRingBytes = kWarps * kStages * kStageBytes;
    static constexpr int kSumBytes = kWarps * kTotals * 32 * 4;
    static constexpr int kListBytes = M == kDense ? 0 : static_cast<int>(sizeof(Lists));
    static constexpr int kSmem = kRingBytes + kSumBytes + kListBytes;
    static_assert((kMoeMaxExperts + kMoeMaxPairs) * 4 <= kRingBytes, "the lists' scratch lies in the ring");
    using Cols = Columns<NT, Terms>;

    const Params& p;
    const Lists& L;
    uint32_t ring;      // this warp's, shared address
    float* sums;        // the CTA's
    int lane, wk, wr, kwarps;
    // the next chunk to copy: unit (group, tile, how many are left), pass, chunk; stage
    int fgi, ftile, fleft, fs, fc, fstage;
    int64_t fbyte;      // where its first weight row begins

    __device__ __forceinline__ int expert_of(int gi) const { return M == kDense ? 0 : L.expert[gi]; }
    __device__ __forceinline__ int count_of(int gi) const {
        return M == kDense ? min(kGroup, p.N - gi * kGroup) : L.count[gi];
    }
    // activation row of column token i of a group
    __device__ __forceinline__ int x_row(int gi, int i) const {
        if (M == kDense) return gi * kGroup + i;
        return M == kGateUp ? L.token[L.start[gi] + i] : L.pair[L.start[gi] + i];
    }

    __device__ __forceinline__ void copy_row() {
        fbyte = (static_cast<int64_t>(expert_of(fgi)) * p.rows + ftile * 32 + fs * 16) * p.row_bytes;
    }

    // Starts the copies of the next chunk (if any), as one group. Staged row 8 j + g
    // (g = lane / 4) is row 8 j + g of the warp's 32 (kGateUp: of the 16 gate rows, then of the
    // up rows of the same numbers). Whole words from the one that holds the chunk's first byte;
    // what they hold behind the chunk is not used.
    __device__ __forceinline__ void issue() {
        if (fleft > 0) {
            const int l = lane & 3;
            const int64_t chunk = fbyte + static_cast<int64_t>(fc) * (kCB * kBB);
            const uint32_t dst = ring + fstage * kStageBytes + (lane >> 2) * kPitch + 16 * l;
            if (p.rows - ftile * 32 >= 32 && chunk + 31 * p.row_bytes + 16 * kWords <= p.total_bytes) {
                int64_t at = chunk + (lane >> 2) * p.row_bytes;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (M == kGateUp && j == 2) at -= 16 * p.row_bytes;
                    const uint8_t* from = (M == kGateUp && j >= 2 ? p.W2 : p.W) + ((at & ~int64_t(15)) + 16 * l);
                    copy16(dst + j * 8 * kPitch, from);
                    copy16(dst + j * 8 * kPitch + 64, from + 64);
                    if (l < kWords - 8) copy16(dst + j * 8 * kPitch + 128, from + 128);
                    at += 8 * p.row_bytes;
                }
            } else {
                issue_last(chunk, dst, l);
            }
            fc += kwarps;
            if (fc >= p.chunks) {
                fc = wk;
                if (++fs == kSub) {
                    fs = 0;
                    --fleft;
                    if (++ftile == p.tiles) {
                        ftile = 0;
                        ++fgi;
                    }
                }
                if (fleft > 0) copy_row();
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        fstage ^= 1;
    }

    // The same where rows are missing or the buffer ends: no byte past either is read.
    __device__ __forceinline__ void issue_last(int64_t chunk, uint32_t dst, int l) const {
#pragma unroll 1
        for (int j = 0; j < 4; ++j) {
            const int r = (M == kGateUp ? j & 1 : j) * 8 + (lane >> 2);
            const int64_t from = (chunk + r * p.row_bytes) & ~static_cast<int64_t>(15);
            const int left = fs * 16 + r < p.rows - ftile * 32
                                 ? static_cast<int>(min(p.total_bytes - from, static_cast<int64_t>(16 * kWords))) : 0;
            const uint8_t* src = (M == kGateUp && j >= 2 ? p.W2 : p.W) + from;
#pragma unroll 1
            for (int i = l; 16 * i < left; i += 4)
                copy16(dst + j * 8 * kPitch + 16 * (i - l), src + 16 * i, min(16, left - 16 * i));
        }
    }

    // A unit's activations: where this lane's next block is, moved on with every load.
    struct Acts {
        const uint4* b[NT];
        const float* s[NT][2];
        const float2* sum[NT];   // Q4_K: the sums of sub-blocks 2t, 2t + 1 for token g
    };

    // The block at hand, and on to the one `step` blocks later.
    __device__ __forceinline__ void load(Cols& c, Acts& a, int step) const {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if constexpr (Terms == 2)
                load32(c.b[n], a.b[n]);
            else
                c.b[n][0] = *a.b[n];
            a.b[n] += step * 4 * Terms;
            if constexpr (kScaled) {
                c.s[n] = make_float2(*a.s[n][0], *a.s[n][1]);
                a.s[n][0] += step;
                a.s[n][1] += step;
            }
        }
    }

    // The codes and scales of one block of the 32 staged rows, as they are.
    struct Raw {
        uint32_t w[2][2][T == GQ_TYPE_Q8_0 ? 2 : 1], d[2][2];
    };

    // The block whose first byte lies `pos` bytes into every row. Rows agree in the low two bits
    // of their places (eight rows are a multiple of 8 bytes): the aligned word before a code
    // word, and the shift that takes the word out of two.
    __device__ __forceinline__ void fetch(Raw& x, const uint32_t (&base)[2][2], int pos) const {
        if constexpr (T == GQ_TYPE_Q8_0) {
            // bytes 8t..8t+7: out of two aligned 8-byte words (a lane's four rows, 8 apart, agree
            // in the low four bits of their places)
            const uint32_t first = base[0][0] + pos + 2 + 8 * (lane & 3);
            const bool odd = first & 4u;
            const int off = static_cast<int>((first & ~7u) - base[0][0]);
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint2 a = lds64(base[mt][h] + off), b = lds64(base[mt][h] + off + 8);
                    const uint32_t mid = odd ? b.x : a.y;
                    x.w[mt][h][0] = __funnelshift_r(odd ? a.y : a.x, mid, first << 3);
                    x.w[mt][h][1] = __funnelshift_r(mid, odd ? b.y : b.x, first << 3);
                    x.d[mt][h] = lds16(base[mt][h] + pos);
                }
            return;
        }
        constexpr int kHead = T == GQ_TYPE_MXFP4 ? 1 : 2;
        const uint32_t r = (base[0][0] + pos + kHead) & 3u;
        const int off = pos + kHead - static_cast<int>(r) + 4 * (lane & 3);
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t at = base[mt][h] + off;
                x.w[mt][h][0] = __funnelshift_r(lds32(at), lds32(at + 4), r << 3);
                x.d[mt][h] = T == GQ_TYPE_MXFP4 ? lds8(base[mt][h] + pos) : lds16(base[mt][h] + pos);
            }
    }

    __device__ __forceinline__ void multiply(float (&tot)[2][NT][4], const Raw& x, const Cols& col) const {
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
            uint32_t q[2][4];
            float d[2], c[NT][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if constexpr (T == GQ_TYPE_Q8_0) {
                    const uint32_t u0 = x.w[mt][h][0] ^ 0x80808080u, u1 = x.w[mt][h][1] ^ 0x80808080u;
                    // 1024 + 128 + code, byte by byte under the exponent
                    q[h][0] = h2_sub(__byte_perm(u0, 0x64u, 0x4140), 0x64806480u);
                    q[h][1] = h2_sub(__byte_perm(u0, 0x64u, 0x4342), 0x64806480u);
                    q[h][2] = h2_sub(__byte_perm(u1, 0x64u, 0x4140), 0x64806480u);
                    q[h][3] = h2_sub(__byte_perm(u1, 0x64u, 0x4342), 0x64806480u);
                } else if constexpr (T == GQ_TYPE_Q4_0) {
                    nibbles_to_f16<8>(x.w[mt][h][0], q[h]);
                } else {
                    e2m1_to_f16(x.w[mt][h][0], q[h]);
                }
                if constexpr (T != GQ_TYPE_MXFP4) d[h] = half_bits_to_float(x.d[mt][h]);
            }
            if constexpr (T == GQ_TYPE_MXFP4) e8m0_to_f32(x.d[mt][0], x.d[mt][1], d[0], d[1]);
            block_products<Terms, NT>(q, col, c);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    tot[mt][n][i] = fmaf(kScaled ? d[i >> 1] * (i & 1 ? col.s[n].y : col.s[n].x) : d[i >> 1],
                                         c[n][i], tot[mt][n][i]);
        }
    }

    // Q4_K: the eight sub-blocks of a super-block, columns loaded ahead as in the other types.
    //     sum_j (d sc_j sum q x - dmin m_j sum x) = d sum_j sum (sc_j q) x - dmin sum_j m_j X_j
    // sc_j q, at most 63 x 15, is an exact fp16 integer and costs no instruction: codes under the
    // exponent of 1024 become sc_j q by one multiply-add. So with one activation scale a row the
    // products of two sub-blocks chain in the accumulators and add to the super-block's; with one a
    // sub-block (kDown) each sub-block's are added under its scale. (Chains of all eight: 1.3e-6
    // off in 61 tokens over 64 experts against 5e-7, at 144 us against 148.) The mins are one more
    // product: m_j in k = j and k = 8 + j, with the two terms of the sub-blocks' sums X_j. (A scale
    // and a min multiply-add for every sub-block, row and token: 56 instructions a sub-block and 16
    // rows instead of 37, 173 us.)
    __device__ __forceinline__ void super_block(float (&tot)[2][NT][4], const uint32_t (&base)[2][2],
                                                Cols (&col)[kDepth], Acts& acts, int jump) const {
        const int t = lane & 3;
        float2 sums[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            sums[n] = *acts.sum[n];
            acts.sum[n] += kwarps * (kCB / 2);
        }
        float acc[2][NT][4];
#pragma unroll
        for (int i = 0; i < kTotals; ++i) (&acc[0][0][0])[i] = 0.0f;
#pragma unroll 1
        for (int b = 0; b < kCB; b += kDepth) {
            const int step = (b + 2 * kDepth) % kCB ? 1 : jump;   // past a chunk's end
            uint32_t scales[2][2];   // byte i: of sub-block b + i
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint4 hd = lds128(base[mt][h]);
                    const uint32_t s = b & 4 ? (hd.w & 0x0F0F0F0Fu) | ((hd.y >> 2) & 0x30303030u) : hd.y & 0x3F3F3F3Fu;
                    scales[mt][h] = kDepth == 4 ? s : s >> (8 * (b & 2));
                }
#pragma unroll
            for (int i = 0; i < kDepth; i += 2) {
#pragma unroll
                for (int mt = 0; mt < 2; ++mt) {
                    uint32_t q[2][2][4];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t at = base[mt][h] + 16 + 16 * (b + i) + 4 * t;
                        const uint32_t w0 = lds32(at), w1 = lds32(at + 16), v0 = w0 >> 8, v1 = w1 >> 8;
                        const uint32_t s0 = h2_sub(__byte_perm(scales[mt][h], 0x64u, 0x4040 | i * 0x101), kMagic);
                        const uint32_t s1 = h2_sub(__byte_perm(scales[mt][h], 0x64u, 0x4040 | (i + 1) * 0x101), kMagic);
                        // low nibbles: (1024 + q) s - 1024 s; high: (1024 + 16 q) s / 16 - 64 s
                        const uint32_t z0 = h2_mul(s0, 0xE400E400u), f1 = h2_mul(s1, kSixteenth), z1 = h2_mul(s1, 0xD400D400u);
                        q[0][h][0] = h2_fma((w0 & 0x000F000Fu) | kMagic, s0, z0);
                        q[0][h][1] = h2_fma((v0 & 0x000F000Fu) | kMagic, s0, z0);
                        q[0][h][2] = h2_fma((w1 & 0x000F000Fu) | kMagic, s0, z0);
                        q[0][h][3] = h2_fma((v1 & 0x000F000Fu) | kMagic, s0, z0);
                        q[1][h][0] = h2_fma((w0 & 0x00F000F0u) | kMagic, f1, z1);
                        q[1][h][1] = h2_fma((v0 & 0x00F000F0u) | kMagic, f1, z1);
                        q[1][h][2] = h2_fma((w1 & 0x00F000F0u) | kMagic, f1, z1);
                        q[1][h][3] = h2_fma((v1 & 0x00F000F0u) | kMagic, f1, z1);
                    }
                    float c[NT][4];
                    if constexpr (kScaled) {
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const Cols& x = col[i + k];
                            block_products<Terms, NT>(q[k], x, c);
#pragma unroll
                            for (int n = 0; n < NT; ++n)
#pragma unroll
                                for (int r = 0; r < 4; ++r)
                                    acc[mt][n][r] = fmaf(r & 1 ? x.s[n].y : x.s[n].x, c[n][r], acc[mt][n][r]);
                        }
                    } else {
                        term_products<true>(q[0], col[i], 1, c);
                        term_products<false>(q[1], col[i + 1], 1, c);
                        term_products<false>(q[0], col[i], 0, c);
                        term_products<false>(q[1], col[i + 1], 0, c);
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int r = 0; r < 4; ++r) acc[mt][n][r] += c[n][r];
                    }
                }
                load(col[i], acts, 1);
                load(col[i + 1], acts, i + 2 < kDepth ? 1 : step);
            }
        }
        // the sums in two terms: in units of 32 where the row has one scale (a sum is below 2^20),
        // else in units of a power of two of the super-block
        uint32_t hi[NT], lo[NT];
        float2 unit[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float f = 1.0f / 32.0f;
            unit[n] = make_float2(32.0f, 32.0f);
            if constexpr (kScaled) {
                uint32_t most = max(__float_as_uint(sums[n].x) & 0x7FFFFFFFu, __float_as_uint(sums[n].y) & 0x7FFFFFFFu);
                most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
                most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
                const int e = block_exponent(most);
                const float u = pow2f(e - 14);   // of token g; the totals' tokens are 2t, 2t + 1
                f = pow2f(14 - e);
                unit[n] = make_float2(__shfl_sync(0xFFFFFFFFu, u, 8 * t), __shfl_sync(0xFFFFFFFFu, u, 8 * t + 4));
            }
            const float x = sums[n].x * f, y = sums[n].y * f;
            const __half2 a = __floats2half2_rn(x, y);
            const __half2 b = __floats2half2_rn(x - __low2float(a), y - __high2float(a));
            hi[n] = reinterpret_cast<const uint32_t&>(a);
            lo[n] = reinterpret_cast<const uint32_t&>(b);
        }
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
            uint32_t m[2];
            float d[2], dmin[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint4 hd = lds128(base[mt][h]);
                const uint32_t mins = t & 2 ? ((hd.w >> 4) & 0x0F0F0F0Fu) | ((hd.z >> 2) & 0x30303030u) : hd.z & 0x3F3F3F3Fu;
                m[h] = h2_sub(__byte_perm(mins, 0x64u, t & 1 ? 0x4342 : 0x4140), kMagic);
                d[h] = half_bits_to_float(hd.x);
                dmin[h] = half_bits_to_float(hd.x >> 16);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float z[4];
                mma_first(z, m[0], m[1], m[0], m[1], hi[n], lo[n]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    tot[mt][n][i] = fmaf(d[i >> 1], acc[mt][n][i], tot[mt][n][i]);
                    tot[mt][n][i] = fmaf(-dmin[i >> 1] * (i & 1 ? unit[n].y : unit[n].x), z[i], tot[mt][n][i]);
                }
            }
        }
    }

    __device__ __forceinline__ void unit(int gi, int tile, int& stage) {
        const int n_tok = count_of(gi);
        const int g = lane >> 2, t = lane & 3;
        const uint32_t e_row = static_cast<uint32_t>(expert_of(gi)) * static_cast<uint32_t>(p.rows) + tile * 32;
        // kGateUp: the unit's hidden values, [token][row], in this warp's part of the sums
        float* const hidden = sums + wr * kwarps * kTotals * 32;
#pragma unroll 1
        for (int s = 0; s < kSub; ++s) {
            // Columns of tokens that the group does not have read token 0's: nothing uses them.
            // Loads run ahead, past a row's end by up to kAhead blocks: the workspace goes on.
            Acts acts;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                acts.b[n] = p.xb + (static_cast<int64_t>(x_row(gi, 8 * n + g < n_tok ? 8 * n + g : 0)) * p.kb + wk * kCB) * 4 * Terms + t * Terms;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int tok = 8 * n + 2 * t + i;
                    const int64_t at = static_cast<int64_t>(x_row(gi, tok < n_tok ? tok : 0)) * p.kb + wk * kCB;
                    if constexpr (kScaled) acts.s[n][i] = p.xs + at;
                }
                if constexpr (kSums)
                    acts.sum[n] = reinterpret_cast<const float2*>(
                        p.xsum + static_cast<int64_t>(x_row(gi, 8 * n + g < n_tok ? 8 * n + g : 0)) * p.kb + wk * kCB + 2 * t);
            }
            float tot[2][NT][4];
#pragma unroll
            for (int i = 0; i < kTotals; ++i) (&tot[0][0][0])[i] = 0.0f;
            Cols col[kDepth];
            const int jump = (kwarps - 1) * kCB + 1;   // from a chunk's last block to the next's first
#pragma unroll
            for (int i = 0; i < kDepth; ++i) load(col[i], acts, (i + 1) % kCB ? 1 : jump);
#pragma unroll 1
            for (int c = wk; c < p.chunks; c += kwarps) {
                asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
                __syncwarp();
                const int nb = min(kCB, p.kb - c * kCB);
                // Where this lane's rows begin inside their staged words (0..15).
                uint32_t base[2][2];
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t row = e_row + (M == kGateUp ? 16 * s + 8 * h + g : 16 * mt + 8 * h + g);
                        base[mt][h] = ring + stage * kStageBytes + (16 * mt + 8 * h + g) * kPitch +
                                      ((row * static_cast<uint32_t>(p.row_bytes) + static_cast<uint32_t>(c) * (kCB * kBB)) & 15u);
                    }
                // A column set is loaded again as soon as it has been used; codes are fetched a
                // block ahead (behind the chunk: bytes of the stage that are not used).
                if constexpr (T == GQ_TYPE_Q4_K) {
                    super_block(tot, base, col, acts, jump);
                } else {
                    Raw raw[2];
                    fetch(raw[0], base, 0);
#pragma unroll 1
                    for (int b = 0; b + kDepth <= nb; b += kDepth) {
                        const int step = (b + 2 * kDepth) % kCB ? 1 : jump;
#pragma unroll
                        for (int i = 0; i < kDepth; ++i) {
                            fetch(raw[(i + 1) & 1], base, (b + i + 1 < kCB ? b + i + 1 : 0) * kBB);
                            multiply(tot, raw[i & 1], col[i]);
                            load(col[i], acts, i + 1 < kDepth ? 1 : step);
                        }
                    }
                    const int rest = nb & (kDepth - 1);   // only in a row's last chunk
#pragma unroll
                    for (int i = 0; i + 1 < kDepth; ++i)
                        if (i < rest) {
                            fetch(raw[0], base, (nb - rest + i) * kBB);
                            multiply(tot, raw[0], col[i]);
                        }
                }
                __syncwarp();   // every lane has read its part of the stage
                issue();
                stage ^= 1;
            }
            if (kwarps > 1) join(&tot[0][0][0]);
            if constexpr (M == kGateUp) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int tok = 8 * n + 2 * t + (i & 1);
                        const float sc = p.xs[x_row(gi, tok < n_tok ? tok : 0)];
                        const float gate = tot[0][n][i] * sc;
                        if (wk == 0)
                            hidden[tok * 32 + 16 * s + 8 * (i >> 1) + g] =
                                gate / (1.0f + expf(-gate)) * (tot[1][n][i] * sc);
                    }
            } else if (wk == 0) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int tok = 8 * n + 2 * t + i;
                        if (tok < n_tok) {
                            const int64_t row = x_row(gi, tok);
                            const float sc = kScaled ? 1.0f : p.xs[row];
                            float* out = p.out + row * p.rows + tile * 32 + g;
#pragma unroll
                            for (int k = 0; k < 4; ++k)   // rows 8 k + g
                                if (8 * k + g < p.rows - tile * 32) out[8 * k] = tot[k >> 1][n][2 * (k & 1) + i] * sc;
                        }
                    }
            }
        }
        if constexpr (M == kGateUp) {
            // the tokens in turn by the unit's warps; lane i: element i of the block
            unit_sync();
            const int place = few_place(p.h_type, lane), hb = p.rows / 32;
#pragma unroll 1
            for (int tok = wk; tok < n_tok; tok += kwarps) {
                const float h = hidden[tok * 32 + lane];
                const int e = block_exponent(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(h) & 0x7FFFFFFFu));
                const Split x(h, e);
                const int64_t at = static_cast<int64_t>(L.pair[L.start[gi] + tok]) * hb + tile;
                __half* out = p.hb + at * 64 + place + (place & ~7);   // hi and lo by eights
                out[0] = x.hi;
                out[8] = x.lo;
                if (p.h_type == GQ_TYPE_Q4_K) {
                    float sum = x.sum();
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
                    if (lane == 0) p.hsum[at] = pow2f(e - 14) * sum;
                }
                if (lane == 0) p.hs[at] = pow2f(e - 14);
            }
            unit_sync();
        }
    }

    // The warps that share a unit.
    __device__ __forceinline__ void unit_sync() const {
        if (kwarps == 1)
            __syncwarp();
        else
            asm volatile("bar.sync %0, %1;" ::"r"(1 + wr), "r"(32 * kwarps) : "memory");
    }

    // Adds the K warps' totals, in their order, into the first one's.
    __device__ __forceinline__ void join(float* tot) {
        float* const at = sums + wr * kwarps * kTotals * 32 + lane;
        if (wk > 0) {
#pragma unroll
            for (int i = 0; i < kTotals; ++i) at[(wk * kTotals + i) * 32] = tot[i];
        }
        unit_sync();
        if (wk == 0) {
#pragma unroll 1
            for (int k = 1; k < kwarps; ++k)
#pragma unroll
                for (int i = 0; i < kTotals; ++i) tot[i] += at[(k * kTotals + i) * 32];
        }
        unit_sync();
    }
};

template <int T, int M, int Terms, int NT>
__global__ void __launch_bounds__(kThreads, 2) few_kernel(const __grid_constant__ Params p) {
    using Wk = Worker<T, M, Terms, NT>;
    extern __shared__ __align__(128) uint8_t smem[];
    Lists& L = *reinterpret_cast<Lists*>(smem + Wk::kRingBytes + Wk::kSumBytes);
    const int warp = threadIdx.x >> 5;
    griddep_launch_dependents();
    if (M != kDense) build_lists(p.ids, p.E, p.top_k, p.pairs, Wk::kGroup, L, reinterpret_cast<int*>(smem));
    Wk w{p, L, smem_addr(smem) + warp * kStages * Wk::kStageBytes, reinterpret_cast<float*>(smem + Wk::kRingBytes)};
    w.lane = threadIdx.x & 31;
    w.kwarps = 1 << p.kshift;
    w.wk = warp & (w.kwarps - 1);
    w.wr = warp >> p.kshift;
    const int groups = M == kDense ? (p.N + Wk::kGroup - 1) / Wk::kGroup : L.groups;
    // consecutive units for each row warp; the host keeps their number below 2^30
    const int rwarps = kWarps >> p.kshift;
    const int64_t units = static_cast<int64_t>(groups) * p.tiles;
    const int row_warp = blockIdx.x * rwarps + w.wr, row_warps = gridDim.x * rwarps;
    const int begin = static_cast<int>(units * row_warp / row_warps);
    int left = static_cast<int>(units * (row_warp + 1) / row_warps) - begin;
    int gi = begin / p.tiles, tile = begin - gi * p.tiles;
    w.fgi = gi;
    w.ftile = tile;
    w.fleft = left;
    w.fs = w.fstage = 0;
    w.fc = w.wk;
    if (left > 0) w.copy_row();
#pragma unroll 1
    for (int i = 0; i < kStages; ++i) w.issue();
    griddep_wait();   // activations, and what this kernel writes, belong to the kernels before
    int stage = 0;
#pragma unroll 1
    for (; left > 0; --left) {
        w.unit(gi, tile, stage);
        if (++tile == p.tiles) {
            tile = 0;
            ++gi;
        }
    }
}

// Y[n] = sum_j weights[n][j] part[n][j], over the pairs that have an expert, in the order of j.
// One CTA row per token.
__global__ void __launch_bounds__(256)
combine_kernel(const float* __restrict__ part, const int* __restrict__ ids,
               const float* __restrict__ weights, int top_k, int E, int D, float* __restrict__ Y) {
    griddep_launch_dependents();
    griddep_wait();   // `part`, and Y, which the kernels before may still read as X
    const int n = blockIdx.y, quads = D / 4;
    const int r = blockIdx.x * 256 + threadIdx.x;
    if (r >= quads) return;
    const float4* const from = reinterpret_cast<const float4*>(part) + static_cast<int64_t>(n) * top_k * quads + r;
    float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int j = 0; j < top_k; ++j) {
        const int id = ids[n * top_k + j];
        if (id < 0 || id >= E) continue;
        const float w = weights[n * top_k + j];
        const float4 v = from[static_cast<int64_t>(j) * quads];
        y.x = fmaf(w, v.x, y.x);
        y.y = fmaf(w, v.y, y.y);
        y.z = fmaf(w, v.z, y.z);
        y.w = fmaf(w, v.w, y.w);
    }
    float* out = Y + static_cast<int64_t>(n) * D + 4 * r;   // only 4-byte aligned
    out[0] = y.x;
    out[1] = y.y;
    out[2] = y.z;
    out[3] = y.w;
}

// ---- Preparation ------------------------------------------------------------------------

// One CTA per row of X: two-term split activations in the order of `type`, one scale for the
// row; for Q4_K the sums of its blocks in scaled units.
__global__ void __launch_bounds__(512)
split_kernel(const float* __restrict__ X, int kb, int type, __half* __restrict__ xb, float* __restrict__ xs,
             float* __restrict__ xsum) {
    __shared__ uint32_t most[16];
    griddep_wait();                // X, and the workspace that kernels before may still read
    griddep_launch_dependents();   // only now: the next kernel reads ids and weights before it waits
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = blockIdx.x;
    const float* x = X + row * kb * 32;
    uint32_t amax = 0;
#pragma unroll 4
    for (int b = warp; b < kb; b += 16) amax = max(amax, __float_as_uint(x[b * 32 + lane]) & 0x7FFFFFFFu);
    amax = __reduce_max_sync(0xFFFFFFFFu, amax);
    if (lane == 0) most[warp] = amax;
    __syncthreads();
    const int e = block_exponent(__reduce_max_sync(0xFFFFFFFFu, most[lane & 15]));
    if (threadIdx.x == 0) xs[row] = pow2f(e - 14);
    const int place = few_place(type, lane);
    __half* out = xb + row * kb * 64 + place + (place & ~7);   // hi and lo by eights
#pragma unroll 4
    for (int b = warp; b < kb; b += 16) {
        const Split s(x[b * 32 + lane], e);
        __half* at = out + static_cast<int64_t>(b) * 64;
        at[0] = s.hi;
        at[8] = s.lo;
        if (type == GQ_TYPE_Q4_K) {
            float sum = s.sum();
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
            if (lane == 0) xsum[row * kb + b] = sum;
        }
    }
}

// One warp per block (blockIdx.y: the row): X quantized to MXFP4, kept as fp16 values and one
// scale.
__global__ void __launch_bounds__(256)
mx_split_kernel(const float* __restrict__ X, int kb, __half* __restrict__ xb, float* __restrict__ xm) {
    griddep_wait();
    griddep_launch_dependents();
    const int blk = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (blk >= kb) return;
    const int64_t b = static_cast<int64_t>(blockIdx.y) * kb + blk;
    const float x = X[b * 32 + lane];
    const uint32_t byte = mx_scale_byte(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(x) & 0x7FFFFFFFu));
    const uint32_t c = byte == 255 ? 0u : e2m1_pair(x * mx_inverse_scale(byte), 0.0f);
    uint32_t h[4];
    e2m1_to_f16(c, h);
    xb[b * 32 + few_place(GQ_TYPE_MXFP4, lane)] = __ushort_as_half(static_cast<unsigned short>(h[0]));
    if (lane == 0) xm[b] = mx_scale(byte);
}

// ---- Host side --------------------------------------------------------------------------

int64_t align256(int64_t n) { return (n + 255) / 256 * 256; }

// The workspace of split activations of n rows: values (and what loads that run ahead may read
// behind them), scales (one a row, or one a block), sums.
constexpr int kAhead = 64;   // blocks: eight warps' chunks of eight

struct SplitSpace {
    int64_t b, s, sum, bytes;
};

SplitSpace split_space(int64_t n, int64_t K, int terms, bool sums) {
    SplitSpace x{};
    x.s = align256((n * K + kAhead * 32) * 2 * terms);
    x.sum = x.s + align256((n * (K / 32) + kAhead) * 4);
    x.bytes = x.sum + (sums ? align256((n * (K / 32) + kAhead) * 4) : 0);
    return x;
}

cudaError_t launch_split(const float* X, int64_t rows, int kb, int type, uint8_t* ws, const SplitSpace& at,
                         cudaStream_t s) {
    return launch_after(split_kernel, dim3(static_cast<unsigned>(rows)), 512, 0, s, X, kb, type,
                        reinterpret_cast<__half*>(ws + at.b), reinterpret_cast<float*>(ws + at.s),
                        reinterpret_cast<float*>(ws + at.sum));
}

void use_split(Params& p, const uint8_t* ws, const SplitSpace& at) {
    p.xb = reinterpret_cast<const uint4*>(ws + at.b);
    p.xs = reinterpret_cast<const float*>(ws + at.s);
    p.xsum = reinterpret_cast<const float*>(ws + at.sum);
}

// log2 of the warps that split a unit's K. Every row warp takes the same number of units but for
// one, so the split that leaves the fewest warps idle wins, less what a join costs: 3 % a doubling
// at 8 tokens a unit, 8 % at 16. With 1, 2, 4 and 8 warps throughout, in us: 16 tokens over 64 Q8_0
// experts 154, 99, 104, 111; 61 over 64 Q4_K experts 167, 147, 153, 170; 4 over 16 of 32 MXFP4
// experts 64, 41, 39, 42 (all 8 tokens a unit); 32000 x 2048 MXFP4 times 13 tokens 28.7, 23.1, 24.1,
// 27.3 (16 a unit).
int pick_kshift(int64_t units, int chunks, int warps, double join) {
    int best = 0;
    double most = -1.0;
    for (int ks = 0; ks <= 3 && (1 << ks) <= chunks; ++ks) {
        const int64_t rw = warps >> ks, rounds = (units + rw - 1) / rw;
        const double use = static_cast<double>(units) / (rw * rounds) * (1.0 - join * ks);
        if (use > most) {
            most = use;
            best = ks;
        }
    }
    return best;
}

// `groups`: how many there are likely to be.
template <int T, int M, int Terms, int NT>
cudaError_t launch_few(Params p, int64_t groups, const DeviceInfo* info, cudaStream_t s) {
    using Wk = Worker<T, M, Terms, NT>;
    p.chunks = (p.kb + Fmt<T>::cb - 1) / Fmt<T>::cb;
    p.tiles = static_cast<int>((static_cast<int64_t>(p.rows) + 31) / 32);
    const int64_t units = static_cast<int64_t>(p.tiles) * groups;
    p.kshift = pick_kshift(units, p.chunks, 2 * info->sm_count * kWarps, NT == 1 ? 0.03 : 0.08);
    const int64_t rwarps = kWarps >> p.kshift;
    const unsigned grid = static_cast<unsigned>(
        std::max<int64_t>(1, std::min<int64_t>((units + rwarps - 1) / rwarps, int64_t(info->sm_count) * 2)));
    auto kernel = few_kernel<T, M, Terms, NT>;
    static std::atomic<uint64_t> ready{0};   // devices whose attribute is set
    const uint64_t bit = uint64_t(1) << info->device;
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        const cudaError_t e =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Wk::kSmem);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    return launch_after(kernel, dim3(grid), kThreads, Wk::kSmem, s, p);
}

// Two-term launch with one or two tiles of 8 tokens.
template <int T, int M>
cudaError_t launch_sized(const Params& p, bool wide, int64_t groups, const DeviceInfo* info, cudaStream_t s) {
    return wide ? launch_few<T, M, 2, 2>(p, groups, info, s) : launch_few<T, M, 2, 1>(p, groups, info, s);
}

template <int M>
cudaError_t launch_typed(gq_type t, const Params& p, bool wide, int64_t groups, const DeviceInfo* info,
                         cudaStream_t s) {
    switch (t) {
        case GQ_TYPE_Q4_0: return launch_sized<GQ_TYPE_Q4_0, M>(p, wide, groups, info, s);
        case GQ_TYPE_Q8_0: return launch_sized<GQ_TYPE_Q8_0, M>(p, wide, groups, info, s);
        case GQ_TYPE_Q4_K: return launch_sized<GQ_TYPE_Q4_K, M>(p, wide, groups, info, s);
        case GQ_TYPE_MXFP4: return launch_sized<GQ_TYPE_MXFP4, M>(p, wide, groups, info, s);
    }
    return cudaErrorInvalidValue;
}

int64_t row_bytes_of(gq_type t, int64_t K) { return K / block_weights_of(t) * block_bytes_of(t); }

Params dense_params(const MatProblem& m, int64_t n0, int64_t n) {
    Params p{};
    p.W = m.W;
    p.row_bytes = row_bytes_of(GQ_TYPE_MXFP4, m.K);
    p.total_bytes = p.row_bytes * m.M;
    p.rows = static_cast<int>(m.M);
    p.kb = static_cast<int>(m.K / 32);
    p.N = static_cast<int>(n);
    p.out = m.Y + n0 * m.M;
    return p;
}

struct MoeSpace {   // offsets in the workspace of one launch over n tokens
    SplitSpace x, h;
    int64_t h_at, part, bytes;
};

MoeSpace moe_space(const MoeProblem& m, int64_t n) {
    const int64_t pairs = n * m.top_k;
    MoeSpace s{};
    s.x = split_space(n, m.D, 2, true);
    s.h = split_space(pairs, m.F, 2, true);
    s.h_at = s.x.bytes;
    s.part = s.h_at + s.h.bytes;
    s.bytes = s.part + align256(pairs * m.D * 4);
    return s;
}

int64_t moe_tokens_per_launch(const MoeProblem& m) {
    return std::min<int64_t>(m.N, kMoeMaxPairs / m.top_k);
}

}  // namespace

// ---- MXFP4 mul_mat ----------------------------------------------------------------------

int64_t few_workspace_bytes(int64_t K, int64_t N) {
    const int64_t n = std::min(N, kFewMaxTokens);
    return split_space(n, K, 2, false).bytes;
}

// Tokens of one launch: few enough for the workspace, and for 2^30 units.
int64_t few_tokens_that_fit(int64_t M, int64_t K, int64_t N, int64_t workspace_bytes) {
    const int64_t units = std::max<int64_t>(16, (int64_t(1) << 30) / ((M + 31) / 32) * 8);
    int64_t n = std::min(std::min(N, kFewMaxTokens), units);
    while (n > 0 && few_workspace_bytes(K, n) > workspace_bytes) n = n > 16 ? n / 2 : n - 1;
    return n;
}

cudaError_t launch_few_mul_mat(const MatProblem& m, int64_t N, void* workspace,
                               int64_t workspace_bytes, cudaStream_t s) {
    DeviceInfo* info = nullptr;
    cudaError_t e = current_device_info(&info);
    if (e != cudaSuccess) return e;
    const int64_t per = few_tokens_that_fit(m.M, m.K, N, workspace_bytes);
    if (per < 1) return cudaErrorInvalidValue;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    for (int64_t n0 = 0; n0 < N && e == cudaSuccess; n0 += per) {
        const int64_t n = std::min(per, N - n0);
        Params p = dense_params(m, n0, n);
        const SplitSpace at = split_space(n, m.K, 2, false);
        use_split(p, ws, at);
        e = launch_split(m.X + n0 * m.K, n, p.kb, GQ_TYPE_MXFP4, ws, at, s);
        if (e == cudaSuccess)
            e = launch_sized<GQ_TYPE_MXFP4, kDense>(p, n > 8, n > 8 ? (n + 15) / 16 : 1, info, s);
    }
    return e;
}

int64_t few_mx_workspace_bytes(int64_t K, int64_t N) {
    return split_space(N, K, 1, false).bytes;
}

cudaError_t launch_few_mx4x(const MatProblem& m, int64_t N, void* workspace, cudaStream_t s) {
    DeviceInfo* info = nullptr;
    cudaError_t e = current_device_info(&info);
    if (e != cudaSuccess) return e;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    Params p = dense_params(m, 0, N);
    const SplitSpace at = split_space(N, m.K, 1, false);
    use_split(p, ws, at);
    const dim3 grid(static_cast<unsigned>((p.kb + 7) / 8), static_cast<unsigned>(N));
    e = launch_after(mx_split_kernel, grid, 256, 0, s, m.X, p.kb, reinterpret_cast<__half*>(ws + at.b),
                     reinterpret_cast<float*>(ws + at.s));
    if (e != cudaSuccess) return e;
    if (N <= 8) return launch_few<GQ_TYPE_MXFP4, kDense, 1, 1>(p, 1, info, s);
    return launch_few<GQ_TYPE_MXFP4, kDense, 1, 2>(p, (N + 15) / 16, info, s);
}

// ---- Mixture of experts -----------------------------------------------------------------

int64_t moe_workspace_bytes(const MoeProblem& m) {
    return moe_space(m, moe_tokens_per_launch(m)).bytes;
}

cudaError_t launch_moe(const MoeProblem& m, void* workspace, cudaStream_t s) {
    DeviceInfo* info = nullptr;
    cudaError_t e = current_device_info(&info);
    if (e != cudaSuccess) return e;
    const int64_t per = moe_tokens_per_launch(m);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    for (int64_t n0 = 0; n0 < m.N; n0 += per) {
        const int64_t n = std::min(per, m.N - n0);
        const MoeSpace at = moe_space(m, n);
        const int pairs = static_cast<int>(n * m.top_k);
        // One tile of 8 tokens, or two where an expert at work has more on average than fit one
        // in most cases. In us with one and two, by tokens an expert on average (4 chosen, D = 2048,
        // F = 1024; the draw of experts moves single figures by a fifth):
        //                       6            8           10           12           16
        //   32 Q4_0          69.1  84.0   98.8  85.3  101.1  86.6  130.5  89.3  167.5 133.8
        //   32 Q8_0          80.4  98.3  115.6 100.0  119.8 102.3  169.3 104.0  211.1 160.5
        //   32 Q4_K          65.6  90.4   94.3  92.6   97.2  94.1  126.9  96.5  159.0 157.8
        //    8 Q4_K          25.8  34.7   34.6  35.2   49.8  36.2   49.7  36.4   51.6  76.9
        //   32 MXFP4         61.5  77.4   89.3  78.3   91.5  80.7  121.9  82.9  139.6 124.3
        // and 61 tokens over 64 Q4_K experts, 7.6 an expert, 147 and 167. The two-tile kernels do not
        // fit their 128 registers: bytes spilled for Q4_K 140 (gate and up) and 356 (down), 8 to 64 for
        // the other types (one tile: at most 16). `groups` as if the pairs were spread by chance.
        const double active = m.E * (1.0 - std::pow(1.0 - 1.0 / m.E, pairs));
        const double mean = pairs / active;
        const bool wide = mean > 10.0;
        const double per_group = wide ? 16.0 : 8.0;
        // groups of Poisson-spread counts: about half a group more than full ones an expert
        const int64_t groups = std::max<int64_t>(
            1, static_cast<int64_t>(active * std::max(1.0, mean / per_group + 0.4) + 0.5));
        Params g{};
        g.W = m.W_gate;
        g.W2 = m.W_up;
        g.row_bytes = row_bytes_of(m.t, m.D);
        g.total_bytes = g.row_bytes * m.F * m.E;
        g.rows = static_cast<int>(m.F);
        g.kb = static_cast<int>(m.D / 32);
        use_split(g, ws, at.x);
        g.N = static_cast<int>(n);
        g.E = static_cast<int>(m.E);
        g.top_k = m.top_k;
        g.pairs = pairs;
        g.ids = m.ids + n0 * m.top_k;
        g.hb = reinterpret_cast<__half*>(ws + at.h_at + at.h.b);
        g.hs = reinterpret_cast<float*>(ws + at.h_at + at.h.s);
        g.hsum = reinterpret_cast<float*>(ws + at.h_at + at.h.sum);
        g.h_type = m.t_down;
        Params d = g;
        d.W = m.W_down;
        d.W2 = nullptr;
        d.row_bytes = row_bytes_of(m.t_down, m.F);
        d.total_bytes = d.row_bytes * m.D * m.E;
        d.rows = static_cast<int>(m.D);
        d.kb = static_cast<int>(m.F / 32);
        use_split(d, ws + at.h_at, at.h);
        d.out = reinterpret_cast<float*>(ws + at.part);
        e = launch_split(m.X + n0 * m.D, n, g.kb, m.t, ws, at.x, s);
        if (e == cudaSuccess) e = launch_typed<kGateUp>(m.t, g, wide, groups, info, s);
        if (e == cudaSuccess) e = launch_typed<kDown>(m.t_down, d, wide, groups, info, s);
        if (e == cudaSuccess) {
            const dim3 grid(static_cast<unsigned>((m.D / 4 + 255) / 256), static_cast<unsigned>(n));
            e = launch_after(combine_kernel, grid, 256, 0, s, static_cast<const float*>(d.out), g.ids,
                             m.weights + n0 * m.top_k, m.top_k, g.E, d.rows, m.Y + n0 * m.D);
        }
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace gq
