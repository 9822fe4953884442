// gq_few.cu -- block-quantized weights times a few fp32 tokens, to fp32 accuracy: the MXFP4
// mul_mat and the two weight passes of the mixture-of-experts layer.
//
// Mathematics. A weight row's block is d (q - z) with small integers q (or E2M1 values), so
//     sum_k What[m][k] x[k] = sum_b d_b s_b sum_{k in b} (q_k - z) xs_k
// with xs = x / s_b split in two fp16 terms (gq_few.cuh). The inner sum runs on the tensor
// cores: mma.m16n8k16 with 16 weight rows as exact fp16 codes, 8 columns = 4 tokens x (hi, lo),
// two instructions a block, fp32 accumulators; the outer sum is one fp32
// multiply-add per block, row and token. Nothing is rounded below 22 bits but the fp32 sums.
//
// What bounds it. One pass over the weights: at most 34 bytes per 32 weights from DRAM, about
// 30 instructions per 16 rows x 32 weights x 4 tokens. At 6.8 TB/s an SM takes in 512 4-bit
// weights every 12 cycles, 47 issue slots, so instructions come close to memory as the limit;
// that is why codes become fp16 by masks alone (subnormals, gq_few.cuh) and why tcgen05 is not
// used here: its operands would have to pass through shared memory once more, with the
// scales applied there, and its 128-row tiles leave most SMs without work at these sizes.
//
// Layout of the work. A unit is (a group of up to 16 tokens, a tile of 32 weight rows per
// warp). The four warps of a CTA take four row tiles or split a tile's K range (kshift).
// Every warp runs its own ring of bulk copies: one copy per weight row and chunk, starting at
// the 16-byte word that holds the chunk's first byte, because rows of 17- and 18-byte blocks
// start anywhere; the words are aligned in registers. The ring runs on across units, so the
// next unit's weights are on their way while a unit ends. Weights do not depend on the kernel
// before, so they start to stream before griddepcontrol.wait.
#include <algorithm>
#include <cstddef>

#include "gq_few.cuh"

namespace gq {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

constexpr int64_t kFewMaxTokens = 4096;   // of one launch: bounds the workspace

enum Mode { kDense = 0, kGateUp = 1, kDown = 2 };

template <int T>
struct Fmt;   // block bytes, 32-weight blocks per chunk, shared-memory pitch of a row's chunk
template <>
struct Fmt<GQ_TYPE_Q4_0> {
    static constexpr int bb = kQ4Bytes, cb = 8, pitch = 176;
};
template <>
struct Fmt<GQ_TYPE_Q8_0> {
    static constexpr int bb = kQ8Bytes, cb = 4, pitch = 176;
};
template <>
struct Fmt<GQ_TYPE_Q4_K> {   // bb: a super-block's bytes over its 8 sub-blocks
    static constexpr int bb = kQ4KBytes / 8, cb = 8, pitch = 144;
};
template <>
struct Fmt<GQ_TYPE_MXFP4> {
    static constexpr int bb = kMxfp4Bytes, cb = 8, pitch = 176;
};
// Pitches: a chunk is 136..144 bytes and starts up to 15 bytes into its first 16-byte word;
// 176 = 44 words puts the eight rows that a warp reads at once on eight distinct groups of four
// banks, as 144 = 36 words does where rows are always aligned (Q4_K).

struct Params {
    const uint8_t* W;
    const uint8_t* W2;        // kGateUp: the up matrices
    int64_t total_bytes;      // of W (and of W2)
    int64_t row_bytes;
    int rows;                 // weight rows (of one expert)
    int kb;                   // 32-weight blocks per row
    int tiles;                // row tiles: ceil(rows / (32 row-warps))
    int kshift;               // log2 of the warps that share a row tile by splitting K
    const uint4* xb;          // split activations, 64 bytes per (row, term, block)
    const float* xm;          // their block factors: float2 (two terms) or float (one)
    int64_t N;                // tokens
    int E, top_k, pairs;
    const int* ids;
    const float* weights;
    float* Y;                 // kDense, kDown
    __half* hb;               // kGateUp: split activations of the result,
    float2* hm;
    int h_type;               //          in the order of the down matrices' type
    float* part;              // kDown: [pair][rows]
    unsigned* arrived;        // kDown: per row tile
    unsigned* status;
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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

// Products of one 16-row tile with one block, for NT column tiles:
// tot += d_row s_token (codes . columns).
template <int MT, int NT, int Terms>
struct Totals {
    // [row tile][row g or g + 8][column tile][two terms: token t; one term: tokens 2t, 2t + 1]
    float v[MT][2][NT][Terms == 2 ? 1 : 2];
};

template <int NT, int Terms>
struct Columns {
    uint4 b[NT];        // this lane's eight fp16 of column g
    float2 m[NT];       // {scale, sum} of token t (two terms), or x, y of tokens 2t, 2t + 1 (one)
};

template <int T, int Terms, int NT>
__device__ __forceinline__ void block_products(const uint32_t (&lo)[4], const uint32_t (&hi)[4],
                                               float dlo, float dhi, float mlo, float mhi,
                                               const Columns<NT, Terms>& col,
                                               float (&t0)[NT][Terms == 2 ? 1 : 2],
                                               float (&t1)[NT][Terms == 2 ? 1 : 2]) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        mma16816(c, lo[0], hi[0], lo[1], hi[1], col.b[n].x, col.b[n].y);
        mma16816(c, lo[2], hi[2], lo[3], hi[3], col.b[n].z, col.b[n].w);
        if (Terms == 2) {
            t0[n][0] = fmaf(dlo * col.m[n].x, c[0] + c[1], t0[n][0]);
            t1[n][0] = fmaf(dhi * col.m[n].x, c[2] + c[3], t1[n][0]);
            if (T == GQ_TYPE_Q4_K) {
                t0[n][0] = fmaf(-mlo, col.m[n].y, t0[n][0]);
                t1[n][0] = fmaf(-mhi, col.m[n].y, t1[n][0]);
            }
        } else {
            t0[n][0] = fmaf(dlo * col.m[n].x, c[0], t0[n][0]);
            t0[n][Terms == 2 ? 0 : 1] = fmaf(dlo * col.m[n].y, c[1], t0[n][Terms == 2 ? 0 : 1]);
            t1[n][0] = fmaf(dhi * col.m[n].x, c[2], t1[n][0]);
            t1[n][Terms == 2 ? 0 : 1] = fmaf(dhi * col.m[n].y, c[3], t1[n][Terms == 2 ? 0 : 1]);
        }
    }
}

// The shared lists of a launch over experts: pairs sorted by expert, and groups of up to
// kFewGroup2 pairs of one expert.
struct Lists {
    uint16_t pair[kMoeMaxPairs];
    uint16_t expert[kMoeMaxPairs];
    uint16_t start[kMoeMaxPairs];
    uint8_t count[kMoeMaxPairs];
    int groups;
};

// Sorts the pairs by expert, in their own order inside an expert: every CTA has to find the
// same groups. ids outside [0, E) are in no group. `scratch`: kMoeMaxExperts + kMoeMaxPairs
// ints. One warp ranks 32 pairs at a time by matching their ids; 512 pairs are 16 steps.
__device__ void build_lists(const Params& p, Lists& L, int* scratch) {
    int* count = scratch;
    int* ids = scratch + kMoeMaxExperts;
    for (int e = threadIdx.x; e < p.E; e += kThreads) count[e] = 0;
    for (int q = threadIdx.x; q < p.pairs; q += kThreads) {
        const int id = p.ids[q];
        ids[q] = id >= 0 && id < p.E ? id : -1;
    }
    __syncthreads();
    constexpr int kPer = kMoeMaxPairs / kThreads;
    if (threadIdx.x < 32) {
        const unsigned below = (1u << threadIdx.x) - 1u;
        for (int q0 = 0; q0 < p.pairs; q0 += 32) {
            const int q = q0 + threadIdx.x;
            const int id = q < p.pairs ? ids[q] : -1;
            const unsigned same = __match_any_sync(0xFFFFFFFFu, id);
            const int before = id >= 0 ? count[id] : 0;
            __syncwarp();
            if (id >= 0) {
                if ((same & below) == 0) count[id] = before + __popc(same);
                ids[q] = id | ((before + __popc(same & below)) << 16);   // id < 1024, rank < 512
            }
            __syncwarp();
        }
    }
    __syncthreads();
    // exclusive sums over the experts: pairs (low half) and groups (high half)
    if (threadIdx.x < 32) {
        int base = 0;
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            const int e = e0 + threadIdx.x;
            const int c = e < p.E ? count[e] : 0;
            const int g = (c + kFewGroup2 - 1) / kFewGroup2;
            int incl = c | (g << 16);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(0xFFFFFFFFu, incl, o);
                if (static_cast<int>(threadIdx.x) >= o) incl += up;
            }
            const int excl = base + incl - (c | (g << 16));
            const int pair0 = excl & 0xFFFF, group0 = excl >> 16;
            for (int i = 0; i < g; ++i) {
                L.expert[group0 + i] = static_cast<uint16_t>(e);
                L.start[group0 + i] = static_cast<uint16_t>(pair0 + i * kFewGroup2);
                L.count[group0 + i] = static_cast<uint8_t>(min(kFewGroup2, c - i * kFewGroup2));
            }
            if (e < p.E) count[e] = pair0;
            base += __shfl_sync(0xFFFFFFFFu, incl, 31);
        }
        if (threadIdx.x == 0) L.groups = base >> 16;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int q = threadIdx.x + i * kThreads;
        if (q < p.pairs && ids[q] >= 0)
            L.pair[count[ids[q] & 0xFFFF] + (ids[q] >> 16)] = static_cast<uint16_t>(q);
    }
    __syncthreads();
}

template <int T, int M, int Terms>
struct Few {
    static constexpr int kMT = M == kGateUp ? 4 : 2;          // 16-row tiles per warp
    static constexpr int kRows = 16 * kMT;                    // weight rows per warp and chunk
    static constexpr int kPitch = Fmt<T>::pitch;
    static constexpr int kStageBytes = kRows * kPitch + 16;   // the last word's second half
    static constexpr int kStages = M == kGateUp ? 2 : 4;
    static constexpr int kGroup = Terms == 2 ? kFewGroup2 : kFewGroup1;
    static constexpr int kTotals = kMT * 2 * 4 * (Terms == 2 ? 1 : 2);   // floats a lane, NT = 4
    static constexpr int kRingBytes = kWarps * kStages * kStageBytes;
    static constexpr int kSumBytes = (kWarps - 1) * kTotals * 32 * 4;
    static constexpr int kSmem = kRingBytes + kSumBytes + static_cast<int>(sizeof(Lists)) + 16;
    static_assert((kMoeMaxExperts + kMoeMaxPairs) * 4 <= kRingBytes, "the lists' scratch lies in the ring");
};

template <int T, int M, int Terms>
struct Worker {
    using F = Few<T, M, Terms>;
    const Params& p;
    const Lists& L;
    uint8_t* ring;      // this warp's
    float* sums;        // the CTA's
    uint64_t* bars;     // this warp's, kStages
    int lane, wk, wr, kwarps, rwarps, chunks;
    int units;
    // copies: next (unit, chunk) to issue and its stage; consumption: stage and phase
    int iu, ic, istage;
    int irow0;
    int64_t ie_row;
    int cstage;
    uint32_t cphase;
    bool dead;

    __device__ __forceinline__ int group_of(int unit) const { return unit / p.tiles; }
    __device__ __forceinline__ int expert_of(int gi) const { return M == kDense ? 0 : L.expert[gi]; }
    __device__ __forceinline__ int count_of(int gi) const {
        if (M != kDense) return L.count[gi];
        return static_cast<int>(min(static_cast<int64_t>(F::kGroup),
                                    p.N - static_cast<int64_t>(gi) * F::kGroup));
    }
    // activation row of column token i of a group
    __device__ __forceinline__ int64_t x_row(int gi, int i) const {
        if (M == kDense) return static_cast<int64_t>(gi) * F::kGroup + i;
        const int q = L.pair[L.start[gi] + i];
        return M == kGateUp ? q / p.top_k : q;
    }
    __device__ __forceinline__ int first_row(int unit) const {
        return ((unit % p.tiles) * rwarps + wr) * 32;
    }

    __device__ __forceinline__ void issue_from(int unit) {
        iu = unit;
        ic = wk;
        if (iu >= units) return;
        irow0 = first_row(iu);
        ie_row = static_cast<int64_t>(expert_of(group_of(iu))) * p.rows;
    }

    // Starts the copies of the next chunk (if any) into the next stage.
    __device__ __forceinline__ void issue() {
        if (iu >= units) return;
        const int r = irow0 + lane;
        const int nb = min(Fmt<T>::cb, p.kb - ic * Fmt<T>::cb);
        const uint32_t bar = smem_addr(&bars[istage]);
        uint8_t* dst = ring + istage * F::kStageBytes + lane * F::kPitch;
        uint32_t bytes = 0;
        int64_t from = 0;
        if (r < p.rows) {
            const int64_t start = (ie_row + r) * p.row_bytes + static_cast<int64_t>(ic) * (Fmt<T>::cb * Fmt<T>::bb);
            from = start & ~static_cast<int64_t>(15);
            int64_t to = (start + nb * Fmt<T>::bb + 15) & ~static_cast<int64_t>(15);
            if (to > p.total_bytes) {   // the matrix ends inside its last 16-byte word
                to = p.total_bytes & ~static_cast<int64_t>(15);
                for (int64_t i = to > from ? to : from; i < p.total_bytes; ++i) {
                    dst[i - from] = p.W[i];
                    if (M == kGateUp) dst[32 * F::kPitch + (i - from)] = p.W2[i];
                }
            }
            bytes = to > from ? static_cast<uint32_t>(to - from) : 0u;
        }
        mbar_arrive_expect_tx(bar, M == kGateUp ? 2 * bytes : bytes);
        if (bytes > 0) {
            bulk_g2s_evict_first(smem_addr(dst), p.W + from, bytes, bar);
            if (M == kGateUp)
                bulk_g2s_evict_first(smem_addr(dst) + 32 * F::kPitch, p.W2 + from, bytes, bar);
        }
        istage = istage + 1 == F::kStages ? 0 : istage + 1;
        ic += kwarps;
        if (ic >= chunks) issue_from(iu + gridDim.x);
    }

    // Waits for the copies of the stage at hand; after a wait that ran out, for those of the
    // others too (again with a limit), so that none is in flight when the CTA leaves.
    __device__ __forceinline__ void wait_stage() {
        if (dead) return;
        const bool ok = mbar_wait(smem_addr(&bars[cstage]), cphase);
        if (__all_sync(0xFFFFFFFFu, ok)) return;
        dead = true;
        report_status(p.status, kStatusTimeout);
        for (int i = 1, st = cstage, ph = cphase; i < F::kStages; ++i) {
            if (++st == F::kStages) {
                st = 0;
                ph ^= 1;
            }
            mbar_wait(smem_addr(&bars[st]), ph);
        }
    }

    template <int NT>
    __device__ __forceinline__ void load_columns(Columns<NT, Terms>& col, const uint4* const (&xp)[NT],
                                                 const float* const (&mp)[NT][Terms == 2 ? 1 : 2],
                                                 int kb) const {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            col.b[n] = xp[n] ? xp[n][static_cast<int64_t>(kb) * 4] : make_uint4(0u, 0u, 0u, 0u);
            if (Terms == 2) {
                col.m[n] = mp[n][0] ? reinterpret_cast<const float2*>(mp[n][0])[kb]
                                    : make_float2(0.0f, 0.0f);
            } else {
                col.m[n].x = mp[n][0] ? mp[n][0][kb] : 0.0f;
                col.m[n].y = mp[n][Terms == 2 ? 0 : 1] ? mp[n][Terms == 2 ? 0 : 1][kb] : 0.0f;
            }
        }
    }

    // One chunk (nb blocks from block kb0) out of the stage's shared memory.
    template <int NT>
    __device__ __forceinline__ void chunk(Totals<F::kMT, NT, Terms>& tot, Columns<NT, Terms>& col,
                                          const uint4* const (&xp)[NT],
                                          const float* const (&mp)[NT][Terms == 2 ? 1 : 2],
                                          const uint8_t* stage, int64_t e_row, int row0, int c,
                                          int next_kb) {
        constexpr int kCB = Fmt<T>::cb, kBB = Fmt<T>::bb;
        const int g = lane >> 2, t = lane & 3;
        const int kb0 = c * kCB;
        const int nb = min(kCB, p.kb - kb0);
        // Where this lane's rows begin inside their staged words (0..15). Rows g and g + 8 of
        // every tile agree in the low two bits, since eight rows are a multiple of 8 bytes.
        const uint8_t* base[F::kMT][2];
#pragma unroll
        for (int mt = 0; mt < F::kMT; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int rr = 16 * mt + 8 * h + g;
                const uint32_t row = static_cast<uint32_t>(e_row) + static_cast<uint32_t>(row0 + (rr & 31));
                const uint32_t mis = (row * static_cast<uint32_t>(p.row_bytes) +
                                      static_cast<uint32_t>(c) * (kCB * kBB)) & 15u;
                base[mt][h] = stage + rr * F::kPitch + mis;
            }
        const uint32_t r3 = smem_addr(base[0][0]) & 3u;
        if constexpr (T == GQ_TYPE_Q4_K) {
            uint4 hd[F::kMT][2];
#pragma unroll
            for (int mt = 0; mt < F::kMT; ++mt)
#pragma unroll
                for (int h = 0; h < 2; ++h) hd[mt][h] = *reinterpret_cast<const uint4*>(base[mt][h]);
#pragma unroll
            for (int b = 0; b < 8; b += 2) {
                uint32_t w[F::kMT][2][2];
#pragma unroll
                for (int mt = 0; mt < F::kMT; ++mt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint8_t* a = base[mt][h] + 16 + 16 * b + 4 * t;
                        w[mt][h][0] = *reinterpret_cast<const uint32_t*>(a);
                        w[mt][h][1] = *reinterpret_cast<const uint32_t*>(a + 16);
                    }
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    Columns<NT, Terms> cur = col;
                    if (b + s + 1 < 8)
                        load_columns<NT>(col, xp, mp, kb0 + b + s + 1);
                    else if (next_kb >= 0)
                        load_columns<NT>(col, xp, mp, next_kb);
#pragma unroll
                    for (int mt = 0; mt < F::kMT; ++mt) {
                        uint32_t q[2][4];
                        float d[2], m[2];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t mask = s ? 0x00F000F0u : 0x000F000Fu;
                            const uint32_t w0 = w[mt][h][0], w1 = w[mt][h][1];
                            q[h][0] = (w0 & mask) | kMagic;
                            q[h][1] = ((w0 >> 8) & mask) | kMagic;
                            q[h][2] = (w1 & mask) | kMagic;
                            q[h][3] = ((w1 >> 8) & mask) | kMagic;
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                q[h][i] = s ? h2_fma(q[h][i], kSixteenth, 0xD400D400u)
                                            : h2_sub(q[h][i], kMagic);
                            uint32_t sc, mn;
                            q4k_scales(hd[mt][h], b >> 1, sc, mn);
                            d[h] = half_bits_to_float(hd[mt][h].x) * static_cast<float>((sc >> (8 * s)) & 0xFFu);
                            m[h] = half_bits_to_float(hd[mt][h].x >> 16) *
                                   static_cast<float>((mn >> (8 * s)) & 0xFFu);
                        }
                        block_products<T, Terms, NT>(q[0], q[1], d[0], d[1], m[0], m[1], cur,
                                                     tot.v[mt][0], tot.v[mt][1]);
                    }
                }
            }
            return;
        }
        // Unaligned words: the aligned word at (base + delta[j] + 4-multiple) and its
        // successor, shifted by shift[j], for byte offsets congruent j modulo 4.
        int delta[4];
        uint32_t shift[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            delta[j] = (r3 + j >= 4 ? 4 : 0) - static_cast<int>(r3) + 4 * t;
            shift[j] = (r3 + j) << 3;   // the funnel shift takes it modulo 32
        }
#pragma unroll
        for (int b = 0; b < kCB; ++b) {
            if (b < nb) {
                Columns<NT, Terms> cur = col;
                if (b + 1 < nb)
                    load_columns<NT>(col, xp, mp, kb0 + b + 1);
                else if (next_kb >= 0)
                    load_columns<NT>(col, xp, mp, next_kb);
#pragma unroll
                for (int mt = 0; mt < F::kMT; ++mt) {
                    uint32_t q[2][4];
                    float d[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        constexpr int kHead = T == GQ_TYPE_MXFP4 ? 1 : 2;
                        const int off = b * kBB + kHead;
                        const uint8_t* a = base[mt][h] + delta[off & 3];
                        const uint32_t* w = reinterpret_cast<const uint32_t*>(a + (off & ~3));
                        const uint32_t w0 = __funnelshift_r(w[0], w[1], shift[off & 3]);
                        if (T == GQ_TYPE_Q8_0) {
                            const uint32_t w1 = __funnelshift_r(w[4], w[5], shift[off & 3]);
                            const uint32_t u0 = w0 ^ 0x80808080u, u1 = w1 ^ 0x80808080u;
                            // 1024 + 128 + code, byte by byte under the exponent
                            q[h][0] = h2_sub(__byte_perm(u0, 0x64u, 0x4140), 0x64806480u);
                            q[h][1] = h2_sub(__byte_perm(u0, 0x64u, 0x4342), 0x64806480u);
                            q[h][2] = h2_sub(__byte_perm(u1, 0x64u, 0x4140), 0x64806480u);
                            q[h][3] = h2_sub(__byte_perm(u1, 0x64u, 0x4342), 0x64806480u);
                        } else if (T == GQ_TYPE_Q4_0) {
                            nibbles_to_f16<8>(w0, q[h]);
                        } else {
                            e2m1_to_f16(w0, q[h]);
                        }
                        d[h] = T == GQ_TYPE_MXFP4
                                   ? mx_scale(base[mt][h][b * kBB])
                                   : half_bits_to_float(*reinterpret_cast<const unsigned short*>(
                                         base[mt][h] + b * kBB));
                    }
                    block_products<T, Terms, NT>(q[0], q[1], d[0], d[1], 0.0f, 0.0f, cur,
                                                 tot.v[mt][0], tot.v[mt][1]);
                }
            }
        }
    }

    // Adds the K ranges' totals in warp order into the wk == 0 warps.
    template <int NT>
    __device__ __forceinline__ void join(Totals<F::kMT, NT, Terms>& tot) {
        if (kwarps == 1) return;
        constexpr int kN = F::kMT * 2 * NT * (Terms == 2 ? 1 : 2);
        float* mine = &tot.v[0][0][0][0];
        if (wk > 0) {
            float* to = sums + (wr * (kwarps - 1) + wk - 1) * F::kTotals * 32 + lane;
#pragma unroll
            for (int i = 0; i < kN; ++i) to[i * 32] = mine[i];
        }
        __syncthreads();
        if (wk == 0) {
            for (int k = 0; k < kwarps - 1; ++k) {
                const float* from = sums + (wr * (kwarps - 1) + k) * F::kTotals * 32 + lane;
#pragma unroll
                for (int i = 0; i < kN; ++i) mine[i] += from[i * 32];
            }
        }
        __syncthreads();
    }

    template <int NT>
    __device__ __forceinline__ void unit(int u) {
        const int gi = group_of(u), n_tok = count_of(gi);
        const int64_t e_row = static_cast<int64_t>(expert_of(gi)) * p.rows;
        const int row0 = first_row(u);
        const int g = lane >> 2, t = lane & 3;
        const uint4* xp[NT];
        const float* mp[NT][Terms == 2 ? 1 : 2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int i = Terms == 2 ? 4 * n + (g >> 1) : 8 * n + g;
            xp[n] = nullptr;
            if (i < n_tok)
                xp[n] = p.xb + ((x_row(gi, i) * Terms + (Terms == 2 ? g & 1 : 0)) * p.kb) * 4 + t;
#pragma unroll
            for (int s = 0; s < (Terms == 2 ? 1 : 2); ++s) {
                const int j = Terms == 2 ? 4 * n + t : 8 * n + 2 * t + s;
                mp[n][s] = nullptr;
                if (j < n_tok) mp[n][s] = p.xm + x_row(gi, j) * p.kb * Terms;
            }
        }
        Totals<F::kMT, NT, Terms> tot;
#pragma unroll
        for (int i = 0; i < F::kMT * 2 * NT * (Terms == 2 ? 1 : 2); ++i) (&tot.v[0][0][0][0])[i] = 0.0f;
        Columns<NT, Terms> col;
        load_columns<NT>(col, xp, mp, wk * Fmt<T>::cb);
        for (int c = wk; c < chunks; c += kwarps) {
            wait_stage();
            chunk<NT>(tot, col, xp, mp, ring + cstage * F::kStageBytes, e_row, row0, c,
                      c + kwarps < chunks ? (c + kwarps) * Fmt<T>::cb : -1);
            release_warp_to_async_proxy(__float_as_uint(tot.v[0][0][0][0]));
            __syncwarp();
            if (!dead) issue();
            if (++cstage == F::kStages) {
                cstage = 0;
                cphase ^= 1;
            }
        }
        join<NT>(tot);
        if (wk == 0) finish<NT>(tot, gi, n_tok, row0);
        if constexpr (M == kDown) arrive(u);
    }

    template <int NT>
    __device__ __forceinline__ void finish(Totals<F::kMT, NT, Terms>& tot, int gi, int n_tok, int row0) {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if constexpr (M == kGateUp) {
                // rows 0-31 are gate, 32-63 up: this lane has elements g, 8 + g, 16 + g, 24 + g
                // of the block and token t of both
                float h[4];
                uint32_t amax = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float gate = tot.v[i >> 1][i & 1][n][0];
                    const float up = tot.v[(F::kMT / 2) + (i >> 1)][i & 1][n][0];
                    h[i] = gate / (1.0f + expf(-gate)) * up;
                    amax = max(amax, __float_as_uint(h[i]) & 0x7FFFFFFFu);
                }
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
                const int e = block_exponent(amax);
                const float inv = pow2f(14 - e);
                __half hi[4], lo[4];
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x = h[i] * inv;
                    hi[i] = __float2half_rn(x);
                    lo[i] = __float2half_rn(x - __half2float(hi[i]));
                    sum += __half2float(hi[i]) + __half2float(lo[i]);
                }
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
                const int i_tok = 4 * n + t;
                if (i_tok < n_tok && row0 < p.rows) {
                    const int64_t q = L.pair[L.start[gi] + i_tok];
                    const int64_t hb = p.rows / 32, blk = row0 / 32;
                    __half* out = p.hb + (q * 2 * hb + blk) * 32;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int at = few_place(p.h_type, 8 * i + g);
                        out[at] = hi[i];
                        out[hb * 32 + at] = lo[i];
                    }
                    if (g == 0) {
                        const float s = pow2f(e - 14);
                        p.hm[q * hb + blk] =
                            make_float2(s, s * sum);
                    }
                }
            } else {
#pragma unroll
                for (int s = 0; s < (Terms == 2 ? 1 : 2); ++s) {
                    const int i_tok = Terms == 2 ? 4 * n + t : 8 * n + 2 * t + s;
                    if (i_tok >= n_tok) break;
                    float* out = M == kDown ? p.part : p.Y;
                    out += x_row(gi, i_tok) * p.rows;
#pragma unroll
                    for (int mt = 0; mt < F::kMT; ++mt)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int row = row0 + 16 * mt + 8 * h + g;
                            if (row < p.rows) out[row] = tot.v[mt][h][n][s];
                        }
                }
            }
        }
    }

    // kDown: the CTA that ends a row tile last adds the pairs of every token, in the order of
    // top_k, so the sum does not depend on which CTA that is.
    __device__ __forceinline__ void arrive(int u) {
        __shared__ bool last;
        const int tile = u % p.tiles;
        __syncthreads();
        if (threadIdx.x == 0) {
            __threadfence();
            last = atomicAdd(&p.arrived[tile], 1u) + 1u == static_cast<unsigned>(L.groups);
        }
        __syncthreads();
        if (last) {
            __threadfence();
            combine(tile);
        }
        __syncthreads();
    }

    __device__ __forceinline__ void combine(int tile) {
        const int width = rwarps * 32, first = tile * width;
        const int n_row = min(width, p.rows - first);
        for (int i = threadIdx.x; i < static_cast<int>(p.N) * width; i += kThreads) {
            const int n = i / width, r = i % width;
            if (r >= n_row) continue;
            float y = 0.0f;
            for (int j = 0; j < p.top_k; ++j) {
                const int q = n * p.top_k + j, id = p.ids[q];
                if (id >= 0 && id < p.E)
                    y = fmaf(p.weights[q], __ldcg(p.part + static_cast<int64_t>(q) * p.rows + first + r), y);
            }
            p.Y[static_cast<int64_t>(n) * p.rows + first + r] = y;
        }
    }
};

template <int T, int M, int Terms>
__global__ void __launch_bounds__(kThreads, 2) few_kernel(const Params p) {
    using F = Few<T, M, Terms>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t bars[kWarps * F::kStages];
    Lists& L = *reinterpret_cast<Lists*>(smem + F::kRingBytes + F::kSumBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    griddep_launch_dependents();
    if (threadIdx.x < kWarps * F::kStages) mbar_init(smem_addr(&bars[threadIdx.x]), 32);
    if (threadIdx.x == 0) fence_mbar_init();
    __syncthreads();
    if (M != kDense) build_lists(p, L, reinterpret_cast<int*>(smem));
    Worker<T, M, Terms> w{p, L, smem + warp * F::kStages * F::kStageBytes,
                          reinterpret_cast<float*>(smem + F::kRingBytes), bars + warp * F::kStages};
    w.lane = lane;
    w.kwarps = 1 << p.kshift;
    w.rwarps = kWarps >> p.kshift;
    w.wk = warp & (w.kwarps - 1);
    w.wr = warp >> p.kshift;
    w.chunks = (p.kb + Fmt<T>::cb - 1) / Fmt<T>::cb;
    const int groups = M == kDense ? static_cast<int>((p.N + F::kGroup - 1) / F::kGroup) : L.groups;
    w.units = groups * p.tiles;
    w.issue_from(blockIdx.x);
    w.istage = w.cstage = 0;
    w.cphase = 0;
    w.dead = false;
    // the lists' scratch lies in the ring: its plain accesses come before the copies' writes
    if (M != kDense) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
#pragma unroll 1
    for (int i = 0; i < F::kStages; ++i) w.issue();
    griddep_wait();   // activations (and, of kDown, Y and the sums) belong to the kernel before
    if (M == kDown && groups == 0)
        for (int tile = blockIdx.x; tile < p.tiles; tile += gridDim.x) w.combine(tile);
    for (int u = blockIdx.x; u < w.units; u += gridDim.x) {
        const int n = w.count_of(w.group_of(u));
        if (n <= F::kGroup / 4)
            w.template unit<1>(u);
        else if (n <= F::kGroup / 2)
            w.template unit<2>(u);
        else
            w.template unit<4>(u);
    }
}

// ---- Preparation ------------------------------------------------------------------------

// One warp per 32-element block of X: two-term split activations in the order of `type`.
// Also zeroes the counters of the kernel after next.
__global__ void __launch_bounds__(256)
split_kernel(const float* __restrict__ X, int64_t n_blocks, int kb, int type,
             __half* __restrict__ xb, float2* __restrict__ xm, unsigned* zero, int n_zero) {
    griddep_launch_dependents();
    const int64_t warp = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < n_zero; i += blockDim.x) zero[i] = 0u;
    const int64_t step = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5;
    const int place = few_place(type, lane);
    for (int64_t b = warp; b < n_blocks; b += step) {
        const float x = X[b * 32 + lane];
        const uint32_t amax = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(x) & 0x7FFFFFFFu);
        const int e = block_exponent(amax);
        const float xs = x * pow2f(14 - e);
        const __half hi = __float2half_rn(xs);
        const __half lo = __float2half_rn(xs - __half2float(hi));
        float sum = __half2float(hi) + __half2float(lo);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        const int64_t row = b / kb, blk = b % kb;
        __half* out = xb + (row * 2 * kb + blk) * 32;
        out[place] = hi;
        out[static_cast<int64_t>(kb) * 32 + place] = lo;
        if (lane == 0) {
            const float s = pow2f(e - 14);
            xm[b] = make_float2(s, s * sum);
        }
    }
}

// One warp per block: X quantized to MXFP4, kept as fp16 values and one scale.
__global__ void __launch_bounds__(256)
mx_split_kernel(const float* __restrict__ X, int64_t n_blocks, __half* __restrict__ xb,
                float* __restrict__ xm) {
    griddep_launch_dependents();
    const int64_t warp = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    const int64_t step = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5;
    const int place = few_place(GQ_TYPE_MXFP4, lane);
    for (int64_t b = warp; b < n_blocks; b += step) {
        const float x = X[b * 32 + lane];
        const uint32_t amax = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(x) & 0x7FFFFFFFu);
        const uint32_t byte = mx_scale_byte(amax);
        uint32_t m = 0;
        if (byte != 255) m = e2m1_code(fabsf(x) * mx_inverse_scale(byte));
        const float mag = m < 4 ? 0.5f * static_cast<float>(m)
                                : static_cast<float>(m < 6 ? m - 2 : 2 * m - 8);
        xb[b * 32 + place] = __float2half_rn(copysignf(mag, x));
        if (lane == 0) xm[b] = mx_scale(byte);
    }
}

// ---- Host side --------------------------------------------------------------------------

int64_t align256(int64_t n) { return (n + 255) / 256 * 256; }

cudaError_t launch_split(const float* X, int64_t rows, int kb, int type, __half* xb, float2* xm,
                         unsigned* zero, int n_zero, const DeviceInfo* info, cudaStream_t s) {
    const int64_t blocks = rows * kb;
    const int64_t grid = std::min<int64_t>((blocks + 7) / 8, int64_t(info->sm_count) * 8);
    split_kernel<<<static_cast<unsigned>(std::max<int64_t>(grid, 1)), 256, 0, s>>>(
        X, blocks, kb, type, xb, xm, zero, n_zero);
    return cudaGetLastError();
}

// How many of a CTA's four warps split K: as many as the chunks allow while the row tiles of
// four-row-warp CTAs would leave SMs idle. `work`: tiles x groups at 32 rows a warp.
int pick_kshift(int64_t work, int chunks, int sms) {
    int ks = 0;
    while (ks < 2 && (2 << ks) <= chunks && work * (1 << ks) < int64_t(4) * 2 * sms) ++ks;
    return ks;
}

template <int T, int M, int Terms>
cudaError_t launch_few(Params& p, int64_t groups, const DeviceInfo* info, cudaStream_t s) {
    using F = Few<T, M, Terms>;
    const int chunks = (p.kb + Fmt<T>::cb - 1) / Fmt<T>::cb;
    const int64_t warp_tiles = (p.rows + 31) / 32;
    p.kshift = pick_kshift(warp_tiles * groups, chunks, info->sm_count);
    const int rwarps = kWarps >> p.kshift;
    p.tiles = static_cast<int>((warp_tiles + rwarps - 1) / rwarps);
    p.status = info->status;
    const int64_t units = p.tiles * groups;
    const unsigned grid = static_cast<unsigned>(std::max<int64_t>(
        1, std::min<int64_t>(units, int64_t(info->sm_count) * 2)));
    auto kernel = few_kernel<T, M, Terms>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, F::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = F::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<const Params>(p));
}

template <int M>
cudaError_t launch_typed(gq_type t, Params& p, int64_t groups, const DeviceInfo* info, cudaStream_t s) {
    switch (t) {
        case GQ_TYPE_Q4_0: return launch_few<GQ_TYPE_Q4_0, M, 2>(p, groups, info, s);
        case GQ_TYPE_Q8_0: return launch_few<GQ_TYPE_Q8_0, M, 2>(p, groups, info, s);
        case GQ_TYPE_Q4_K: return launch_few<GQ_TYPE_Q4_K, M, 2>(p, groups, info, s);
        case GQ_TYPE_MXFP4: return launch_few<GQ_TYPE_MXFP4, M, 2>(p, groups, info, s);
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
    p.N = n;
    p.Y = m.Y + n0 * m.M;
    return p;
}

struct MoeSpace {   // offsets in the workspace of one launch over n tokens
    int64_t xb, xm, hb, hm, part, arrived, bytes;
};

MoeSpace moe_space(const MoeProblem& m, int64_t n) {
    const int64_t pairs = n * m.top_k;
    MoeSpace s{};
    s.xb = 0;
    s.xm = s.xb + align256(n * m.D * 4);
    s.hb = s.xm + align256(n * (m.D / 32) * 8);
    s.hm = s.hb + align256(pairs * m.F * 4);
    s.part = s.hm + align256(pairs * (m.F / 32) * 8);
    s.arrived = s.part + align256(pairs * m.D * 4);
    s.bytes = s.arrived + align256((m.D / 32) * 4);
    return s;
}

int64_t moe_tokens_per_launch(const MoeProblem& m) {
    return std::min<int64_t>(m.N, kMoeMaxPairs / m.top_k);
}

}  // namespace

// ---- MXFP4 mul_mat ----------------------------------------------------------------------

int64_t few_workspace_bytes(int64_t K, int64_t N) {
    const int64_t n = std::min(N, kFewMaxTokens);
    return align256(n * K * 4) + align256(n * (K / 32) * 8);
}

// Tokens of one launch: few enough for the workspace, and for 2^30 units.
int64_t few_tokens_that_fit(int64_t M, int64_t K, int64_t N, int64_t workspace_bytes) {
    const int64_t units = std::max<int64_t>(kFewGroup2, (int64_t(1) << 30) / ((M + 31) / 32) * kFewGroup2);
    int64_t n = std::min(std::min(N, kFewMaxTokens), units);
    while (n > 0 && few_workspace_bytes(K, n) > workspace_bytes) n = n > kFewGroup2 ? n / 2 : n - 1;
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
        float2* xm = reinterpret_cast<float2*>(ws + align256(n * m.K * 4));
        p.xb = reinterpret_cast<const uint4*>(ws);
        p.xm = reinterpret_cast<const float*>(xm);
        e = launch_split(m.X + n0 * m.K, n, p.kb, GQ_TYPE_MXFP4, reinterpret_cast<__half*>(ws), xm,
                         nullptr, 0, info, s);
        if (e == cudaSuccess)
            e = launch_few<GQ_TYPE_MXFP4, kDense, 2>(p, (n + kFewGroup2 - 1) / kFewGroup2, info, s);
    }
    return e;
}

int64_t few_mx_workspace_bytes(int64_t K, int64_t N) {
    return align256(N * K * 2) + align256(N * (K / 32) * 4);
}

cudaError_t launch_few_mx4x(const MatProblem& m, int64_t N, void* workspace, cudaStream_t s) {
    DeviceInfo* info = nullptr;
    cudaError_t e = current_device_info(&info);
    if (e != cudaSuccess) return e;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    Params p = dense_params(m, 0, N);
    float* xm = reinterpret_cast<float*>(ws + align256(N * m.K * 2));
    p.xb = reinterpret_cast<const uint4*>(ws);
    p.xm = xm;
    const int64_t blocks = N * p.kb;
    const int64_t grid = std::min<int64_t>((blocks + 7) / 8, int64_t(info->sm_count) * 8);
    mx_split_kernel<<<static_cast<unsigned>(grid), 256, 0, s>>>(
        m.X, blocks, reinterpret_cast<__half*>(ws), xm);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_few<GQ_TYPE_MXFP4, kDense, 1>(p, (N + kFewGroup1 - 1) / kFewGroup1, info, s);
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
        unsigned* arrived = reinterpret_cast<unsigned*>(ws + at.arrived);
        // groups there can be: every pair its own expert, or full groups over few experts
        const int64_t groups = std::min<int64_t>(pairs, m.E + pairs / kFewGroup2);
        Params g{};
        g.W = m.W_gate;
        g.W2 = m.W_up;
        g.row_bytes = row_bytes_of(m.t, m.D);
        g.total_bytes = g.row_bytes * m.F * m.E;
        g.rows = static_cast<int>(m.F);
        g.kb = static_cast<int>(m.D / 32);
        g.xb = reinterpret_cast<const uint4*>(ws + at.xb);
        g.xm = reinterpret_cast<const float*>(ws + at.xm);
        g.N = n;
        g.E = static_cast<int>(m.E);
        g.top_k = m.top_k;
        g.pairs = pairs;
        g.ids = m.ids + n0 * m.top_k;
        g.weights = m.weights + n0 * m.top_k;
        g.hb = reinterpret_cast<__half*>(ws + at.hb);
        g.hm = reinterpret_cast<float2*>(ws + at.hm);
        g.h_type = m.t_down;
        Params d = g;
        d.W = m.W_down;
        d.W2 = nullptr;
        d.row_bytes = row_bytes_of(m.t_down, m.F);
        d.total_bytes = d.row_bytes * m.D * m.E;
        d.rows = static_cast<int>(m.D);
        d.kb = static_cast<int>(m.F / 32);
        d.xb = reinterpret_cast<const uint4*>(ws + at.hb);
        d.xm = reinterpret_cast<const float*>(ws + at.hm);
        d.Y = m.Y + n0 * m.D;
        d.part = reinterpret_cast<float*>(ws + at.part);
        d.arrived = arrived;
        e = launch_split(m.X + n0 * m.D, n, g.kb, m.t, reinterpret_cast<__half*>(ws + at.xb),
                         reinterpret_cast<float2*>(ws + at.xm), arrived, static_cast<int>(m.D / 32),
                         info, s);
        if (e == cudaSuccess) e = launch_typed<kGateUp>(m.t, g, groups, info, s);
        if (e == cudaSuccess) e = launch_typed<kDown>(m.t_down, d, groups, info, s);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace gq
