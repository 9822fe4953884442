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
// Layout of the work. One persistent CTA per SM, 16 warps, and a ring of stages, each some weight
// rows x up to 64 blocks of K, one bulk copy per row: runs of about a kilobyte, which is what DRAM pages and the copy engine want (16-
// byte cp.async in 136-byte runs reached 3.3 TB/s, bulk copies of 136 bytes 1.6). A row's copy
// starts at the 16-byte word that holds its first byte, because rows of 17- and 18-byte blocks
// start anywhere; words are aligned in registers. The warps split a stage's K range
// (kwarps), four blocks of 32 rows each, so that the activations of those four blocks stay in
// registers from stage to stage; then their sums join through shared memory in a fixed order, and the
// barrier of that join frees the stage for its refill.
// The ring runs on across units, and weights do not depend on the kernel before, so they start
// to stream before griddepcontrol.wait.
#include <algorithm>
#include <atomic>
#include <cstddef>

#include "gq_few.cuh"

namespace gq {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxBlocks = 4;              // of one warp and stage

constexpr int64_t kFewMaxTokens = 4096;   // of one launch: bounds the workspace

enum Mode { kDense = 0, kGateUp = 1, kDown = 2 };

template <int T>
struct Fmt;   // bytes of 32 weights, and the 16-row tiles that a consumer warp takes of a stage
template <>
struct Fmt<GQ_TYPE_Q4_0> {
    static constexpr int bb = kQ4Bytes, tiles = 2;
};
template <>
struct Fmt<GQ_TYPE_Q8_0> {
    static constexpr int bb = kQ8Bytes, tiles = 1;   // twice the bytes: the same stage
};
template <>
struct Fmt<GQ_TYPE_Q4_K> {   // a super-block's bytes over its 8 sub-blocks
    static constexpr int bb = kQ4KBytes / 8, tiles = 2;
};
template <>
struct Fmt<GQ_TYPE_MXFP4> {
    static constexpr int bb = kMxfp4Bytes, tiles = 2;
};

struct Params {
    const uint8_t* W;
    const uint8_t* W2;        // kGateUp: the up matrices
    int64_t total_bytes;      // of W (and of W2)
    int64_t row_bytes;
    int rows;                 // weight rows (of one expert)
    int kb;                   // 32-weight blocks per row
    int kc;                   // blocks of one stage (chunk) of a row
    int chunks;               // ceil(kb / kc)
    int kwarps;               // consumer warps that split a chunk, `per` blocks each
    int per;
    int units;                // of one group: row tiles of unit_rows
    int pitch, stage_bytes;   // of a staged row, of a stage
    int stages;
    const uint4* xb;          // split activations, 64 bytes per (row, term, block)
    const float* xm;          // their block factors: float2 (two terms) or float (one)
    int64_t N;                // tokens
    int E, top_k, pairs;
    const int* ids;
    float* Y;                 // kDense
    __half* hb;               // kGateUp: split activations of the result,
    float2* hm;
    int h_type;               //          in the order of the down matrices' type
    float* part;              // kDown: [pair][rows]
    unsigned* status;
};

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
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

// Byte i of w as fp32: 2^23 + byte under the exponent, less 2^23 (no conversion unit).
__device__ __forceinline__ float byte_to_float(uint32_t w, int i) {
    return __uint_as_float(__byte_perm(w, 0x4B000000u, i ? 0x7651 : 0x7650)) - 8388608.0f;
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
    uint4 b[NT];               // eight fp16 of column g
    float2 m[NT];              // {scale, sum} of token t (two terms), scales of 2t, 2t + 1 (one)
};

// Products of one 16-row tile with one block, for NT column tiles: tot += d_row s_token (codes
// . columns), less m_row sum_token for Q4_K. tot: [column tile][rows g, g + 8][tokens].
template <int T, int Terms, int NT>
__device__ __forceinline__ void block_products(const uint32_t (&q)[2][4], const float (&d)[2],
                                               const float (&m)[2], const Columns<NT, Terms>& col,
                                               float (&tot)[NT][2][3 - Terms]) {
    float c[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
        mma_first(c[n], q[0][0], q[1][0], q[0][1], q[1][1], col.b[n].x, col.b[n].y);
#pragma unroll
    for (int n = 0; n < NT; ++n)
        mma_next(c[n], q[0][2], q[1][2], q[0][3], q[1][3], col.b[n].z, col.b[n].w);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if constexpr (Terms == 2) {
                tot[n][h][0] = fmaf(d[h] * col.m[n].x, c[n][2 * h] + c[n][2 * h + 1], tot[n][h][0]);
                if constexpr (T == GQ_TYPE_Q4_K) tot[n][h][0] = fmaf(-m[h], col.m[n].y, tot[n][h][0]);
            } else {
                tot[n][h][0] = fmaf(d[h] * col.m[n].x, c[n][2 * h], tot[n][h][0]);
                tot[n][h][1] = fmaf(d[h] * col.m[n].y, c[n][2 * h + 1], tot[n][h][1]);
            }
        }
}

// The shared lists of a launch over experts: pairs sorted by expert, and groups of up to
// kFewGroup pairs of one expert.
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
            const int g = (c + kFewGroup - 1) / kFewGroup;
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
                L.start[group0 + i] = static_cast<uint16_t>(pair0 + i * kFewGroup);
                L.count[group0 + i] = static_cast<uint8_t>(min(kFewGroup, c - i * kFewGroup));
            }
            if (e < p.E) count[e] = pair0;
            base += __shfl_sync(0xFFFFFFFFu, incl, 31);
        }
        if (threadIdx.x == 0) L.groups = base >> 16;
    }
    __syncthreads();
    for (int q = threadIdx.x; q < p.pairs; q += kThreads)
        if (ids[q] >= 0) L.pair[count[ids[q] & 0xFFFF] + (ids[q] >> 16)] = static_cast<uint16_t>(q);
    __syncthreads();
}

// One warp writes a block of a split activation row: lane i holds element i. `xb` and `xm` are
// the row's places of this block; `lo_at` the distance from hi to lo.
__device__ __forceinline__ void write_split(float x, int lane, int place, __half* xb, int64_t lo_at,
                                            float2* xm) {
    const uint32_t amax = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(x) & 0x7FFFFFFFu);
    const int e = block_exponent(amax);
    const float xs = x * pow2f(14 - e);
    const __half hi = __float2half_rn(xs);
    const __half lo = __float2half_rn(xs - __half2float(hi));
    float sum = __half2float(hi) + __half2float(lo);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    xb[place] = hi;
    xb[lo_at + place] = lo;
    if (lane == 0) {
        const float s = pow2f(e - 14);
        *xm = make_float2(s, s * sum);
    }
}

// Shared memory: the lists (and, of kGateUp, the hidden values of a unit), the consumers' sums,
// the ring.
constexpr int kSumFloats = 2 * kWarps * 32 * (kFewGroup + 1);   // two halves, in turn
constexpr int kHiddenFloats = 64 * (kFewGroup + 1);
constexpr int kListBytes = (static_cast<int>(sizeof(Lists)) + 127) / 128 * 128;
constexpr int kRingAt = kListBytes + (kSumFloats + kHiddenFloats) * 4;
constexpr int kMaxStages = 5;
constexpr int kSmemMax = 227 * 1024 - 512;   // 512: the barriers and what else is static
static_assert(kRingAt % 128 == 0 && (kMoeMaxExperts + kMoeMaxPairs) * 4 <= kSumFloats * 4,
              "the lists' scratch lies in the sums");

// A unit: group, row tile, and how many this CTA has from here on.
struct Place {
    int gi, tile;
    int64_t left;
    __device__ __forceinline__ void next(int units) {
        --left;
        if (++tile == units) {
            tile = 0;
            ++gi;
        }
    }
};

template <int T, int M, int Terms>
struct Worker {
    static constexpr int kTiles = Fmt<T>::tiles;
    static constexpr int kBB = Fmt<T>::bb;
    const Params& p;
    const Lists& L;
    float* sums;
    float* hidden;
    uint32_t ring, full;          // shared addresses
    int lane, warp;
    int stage_rows;               // staged rows
    int sub;                      // stages of a unit and chunk (kGateUp: a unit is whole 32-blocks)
    int res_shift;                // log2 of a stage's result rows
    int groups;
    Place f;                      // the next stage to fill: unit,
    int fs, fc, fslot;            // stage in it, chunk; slot
    bool dead;

    __device__ __forceinline__ int expert_of(int gi) const { return M == kDense ? 0 : L.expert[gi]; }
    __device__ __forceinline__ int count_of(int gi) const {
        if (M != kDense) return L.count[gi];
        return static_cast<int>(min(static_cast<int64_t>(kFewGroup),
                                    p.N - static_cast<int64_t>(gi) * kFewGroup));
    }
    // activation row of column token i of a group
    __device__ __forceinline__ int64_t x_row(int gi, int i) const {
        if (M == kDense) return static_cast<int64_t>(gi) * kFewGroup + i;
        const int q = L.pair[L.start[gi] + i];
        return M == kGateUp ? q / p.top_k : q;
    }
    // Result rows of a stage; a kGateUp tile is 8 gate rows and the 8 up rows of the same numbers.
    __device__ __forceinline__ int first_row(int tile, int s) const { return (tile * sub + s) << res_shift; }
    __device__ __forceinline__ static int row_in_stage(int sr) {
        return M == kGateUp ? (sr >> 4) * 8 + (sr & 7) : sr;
    }

    // ---- copies ----

    // Starts the copies of the next stage, if there is one: warp w copies rows w, w + 16, ... of
    // up to 128, a lane each. Every row arrives once on the stage's barrier.
    __device__ __forceinline__ void fill() {
        if (f.left == 0) return;
        const int sr = warp + kWarps * lane;
        if (sr < stage_rows) {
            const uint32_t dst = ring + fslot * p.stage_bytes + sr * p.pitch;
            const uint32_t bar = full + 8 * fslot;
            const int r = ((f.tile * sub + fs) << res_shift) + row_in_stage(sr);
            const uint8_t* W = M == kGateUp && (sr & 8) ? p.W2 : p.W;
            uint32_t n = 0;
            int64_t from = 0;
            if (r < p.rows) {
                const int64_t row = static_cast<int64_t>(expert_of(f.gi)) * p.rows + r;
                const int64_t start = row * p.row_bytes + fc * p.kc * kBB;
                from = start & ~static_cast<int64_t>(15);
                int64_t to = (start + min(p.kc, p.kb - fc * p.kc) * kBB + 15) & ~static_cast<int64_t>(15);
                if (to > p.total_bytes) {   // the matrix ends inside its last 16-byte word
                    to = p.total_bytes & ~static_cast<int64_t>(15);
                    for (int64_t k = to > from ? to : from; k < p.total_bytes; ++k)
                        asm volatile("st.shared.u8 [%0], %1;" ::"r"(dst + static_cast<uint32_t>(k - from)),
                                     "r"(static_cast<uint32_t>(W[k])) : "memory");
                }
                if (to > from) n = static_cast<uint32_t>(to - from);
            }
            // the stage's plain reads, before the barrier that brought us here, come first
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            mbar_arrive_expect_tx(bar, n);
            if (n > 0) bulk_g2s_evict_first(dst, W + from, n, bar);
        }
        if (++fslot == p.stages) fslot = 0;
        if (++fc == p.chunks) {
            fc = 0;
            if (++fs == sub) {
                fs = 0;
                f.next(p.units);
            }
        }
    }

    // Waits for the stage at hand. After a wait that ran out, and an equal one for the other
    // stages that are under way, goes on without waiting: the results are lost.
    __device__ __forceinline__ void wait_stage(int slot, uint32_t phase) {
        if (dead || __all_sync(0xFFFFFFFFu, mbar_wait(full + 8 * slot, phase))) return;
        dead = true;
        report_status(p.status, kStatusTimeout);
        for (int i = 1; i < p.stages; ++i) {
            if (++slot == p.stages) {
                slot = 0;
                phase ^= 1;
            }
            mbar_wait(full + 8 * slot, phase);
        }
    }

    // ---- products ----

    template <int NT>
    struct Acts {
        Columns<NT, Terms> col[kMaxBlocks];
    };

    // This lane's share of nb blocks from block kb0 of the group's activations. Columns of
    // tokens that the group does not have read token 0's: nothing uses them.
    template <int NT>
    __device__ __forceinline__ void load_acts(Acts<NT>& a, int gi, int n_tok, int kb0, int nb) const {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int i = Terms == 2 ? 4 * n + (g >> 1) : 8 * n + g;
            const int64_t row = x_row(gi, i < n_tok ? i : 0) * Terms + (Terms == 2 ? g & 1 : 0);
            const uint4* xp = p.xb + (row * p.kb + kb0) * 4 + t;
#pragma unroll
            for (int b = 0; b < kMaxBlocks; ++b)
                if (b < nb) a.col[b].b[n] = xp[b * 4];
            if constexpr (Terms == 2) {
                const int j = 4 * n + t;
                const float2* mp = reinterpret_cast<const float2*>(p.xm) + x_row(gi, j < n_tok ? j : 0) * p.kb + kb0;
#pragma unroll
                for (int b = 0; b < kMaxBlocks; ++b)
                    if (b < nb) a.col[b].m[n] = mp[b];
            } else {
                const int j0 = 8 * n + 2 * t;
                const float* m0 = p.xm + x_row(gi, j0 < n_tok ? j0 : 0) * p.kb + kb0;
                const float* m1 = p.xm + x_row(gi, j0 + 1 < n_tok ? j0 + 1 : 0) * p.kb + kb0;
#pragma unroll
                for (int b = 0; b < kMaxBlocks; ++b)
                    if (b < nb) a.col[b].m[n] = make_float2(m0[b], m1[b]);
            }
        }
    }

    // nb blocks, from block kb0 of the row (kq0 of the chunk), of this warp's rows of a stage.
    template <int NT>
    __device__ __forceinline__ void products(float (&tot)[kTiles][NT][2][3 - Terms], const Acts<NT>& a,
                                             uint32_t stage, uint32_t row0, int c, int kq0, int nb) const {
        const int g = lane >> 2, t = lane & 3;
        const int wr = warp / p.kwarps;
        // Where this lane's rows begin: the staged word's offset (0..15) of their chunk. Rows g
        // and g + 8 of every tile agree in the low two bits, as eight rows are a multiple of 8
        // bytes.
        uint32_t base[kTiles][2];
#pragma unroll
        for (int ti = 0; ti < kTiles; ++ti)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int sr = (wr * kTiles + ti) * 16 + 8 * h + g;
                const uint32_t mis = ((row0 + row_in_stage(sr)) * static_cast<uint32_t>(p.row_bytes) +
                                      static_cast<uint32_t>(c * p.kc) * kBB) & 15u;
                base[ti][h] = stage + sr * p.pitch + mis;
            }
        if constexpr (T == GQ_TYPE_Q4_K) {
            // four (or two) sub-blocks of one super-block
            const int in = (kq0 & 7) >> 1;
#pragma unroll
            for (int ti = 0; ti < kTiles; ++ti) {
                uint4 hd[2];
                float D[2], Dm[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    base[ti][h] += (kq0 >> 3) * kQ4KBytes;
                    hd[h] = lds128(base[ti][h]);
                    base[ti][h] += 16 + 32 * in + 4 * t;
                    D[h] = half_bits_to_float(hd[h].x);
                    Dm[h] = half_bits_to_float(hd[h].x >> 16);
                }
#pragma unroll
                for (int b = 0; b < kMaxBlocks; b += 2) {
                    if (b >= nb) break;
                    uint32_t w[2][2], sc[2], mn[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        w[h][0] = lds32(base[ti][h] + 16 * b);
                        w[h][1] = lds32(base[ti][h] + 16 + 16 * b);
                        q4k_scales(hd[h], in + (b >> 1), sc[h], mn[h]);
                    }
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        uint32_t q[2][4];
                        float d[2], m[2];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t mask = s ? 0x00F000F0u : 0x000F000Fu;
                            q[h][0] = (w[h][0] & mask) | kMagic;
                            q[h][1] = ((w[h][0] >> 8) & mask) | kMagic;
                            q[h][2] = (w[h][1] & mask) | kMagic;
                            q[h][3] = ((w[h][1] >> 8) & mask) | kMagic;
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                q[h][i] = s ? h2_fma(q[h][i], kSixteenth, 0xD400D400u)
                                            : h2_sub(q[h][i], kMagic);
                            d[h] = D[h] * byte_to_float(sc[h], s);
                            m[h] = Dm[h] * byte_to_float(mn[h], s);
                        }
                        block_products<T, Terms, NT>(q, d, m, a.col[b + s], tot[ti]);
                    }
                }
            }
        } else {
#pragma unroll
            for (int ti = 0; ti < kTiles; ++ti)
#pragma unroll
                for (int h = 0; h < 2; ++h) base[ti][h] += kq0 * kBB;
            // Unaligned words: the aligned word at (base + delta[j] + 4-multiple) and its
            // successor, shifted by shift[j], for byte offsets congruent j modulo 4.
            const uint32_t r3 = base[0][0] & 3u;
            int delta[4];
            uint32_t shift[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                delta[j] = (r3 + j >= 4 ? 4 : 0) - static_cast<int>(r3) + 4 * t;
                shift[j] = (r3 + j) << 3;   // the funnel shift takes it modulo 32
            }
#pragma unroll
            for (int b = 0; b < kMaxBlocks; ++b) {
                if (b >= nb) break;
#pragma unroll
                for (int ti = 0; ti < kTiles; ++ti) {
                    uint32_t q[2][4];
                    float d[2], m[2] = {0.0f, 0.0f};
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        constexpr int kHead = T == GQ_TYPE_MXFP4 ? 1 : 2;
                        const int off = b * kBB + kHead;
                        const uint32_t at = base[ti][h] + delta[off & 3] + (off & ~3);
                        const uint32_t w0 = __funnelshift_r(lds32(at), lds32(at + 4), shift[off & 3]);
                        if constexpr (T == GQ_TYPE_Q8_0) {
                            const uint32_t w1 = __funnelshift_r(lds32(at + 16), lds32(at + 20), shift[off & 3]);
                            const uint32_t u0 = w0 ^ 0x80808080u, u1 = w1 ^ 0x80808080u;
                            // 1024 + 128 + code, byte by byte under the exponent
                            q[h][0] = h2_sub(__byte_perm(u0, 0x64u, 0x4140), 0x64806480u);
                            q[h][1] = h2_sub(__byte_perm(u0, 0x64u, 0x4342), 0x64806480u);
                            q[h][2] = h2_sub(__byte_perm(u1, 0x64u, 0x4140), 0x64806480u);
                            q[h][3] = h2_sub(__byte_perm(u1, 0x64u, 0x4342), 0x64806480u);
                        } else if constexpr (T == GQ_TYPE_Q4_0) {
                            nibbles_to_f16<8>(w0, q[h]);
                        } else {
                            e2m1_to_f16(w0, q[h]);
                        }
                        if constexpr (T != GQ_TYPE_MXFP4) d[h] = half_bits_to_float(lds16(base[ti][h] + b * kBB));
                    }
                    if constexpr (T == GQ_TYPE_MXFP4)
                        e8m0_to_f32(lds8(base[ti][0] + b * kBB), lds8(base[ti][1] + b * kBB), d[0], d[1]);
                    block_products<T, Terms, NT>(q, d, m, a.col[b], tot[ti]);
                }
            }
        }
    }

    // The units of this CTA from `at` on whose groups have as many tokens as NT column tiles are
    // for.
    template <int NT>
    __device__ __forceinline__ void consume(Place& at, int& slot, uint32_t& phase) {
        constexpr int kTile = 4 * (3 - Terms);
        constexpr int kPitch = NT * kTile + 1;   // of a row of sums
        const int wk = warp & (p.kwarps - 1);
        const int kq0 = wk * p.per;
        Acts<NT> acts;
        int held = -1, side = 0;
        __syncthreads();   // the sums are free
#pragma unroll 1
        for (; at.left > 0; at.next(p.units)) {
            const int n_tok = count_of(at.gi);
            if (n_tok > NT * kTile || n_tok <= (NT - 1) * kTile) break;
            const uint32_t e_row = static_cast<uint32_t>(expert_of(at.gi)) * static_cast<uint32_t>(p.rows);
#pragma unroll 1
            for (int s = 0; s < sub; ++s) {
                float tot[kTiles][NT][2][3 - Terms];
#pragma unroll
                for (int i = 0; i < kTiles * NT * 2 * (3 - Terms); ++i) (&tot[0][0][0][0])[i] = 0.0f;
                const int row0 = first_row(at.tile, s);
#pragma unroll 1
                for (int c = 0; c < p.chunks; ++c) {
                    const int nb = min(p.per, min(p.kc, p.kb - c * p.kc) - kq0);
                    if (held != at.gi || p.chunks > 1) {
                        load_acts<NT>(acts, at.gi, n_tok, c * p.kc + kq0, nb);
                        held = at.gi;
                    }
                    wait_stage(slot, phase);
                    if (nb > 0) products<NT>(tot, acts, ring + slot * p.stage_bytes, e_row + row0, c, kq0, nb);
                    if (++slot == p.stages) {
                        slot = 0;
                        phase ^= 1;
                    }
                    if (c + 1 < p.chunks) {   // after the last chunk, the join's barrier does this
                        __syncthreads();
                        if (!dead) fill();
                    }
                }
                // Two halves of the sums in turn: one barrier is enough.
                float* const half = sums + (side ? kSumFloats / 2 : 0);
                side ^= 1;
                float* mine = half + (warp * kTiles * 16 + (lane >> 2)) * kPitch;
#pragma unroll
                for (int ti = 0; ti < kTiles; ++ti)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int i = 0; i < 3 - Terms; ++i) {
                                const int tok = Terms == 2 ? 4 * n + (lane & 3) : 8 * n + 2 * (lane & 3) + i;
                                mine[(16 * ti + 8 * h) * kPitch + tok] = tot[ti][n][h][i];
                            }
                __syncthreads();
                if (!dead) fill();
                finish<kPitch>(half, at.gi, n_tok, s, row0);
            }
            if constexpr (M == kGateUp) split_hidden(at.gi, n_tok, at.tile);
        }
    }

    // Staged row sr, token i: the K warps' sums in their order.
    template <int Pitch>
    __device__ __forceinline__ float joined(const float* at, int sr, int i) const {
        constexpr int kRows = 16 * kTiles;
        const float* from = at + ((sr / kRows) * p.kwarps * kRows + sr % kRows) * Pitch + i;
        float v = 0.0f;
        for (int k = 0; k < p.kwarps; k += 4) {   // 4, 8 or 16 of them
            float x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = from[(k + j) * kRows * Pitch];
#pragma unroll
            for (int j = 0; j < 4; ++j) v += x[j];
        }
        return v;
    }

    template <int Pitch>
    __device__ __forceinline__ void finish(const float* at, int gi, int n_tok, int s, int row0) const {
        for (int i = threadIdx.x; i < (n_tok << res_shift); i += kThreads) {
            const int r = i & ((1 << res_shift) - 1), tok = i >> res_shift;
            if constexpr (M == kGateUp) {
                const int sr = (r >> 3) * 16 + (r & 7);
                const float gate = joined<Pitch>(at, sr, tok), up = joined<Pitch>(at, sr + 8, tok);
                hidden[((s << res_shift) + r) * (kFewGroup + 1) + tok] = gate / (1.0f + expf(-gate)) * up;
            } else if (row0 + r < p.rows) {
                float* const out = M == kDown ? p.part : p.Y;
                out[x_row(gi, tok) * p.rows + row0 + r] = joined<Pitch>(at, r, tok);
            }
        }
    }

    // kGateUp: the unit's hidden values to split activations, one warp per (block, token).
    __device__ __forceinline__ void split_hidden(int gi, int n_tok, int tile) const {
        __syncthreads();
        const int blocks = (sub << res_shift) / 32;   // 1 or 2
        const int hb = p.rows / 32;
        const int place = few_place(p.h_type, lane);
        for (int i = warp; i < blocks * n_tok; i += kWarps) {
            const int bl = i & (blocks - 1), tok = i / blocks;
            const int blk = tile * blocks + bl;
            if (blk >= hb) continue;
            const int64_t q = L.pair[L.start[gi] + tok];
            write_split(hidden[(32 * bl + lane) * (kFewGroup + 1) + tok], lane, place,
                        p.hb + (q * 2 * hb + blk) * 32, hb * 32, p.hm + q * hb + blk);
        }
    }
};

template <int T, int M, int Terms>
__global__ void __launch_bounds__(kThreads, 1) few_kernel(const __grid_constant__ Params p) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t bars[kMaxStages];
    Lists& L = *reinterpret_cast<Lists*>(smem);
    float* const sums = reinterpret_cast<float*>(smem + kListBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    griddep_launch_dependents();
    Worker<T, M, Terms> w{p, L, sums, sums + kSumFloats, smem_addr(smem) + kRingAt, smem_addr(bars), lane, warp};
    w.stage_rows = 16 * Fmt<T>::tiles * (kWarps / p.kwarps);
    if (threadIdx.x < p.stages) mbar_init(smem_addr(&bars[threadIdx.x]), w.stage_rows);
    if (threadIdx.x == 0) fence_mbar_init();
    if (M != kDense) build_lists(p, L, reinterpret_cast<int*>(sums));
    __syncthreads();
    w.res_shift = 31 - __clz(M == kGateUp ? w.stage_rows / 2 : w.stage_rows);
    w.sub = M == kGateUp ? max(1, 32 >> w.res_shift) : 1;
    w.groups = M == kDense ? static_cast<int>((p.N + kFewGroup - 1) / kFewGroup) : L.groups;
    // consecutive units for each CTA: those of one group follow each other
    const int64_t total = static_cast<int64_t>(w.groups) * p.units;
    const int64_t begin = total * blockIdx.x / gridDim.x;
    Place at{static_cast<int>(begin / p.units), static_cast<int>(begin % p.units),
             total * (blockIdx.x + 1) / gridDim.x - begin};
    w.f = at;
    w.fs = w.fc = w.fslot = 0;
    w.dead = false;
#pragma unroll 1
    for (int i = 0; i < p.stages; ++i) w.fill();
    griddep_wait();   // activations (and what this kernel writes) belong to the kernels before
    int slot = 0;
    uint32_t phase = 0;
#pragma unroll 1
    while (at.left > 0) {
        if (w.count_of(at.gi) <= 4 * (3 - Terms)) {
            w.template consume<1>(at, slot, phase);
        } else {
            if constexpr (Terms == 2) w.template consume<2>(at, slot, phase);
        }
    }
}

// Y[n] = sum_j weights[n][j] part[n][j], over the pairs that have an expert, in the order of j.
__global__ void __launch_bounds__(256)
combine_kernel(const float* __restrict__ part, const int* __restrict__ ids,
               const float* __restrict__ weights, int64_t N, int top_k, int E, int D,
               float* __restrict__ Y) {
    griddep_wait();   // `part`, and Y, which the kernels before may still read as X
    const int quads = D / 4;
    const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < N * quads; i += step) {
        const int64_t n = i / quads;
        const int r = static_cast<int>(i - n * quads);
        float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
        for (int j = 0; j < top_k; ++j) {
            const int64_t q = n * top_k + j;
            const int id = ids[q];
            if (id < 0 || id >= E) continue;
            const float w = weights[q];
            const float4 v = reinterpret_cast<const float4*>(part)[q * quads + r];
            y.x = fmaf(w, v.x, y.x);
            y.y = fmaf(w, v.y, y.y);
            y.z = fmaf(w, v.z, y.z);
            y.w = fmaf(w, v.w, y.w);
        }
        float* out = Y + n * D + 4 * r;   // only 4-byte aligned
        out[0] = y.x;
        out[1] = y.y;
        out[2] = y.z;
        out[3] = y.w;
    }
}

// ---- Preparation ------------------------------------------------------------------------

// One warp per 32-element block of X: two-term split activations in the order of `type`.
__global__ void __launch_bounds__(256)
split_kernel(const float* __restrict__ X, int64_t n_blocks, int kb, int type,
             __half* __restrict__ xb, float2* __restrict__ xm) {
    griddep_launch_dependents();
    const int64_t warp = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    const int64_t step = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5;
    const int place = few_place(type, lane);
    for (int64_t b = warp; b < n_blocks; b += step) {
        const int64_t row = b / kb, blk = b % kb;
        write_split(X[b * 32 + lane], lane, place, xb + (row * 2 * kb + blk) * 32,
                    static_cast<int64_t>(kb) * 32, xm + b);
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
                         const DeviceInfo* info, cudaStream_t s) {
    const int64_t blocks = rows * kb;
    const int64_t grid = std::min<int64_t>((blocks + 7) / 8, int64_t(info->sm_count) * 8);
    split_kernel<<<static_cast<unsigned>(std::max<int64_t>(grid, 1)), 256, 0, s>>>(
        X, blocks, kb, type, xb, xm);
    return cudaGetLastError();
}

// A launch that may start while the kernel before it on the stream still runs (it waits with
// griddep_wait).
template <typename... Sig, typename... Args>
cudaError_t launch_after(void (*kernel)(Sig...), unsigned grid, int threads, int smem, cudaStream_t s,
                         const Args&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int T, int M, int Terms>
cudaError_t launch_few(Params& p, int64_t groups, const DeviceInfo* info, cudaStream_t s) {
    // Chunks of up to 64 blocks (four for each of the 16 consumer warps), of equal size but for
    // the last; with fewer blocks, fewer warps share a chunk and a stage has more rows.
    constexpr int kMax = kWarps * kMaxBlocks;
    constexpr int kUnit = T == GQ_TYPE_Q4_K ? 8 : 1;   // super-blocks stay whole
    p.chunks = (p.kb + kMax - 1) / kMax;
    p.kc = ((p.kb + p.chunks - 1) / p.chunks + kUnit - 1) / kUnit * kUnit;
    p.kwarps = p.kc > kMax / 2 ? kWarps : (p.kc > kMax / 4 ? kWarps / 2 : kWarps / 4);
    p.per = (p.kc + p.kwarps - 1) / p.kwarps;
    if (T == GQ_TYPE_Q4_K) p.per = (p.per + 1) / 2 * 2 == 2 ? 2 : 4;   // inside one super-block
    const int stage_rows = 16 * Fmt<T>::tiles * (kWarps / p.kwarps);
    const int results = M == kGateUp ? stage_rows / 2 : stage_rows;
    const int unit_rows = M == kGateUp ? std::max(32, results) : results;
    p.units = (p.rows + unit_rows - 1) / unit_rows;
    // A row's words, at an odd multiple of 16 bytes: the eight rows that a warp reads at once
    // then lie on distinct groups of four banks.
    p.pitch = (p.kc * Fmt<T>::bb + 15 + 15) / 16 * 16;
    if (p.pitch % 32 == 0) p.pitch += 16;
    p.stage_bytes = (stage_rows * p.pitch + 16 + 127) / 128 * 128;   // 16: the last word's second half
    p.stages = std::min(kMaxStages, (kSmemMax - kRingAt) / p.stage_bytes);
    p.status = info->status;
    const unsigned grid = static_cast<unsigned>(
        std::max<int64_t>(1, std::min<int64_t>(p.units * groups, info->sm_count)));
    const int smem = kRingAt + p.stages * p.stage_bytes;
    auto kernel = few_kernel<T, M, Terms>;
    static std::atomic<uint64_t> ready{0};   // devices whose attribute is set
    const uint64_t bit = uint64_t(1) << info->device;
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        const cudaError_t e =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    return launch_after(kernel, grid, kThreads, smem, s, static_cast<const Params&>(p));
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
    int64_t xb, xm, hb, hm, part, bytes;
};

MoeSpace moe_space(const MoeProblem& m, int64_t n) {
    const int64_t pairs = n * m.top_k;
    MoeSpace s{};
    s.xb = 0;
    s.xm = s.xb + align256(n * m.D * 4);
    s.hb = s.xm + align256(n * (m.D / 32) * 8);
    s.hm = s.hb + align256(pairs * m.F * 4);
    s.part = s.hm + align256(pairs * (m.F / 32) * 8);
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
    return align256(n * K * 4) + align256(n * (K / 32) * 8);
}

// Tokens of one launch: few enough for the workspace, and for 2^30 units.
int64_t few_tokens_that_fit(int64_t M, int64_t K, int64_t N, int64_t workspace_bytes) {
    const int64_t units = std::max<int64_t>(kFewGroup, (int64_t(1) << 30) / ((M + 31) / 32) * kFewGroup);
    int64_t n = std::min(std::min(N, kFewMaxTokens), units);
    while (n > 0 && few_workspace_bytes(K, n) > workspace_bytes) n = n > kFewGroup ? n / 2 : n - 1;
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
                         info, s);
        if (e == cudaSuccess)
            e = launch_few<GQ_TYPE_MXFP4, kDense, 2>(p, (n + kFewGroup - 1) / kFewGroup, info, s);
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
    return launch_few<GQ_TYPE_MXFP4, kDense, 1>(p, (N + kFewGroup - 1) / kFewGroup, info, s);
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
        // groups there can be: every pair its own expert, or full groups over few experts
        const int64_t groups = std::min<int64_t>(pairs, m.E + pairs / kFewGroup);
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
        d.part = reinterpret_cast<float*>(ws + at.part);
        e = launch_split(m.X + n0 * m.D, n, g.kb, m.t, reinterpret_cast<__half*>(ws + at.xb),
                         reinterpret_cast<float2*>(ws + at.xm), info, s);
        if (e == cudaSuccess) e = launch_typed<kGateUp>(m.t, g, groups, info, s);
        if (e == cudaSuccess) e = launch_typed<kDown>(m.t_down, d, groups, info, s);
        if (e == cudaSuccess) {
            const int64_t blocks = (n * (m.D / 4) + 255) / 256;
            e = launch_after(combine_kernel, static_cast<unsigned>(std::min<int64_t>(blocks, info->sm_count * 8)),
                             256, 0, s, static_cast<const float*>(d.part), g.ids, m.weights + n0 * m.top_k,
                             n, m.top_k, g.E, d.rows, m.Y + n0 * m.D);
        }
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace gq
