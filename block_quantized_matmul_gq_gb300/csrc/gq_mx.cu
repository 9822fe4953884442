// gq_mx.cu -- the microscaled mul_mat: MXFP4 weights times X quantized to MXFP4, on the
// block-scaled tensor cores.
//
// Mathematics. Y[n][m] = sum_b 2^(s_w[m][b] + s_x[n][b]) sum_{k in b} w_k x_k over 32-element
// blocks of E2M1 values. tcgen05.mma kind::mxf4 takes exactly this: packed E2M1 operands, one
// E8M0 scale per row and block, fp32 accumulators in TMEM. Every product and scale is exact, so
// the sums are the only roundings. The order of the 32 values inside a block does not matter as
// long as both sides agree, so the codes keep the file's arrangement (value j beside j + 16) and
// X is packed likewise: no weight is unpacked anywhere.
//
// Two launches. mx_prepare_kernel lays both operands out as the MMA reads them: records of
// 128 weight rows (kBN token rows) x 256 k, i.e. rows of 128 bytes in the 128-byte swizzle, then
// the scales as 32-row x 16-byte atoms (row r's four scales at (r % 32) 16 + (r / 32) 4), so that
// one bulk copy brings a stage's operand. X is quantized on the way. This costs the weights one
// more read and write (15 us of 65 for 11008 x 4096 times 2048 tokens); laid out inside the
// product it would be paid again for every token tile, and would put warps between the copies and
// the MMA.
//
// mx_gemm_kernel: one persistent CTA per SM; one thread copies, one issues MMAs (four of K = 64
// a stage), four warps bring a stage's scales from shared memory to TMEM, four read one accumulator
// out while the other fills. (With copies of the scales issued by the MMA thread, six a stage in
// the MMAs' own pipe, the call below took 78.7 us.) What bounds it: 11008 x 4096 times 2048 tokens
// is 65.3 us, 2840 TFLOP/s: 15 us of preparation, then 946 tiles in 7 rounds over the SMs, where
// 6.2 would do, a stage every 0.4 us: the chain of a stage's waits, from the copy to the scales, the
// MMAs and back, over five stages. Timing copies with one piece left out (67.1 us whole then): 58 us
// without the fp32 results (90 MB, and the last round's with nothing beside them), 60 us with a
// quarter of the MMAs, 63 us without the wait for scales, no change with half of the X operand's
// bytes. Tiles of 128 x 192 because two accumulators of 192 columns and five
// sets of scales fit TMEM's 512 columns (256 would leave no room to overlap).
#include <algorithm>
#include <atomic>

#include "gq_few.cuh"
#include "gq_umma.cuh"

namespace gq {
namespace {

constexpr int kBM = 128;          // weight rows of a tile
constexpr int kStageK = 256;      // k of a stage: 128 bytes a row
constexpr int kStageBlocks = kStageK / 32;
constexpr int kRowBytes = kStageK / 2;
constexpr int kAtom = 512;        // scales of 128 rows x 4 blocks
constexpr int kMxThreads = 320;   // producer warp, MMA warp, four epilogue warps, four scale warps

__host__ __device__ constexpr int chunks_of(int rows) { return (rows + 127) / 128; }
// Bytes of an operand record of `rows` rows: codes, then for each four blocks the atoms.
__host__ __device__ constexpr int record_bytes(int rows) { return rows * kRowBytes + 2 * chunks_of(rows) * kAtom; }

template <int BN>
struct Mx {
    static constexpr int kA = record_bytes(kBM), kB = record_bytes(BN);
    static constexpr int kStage = kA + kB;
    static constexpr int kStages = 5;
    static constexpr int kSmem = kStages * kStage + 1024;   // stages on 1024-byte boundaries
    // TMEM columns: two accumulators, then a set of scales for each stage (8 for A, 8 or 16 for B)
    static constexpr int kScales = 2 * BN, kScaleSet = 8 + 8 * chunks_of(BN);
    static constexpr int kUsed = 2 * BN + kStages * kScaleSet, kColumns = kUsed <= 256 ? 256 : 512;
    static_assert(kUsed <= 512 && kStage % 1024 == 0 && kA % 1024 == 0, "layout");
};

// ---- Preparation ------------------------------------------------------------------------

// Where the 16 code bytes of block j (0..7) of row r lie in a record, and its scale.
__device__ __forceinline__ int code_at(int r, int j) { return r * kRowBytes + ((j ^ (r & 7)) << 4); }
__device__ __forceinline__ int scale_at(int rows, int r, int j) {
    return rows * kRowBytes + ((j >> 2) * chunks_of(rows) + (r >> 7)) * kAtom + (r & 31) * 16 +
           ((r >> 5) & 3) * 4 + (j & 3);
}

struct PrepareParams {
    const uint8_t* W;
    const float* X;
    uint8_t* wrec;       // [row tile][k tile]
    uint8_t* xrec;
    int64_t M, N;
    int kb, ktiles;      // blocks of a row; 256-k tiles
    int bn;
    int64_t w_ctas;      // CTAs that lay out weights; the others quantize X
    int64_t w_units, x_units;
};

// Weights: one thread per 17-byte block, a unit is 32 Each rows of a record. X: four lanes per
// block (lane q: elements 4q..4q+3 and 16+4q..), as in the quantizer, a unit is 8 Each rows. Rows
// and k that pad a record are zeros with scale 2^0. What bounds it is the latency of the reads:
// with Each = 4 four blocks a thread are on their way (one and four, whole products in us:
// 32000 x 2048 times 17 tokens 21.7 and 20.2, 11008 x 4096 times 2048 80.7 and 77.4, before the
// scales had warps of their own; but
// 256 x 2048 times 64, where CTAs are few, 7.4 and 8.1).
template <int Each>
__global__ void __launch_bounds__(256, 4) mx_prepare_kernel(const __grid_constant__ PrepareParams p) {
    griddep_wait();   // X, and the records that a product before may still read
    griddep_launch_dependents();
    const unsigned ktiles = static_cast<unsigned>(p.ktiles);
    if (blockIdx.x < p.w_ctas) {
        constexpr unsigned kParts = kBM / 32 / Each;   // units of a record
        const int64_t total = p.M * p.kb * kMxfp4Bytes;
        const int j = threadIdx.x & 7;
        for (int64_t u = blockIdx.x; u < p.w_units; u += p.w_ctas) {
            const unsigned record = static_cast<unsigned>(u) / kParts, tile = record / ktiles, k = record - tile * ktiles;
            const int r0 = static_cast<int>(static_cast<unsigned>(u) % kParts) * (32 * Each) + (threadIdx.x >> 3);
            const int64_t row0 = static_cast<int64_t>(tile) * kBM + r0;
            const int kb = static_cast<int>(k) * kStageBlocks + j;
            uint32_t w[Each][5], lead[Each];
#pragma unroll
            for (int e = 0; e < Each; ++e) {
                const int64_t row = row0 + 32 * e, at = (row * p.kb + kb) * kMxfp4Bytes, from = at & ~int64_t(3);
                const bool real = row < p.M && kb < p.kb;
                lead[e] = real ? static_cast<uint32_t>(at - from) : 4u;
                if (real && from + 20 <= total) {
#pragma unroll
                    for (int i = 0; i < 5; ++i) w[e][i] = *reinterpret_cast<const uint32_t*>(p.W + from + 4 * i);
                } else {   // the matrix ends inside these words
#pragma unroll
                    for (int i = 0; i < 5; ++i) {
                        w[e][i] = 0;
                        if (real)
                            for (int b = 0; b < 4; ++b)
                                if (from + 4 * i + b < total) w[e][i] |= uint32_t(p.W[from + 4 * i + b]) << (8 * b);
                    }
                }
            }
            uint8_t* rec = p.wrec + static_cast<int64_t>(record) * record_bytes(kBM);
#pragma unroll
            for (int e = 0; e < Each; ++e) {
                // byte 0 of the block `lead` bytes into the words, bytes 1..16 behind it
                uint4 codes = make_uint4(w[e][1], w[e][2], w[e][3], w[e][4]);
                uint32_t scale = w[e][0] >> 24;
                if (lead[e] < 3) {
                    const uint32_t sh = 8 * (lead[e] + 1);
                    scale = (w[e][0] >> (8 * lead[e])) & 0xFFu;
                    codes = make_uint4(__funnelshift_r(w[e][0], w[e][1], sh), __funnelshift_r(w[e][1], w[e][2], sh),
                                       __funnelshift_r(w[e][2], w[e][3], sh), __funnelshift_r(w[e][3], w[e][4], sh));
                }
                const int r = r0 + 32 * e;
                *reinterpret_cast<uint4*>(rec + code_at(r, j)) = codes;   // padding: all zeros
                rec[scale_at(kBM, r, j)] = static_cast<uint8_t>(lead[e] == 4 ? 127u : scale);
            }
        }
        return;
    }
    const int q = threadIdx.x & 3, j = (threadIdx.x >> 2) & 7;
    const bool vec = (reinterpret_cast<uintptr_t>(p.X) & 15) == 0;
    const unsigned parts = static_cast<unsigned>(p.bn) / (8 * Each);   // units of a record
    for (int64_t u = blockIdx.x - p.w_ctas; u < p.x_units; u += gridDim.x - p.w_ctas) {
        const unsigned record = static_cast<unsigned>(u) / parts, part = static_cast<unsigned>(u) - record * parts;
        const unsigned tile = record / ktiles, k = record - tile * ktiles;
        const int kb = static_cast<int>(k) * kStageBlocks + j;
        const int r0 = static_cast<int>(part) * (8 * Each) + (threadIdx.x >> 5);
        const int64_t row0 = static_cast<int64_t>(tile) * p.bn + r0;
        uint8_t* rec = p.xrec + static_cast<int64_t>(record) * record_bytes(p.bn);
        float v[Each][8];
#pragma unroll
        for (int e = 0; e < Each; ++e) {
            const float* src = p.X + ((row0 + 8 * e) * p.kb + kb) * 32 + 4 * q;   // only 4-byte aligned
#pragma unroll
            for (int i = 0; i < 8; ++i) v[e][i] = 0.0f;
            if (row0 + 8 * e < p.N && kb < p.kb) {
                if (vec) {
                    const float4 a = *reinterpret_cast<const float4*>(src);
                    const float4 b = *reinterpret_cast<const float4*>(src + 16);
                    v[e][0] = a.x; v[e][1] = a.y; v[e][2] = a.z; v[e][3] = a.w;
                    v[e][4] = b.x; v[e][5] = b.y; v[e][6] = b.z; v[e][7] = b.w;
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        v[e][i] = src[i];
                        v[e][4 + i] = src[16 + i];
                    }
                }
            }
        }
#pragma unroll
        for (int e = 0; e < Each; ++e) {
            const int r = r0 + 8 * e;
            const bool real = row0 + 8 * e < p.N && kb < p.kb;
            uint32_t amax = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(v[e][i]) & 0x7FFFFFFFu);
            amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
            amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
            const uint32_t byte = real ? mx_scale_byte(amax) : 127u;
            const uint32_t codes = real && byte != 255 ? mx_codes(v[e], mx_inverse_scale(byte)) : 0u;
            *reinterpret_cast<uint32_t*>(rec + code_at(r, j) + 4 * q) = codes;
            if (q == 0) rec[scale_at(p.bn, r, j)] = static_cast<uint8_t>(byte);
        }
    }
}

// ---- Product ----------------------------------------------------------------------------

// Instruction descriptor, kind::mxf4: A and B E2M1 (1 at bits 7 and 10), N >> 3 at [17,23),
// E8M0 scales (bit 23), M >> 4 at [24,29), K = 64 (bit 31 = 0); which of a word's four scale bytes
// belong to the instruction's two blocks: 0 or 2, for B at [4,6) and for A at [29,31).
__host__ __device__ constexpr uint32_t mx_idesc(int m, int n, int sf) {
    return (static_cast<uint32_t>(sf) << 4) | (1u << 7) | (1u << 10) |
           (static_cast<uint32_t>(n >> 3) << 17) | (1u << 23) | (static_cast<uint32_t>(m >> 4) << 24) |
           (static_cast<uint32_t>(sf) << 29);
}

__device__ __forceinline__ void umma_mxf4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                          uint32_t sfb, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// Eight TMEM columns of a warp's 32 lanes.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

__device__ __forceinline__ void lds128(uint32_t a, uint32_t* r) {
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}

struct GemmParams {
    const uint8_t* wrec;
    const uint8_t* xrec;
    float* Y;
    int64_t M, N;
    int ktiles, m_tiles, n_tiles;
    unsigned* status;
};

template <int BN>
__global__ void __launch_bounds__(kMxThreads, 1) mx_gemm_kernel(const __grid_constant__ GemmParams p) {
    using C = Mx<BN>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[C::kStages], empty[C::kStages], scaled[C::kStages], acc_full[2], acc_empty[2], drained;
    __shared__ uint32_t tmem_at;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t ring = (smem_addr(smem_raw) + 1023u) & ~1023u;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(smem_addr(&full[i]), 1);
            mbar_init(smem_addr(&empty[i]), 1);
            mbar_init(smem_addr(&scaled[i]), 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&acc_full[i]), 1);
            mbar_init(smem_addr(&acc_empty[i]), 4);
        }
        mbar_init(smem_addr(&drained), 1);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_addr(&tmem_at), C::kColumns);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_at;
    const int64_t tiles = static_cast<int64_t>(p.m_tiles) * p.n_tiles;
    griddep_wait();   // the records; and Y may still be in use before

    if (warp == 0) {
        if (lane == 0) {
            int slot = 0;
            uint32_t phase = 1;   // of `empty`: the first round passes at once
            int used = 0;
            bool ok = true;
            for (int64_t t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
                const int64_t mt = t / p.n_tiles, nt = t % p.n_tiles;
                const uint8_t* a = p.wrec + mt * p.ktiles * static_cast<int64_t>(C::kA);
                const uint8_t* b = p.xrec + nt * p.ktiles * static_cast<int64_t>(C::kB);
                for (int k = 0; k < p.ktiles; ++k) {
                    ok = mbar_wait(smem_addr(&empty[slot]), phase);
                    if (!ok) break;
                    const uint32_t bar = smem_addr(&full[slot]), dst = ring + slot * C::kStage;
                    mbar_arrive_expect_tx(bar, C::kStage);
                    bulk_g2s(dst, a + static_cast<int64_t>(k) * C::kA, C::kA, bar);
                    bulk_g2s(dst + C::kA, b + static_cast<int64_t>(k) * C::kB, C::kB, bar);
                    ++used;
                    if (++slot == C::kStages) {
                        slot = 0;
                        phase ^= 1;
                    }
                }
            }
            if (!ok) report_status(p.status, kStatusTimeout);
            // no copy may be in flight when the CTA leaves
            for (int i = 0; i < min(used, C::kStages); ++i) {
                if (--slot < 0) {
                    slot = C::kStages - 1;
                    phase ^= 1;
                }
                mbar_wait(smem_addr(&full[slot]), phase ^ 1);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            int slot = 0, n_tile = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int64_t t = blockIdx.x; ok && t < tiles; t += gridDim.x, ++n_tile) {
                const int buf = n_tile & 1;
                ok = mbar_wait(smem_addr(&acc_empty[buf]), (n_tile >> 1 & 1) ^ 1);
                if (!ok) break;
                tc_fence_after();
                const uint32_t d = tmem + buf * BN;
                for (int k = 0; k < p.ktiles; ++k) {
                    // four arrivals of warps that have waited for the stage's copies: they are
                    // here, too (a wait for `full` as well costs 1.7 us of 67)
                    ok = mbar_wait(smem_addr(&scaled[slot]), phase);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t a = ring + slot * C::kStage, b = a + C::kA;
                    const uint32_t sfa = tmem + C::kScales + slot * C::kScaleSet, sfb = sfa + 8;
                    const uint64_t ad = sw128_kmajor_desc(a), bd = sw128_kmajor_desc(b);
#pragma unroll
                    for (int i = 0; i < 4; ++i)   // 32 bytes of a row each
                        umma_mxf4(d, ad + 2 * i, bd + 2 * i, i & 1 ? mx_idesc(kBM, BN, 2) : mx_idesc(kBM, BN, 0),
                                  sfa + 4 * (i >> 1), sfb + 4 * chunks_of(BN) * (i >> 1), k > 0 || i > 0);
                    umma_commit(smem_addr(&empty[slot]));
                    if (++slot == C::kStages) {
                        slot = 0;
                        phase ^= 1;
                    }
                }
                if (ok) umma_commit(smem_addr(&acc_full[buf]));
            }
            if (!ok) report_status(p.status, kStatusTimeout);
            umma_commit(smem_addr(&drained));   // nothing may run when TMEM is given back
            mbar_wait(smem_addr(&drained), 0);
        }
    } else if (warp >= 6) {
        // scales: the same 32 rows of every atom into each quarter of the TMEM lanes
        constexpr int kB = chunks_of(BN);
        int slot = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int64_t t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
            for (int k = 0; k < p.ktiles; ++k) {
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(smem_addr(&full[slot]), phase));
                if (!ok) break;
                tc_fence_after();
                const uint32_t a = ring + slot * C::kStage + kBM * kRowBytes + lane * 16;
                const uint32_t b = ring + slot * C::kStage + C::kA + BN * kRowBytes + lane * 16;
                const uint32_t to = tmem + C::kScales + slot * C::kScaleSet + (static_cast<uint32_t>(warp & 3) << 21);
                uint32_t r[8 + 8 * kB];
#pragma unroll
                for (int i = 0; i < 2; ++i) lds128(a + i * kAtom, r + 4 * i);
#pragma unroll
                for (int i = 0; i < 2 * kB; ++i) lds128(b + i * kAtom, r + 8 + 4 * i);
#pragma unroll
                for (int i = 0; i < 1 + kB; ++i) tmem_st8(to + 8 * i, r + 8 * i);
                tmem_st_wait();
                tc_fence_before();
                uint32_t all = 0;
#pragma unroll
                for (int i = 0; i < 8 + 8 * kB; ++i) all |= r[i];
                release_warp_to_async_proxy(all);
                if (lane == 0) mbar_arrive(smem_addr(&scaled[slot]));
                if (++slot == C::kStages) {
                    slot = 0;
                    phase ^= 1;
                }
            }
        }
        if (!ok && lane == 0) report_status(p.status, kStatusTimeout);
    } else {
        const int quarter = warp & 3;   // the TMEM lanes that this warp may read
        int n_tile = 0;
        for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x, ++n_tile) {
            const int buf = n_tile & 1;
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(smem_addr(&acc_full[buf]), n_tile >> 1 & 1))) {
                report_status(p.status, kStatusTimeout);
                break;
            }
            tc_fence_after();
            const int64_t m = (t / p.n_tiles) * kBM + quarter * 32 + lane, n0 = (t % p.n_tiles) * BN;
            const int n_left = static_cast<int>(min(static_cast<int64_t>(BN), p.N - n0));
            const uint32_t src = tmem + buf * BN + (static_cast<uint32_t>(quarter * 32) << 16);
            float* out = p.Y + n0 * p.M + m;
            // 32 columns (tokens) at a time: each store is 128 consecutive bytes of a token's row
            for (int c = 0; c < BN; c += 32) {
                if (c >= n_left) break;
                uint32_t r[32];
                tmem_ld16_async(src + c, r);
                tmem_ld16_async(src + c + 16, r + 16);
                tmem_ld_wait();
                if (m < p.M) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (c + i < n_left) __stcs(out + (c + i) * p.M, __uint_as_float(r[i]));
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&acc_empty[buf]));
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, C::kColumns);
}

// ---- Host side --------------------------------------------------------------------------

// Below, the few-token kernel. It reads the weights once for 8 or 16 tokens and prepares only X;
// here all weights are laid out first. Both, in us for 8, 16 and 17 tokens (there, here):
//   M x K 2048 x 2048     5.2  7.4    6.7  7.4    6.9  7.4
//         5632 x 2048     7.4  8.6    9.4  8.6   13.3  8.6
//        32000 x 2048    19.2 19.5   24.2 19.5   40.5 19.5
//        11008 x 4096    18.8 16.6   23.4 16.6   34.1 16.6
//         2048 x 5632     9.2 13.6   12.1 13.6   12.2 13.6
// The border is a number of tokens, whatever the matrix: the few-token kernel's second group begins
// there, which doubles its time on matrices that fill the SMs. It is not each matrix's best: with 8
// to 16 tokens the larger three lose up to 40 % to this side, with 17 the two of 2048 rows up to 11 %
// to the other.
constexpr int64_t kMxMinTokens = 17;

// Token columns of a tile: the fewest rounds of tiles over the SMs, of which a round costs a share
// that does not depend on its columns (about 250 columns' worth), and the last one's results leave
// with nothing beside them. In us with 64, 128 and 192 columns (tiles over 152 SMs in brackets):
//   2048 x 2048, N = 512    8.5 (1)   9.4 (1)  10.3 (1)
//   2048 x 2048, N = 2048  20.3 (4)  15.1 (2)  16.0 (2)
//   5632 x 2048, N = 256   12.3 (2)  10.0 (1)  11.1 (1)
//   5632 x 2048, N = 512   16.0 (3)  13.9 (2)  11.5 (1)
//   11008 x 4096, N = 2048 131.5 (19) 81.6 (10) 66.2 (7)
int bn_for(int64_t M, int64_t N) {
    constexpr int64_t kSms = 152;   // a GB300's; the workspace's size is asked for without a device
    const int64_t m_tiles = (M + kBM - 1) / kBM;
    int best = 0;
    int64_t least = 0;
    for (int bn = 64; bn <= 192; bn += 64) {
        const int64_t rounds = (m_tiles * ((N + bn - 1) / bn) + kSms - 1) / kSms;
        const int64_t cost = rounds * (250 + bn) + bn;
        if (best == 0 || cost < least) {
            best = bn;
            least = cost;
        }
    }
    return best;
}

struct MxSpace {
    int64_t m_tiles, n_tiles, ktiles, w_bytes, x_bytes;
};

MxSpace mx_space(int64_t M, int64_t K, int64_t N) {
    const int bn = bn_for(M, N);
    MxSpace s{};
    s.m_tiles = (M + kBM - 1) / kBM;
    s.n_tiles = (N + bn - 1) / bn;
    s.ktiles = (K + kStageK - 1) / kStageK;
    s.w_bytes = s.m_tiles * s.ktiles * record_bytes(kBM);
    s.x_bytes = s.n_tiles * s.ktiles * record_bytes(bn);
    return s;
}

template <int BN>
cudaError_t launch_mx_gemm(const GemmParams& g, const DeviceInfo* info, cudaStream_t s) {
    auto kernel = mx_gemm_kernel<BN>;
    static std::atomic<uint64_t> ready{0};   // devices whose attribute is set
    const uint64_t bit = uint64_t(1) << info->device;
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        const cudaError_t e =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Mx<BN>::kSmem);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    const int64_t tiles = static_cast<int64_t>(g.m_tiles) * g.n_tiles;
    return launch_after(kernel, dim3(static_cast<unsigned>(std::min<int64_t>(tiles, info->sm_count))), kMxThreads,
                        Mx<BN>::kSmem, s, g);
}

}  // namespace

int64_t mx4x_workspace_bytes(int64_t M, int64_t K, int64_t N) {
    if (N < kMxMinTokens) return few_mx_workspace_bytes(K, N);
    const MxSpace s = mx_space(M, K, N);
    return s.w_bytes + s.x_bytes;   // records are multiples of 1024 bytes
}

cudaError_t launch_mx4x(const MatProblem& m, int64_t N, void* workspace, cudaStream_t s) {
    if (N < kMxMinTokens) return launch_few_mx4x(m, N, workspace, s);
    DeviceInfo* info = nullptr;
    cudaError_t e = current_device_info(&info);
    if (e != cudaSuccess) return e;
    const MxSpace at = mx_space(m.M, m.K, N);
    if (at.m_tiles * at.ktiles > 0x07FFFFFF || at.n_tiles * at.ktiles > 0x07FFFFFF) return cudaErrorInvalidValue;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    PrepareParams p{};
    p.W = m.W;
    p.X = m.X;
    p.wrec = ws;
    p.xrec = ws + at.w_bytes;
    p.M = m.M;
    p.N = N;
    p.kb = static_cast<int>(m.K / 32);
    p.ktiles = static_cast<int>(at.ktiles);
    p.bn = bn_for(m.M, N);
    // four blocks a thread where that leaves every SM its four CTAs
    const int64_t w4 = at.m_tiles * at.ktiles * (kBM / 128), x4 = at.n_tiles * at.ktiles * (p.bn / 32);
    const int64_t most = int64_t(info->sm_count) * 8;
    const int each = w4 + x4 >= info->sm_count * 4 ? 4 : 1;
    p.w_units = w4 * (4 / each);
    p.x_units = x4 * (4 / each);
    p.w_ctas = std::min(p.w_units, most);
    const unsigned grid = static_cast<unsigned>(p.w_ctas + std::min(p.x_units, most));
    e = launch_after(each == 4 ? mx_prepare_kernel<4> : mx_prepare_kernel<1>, dim3(grid), 256, 0, s, p);
    if (e != cudaSuccess) return e;
    const GemmParams g{p.wrec, p.xrec, m.Y, m.M, N, p.ktiles, static_cast<int>(at.m_tiles),
                       static_cast<int>(at.n_tiles), info->status};
    switch (p.bn) {
        case 64: return launch_mx_gemm<64>(g, info, s);
        case 128: return launch_mx_gemm<128>(g, info, s);
        default: return launch_mx_gemm<192>(g, info, s);
    }
}

}  // namespace gq
