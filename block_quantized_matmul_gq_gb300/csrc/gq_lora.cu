// gq_lora.cu -- low-rank adapters of many requests beside a shared projection:
//     Y[n] = Y0[n] + s_l B_l (A_l X[n]),  l = ids[n],
// A_l (r x K) and B_l (M x r) in fp16 or bf16, X and Y fp32, to fp32 accuracy. Two launches: down to the
// r numbers of each token (in parts of K, added in order by the second), then up.
//
// A few tokens: every token has its own CTAs and reads its own adapter (of tokens that share one, all
// but the first from L2); fp32 multiply-adds. Bound by the latency of two dependent launches.
// More: 16 tokens are the rows of mma.m16n8k16, adapters its columns as they are stored. X and the r
// numbers come in terms of the adapters' type: two of fp16 (22 bits) under a power of two that a row's
// 32 k (the r numbers of a token) share, or three of bf16 (24 bits). Each 32 k have accumulators of
// their own, small terms first, which fp32 additions join: the tensor cores cut, they do not round. They align by
// nominal exponents, so fp16 entries of A and B among the subnormals are cut as if they were 2^-14: with all of A or B
// at 2^-22, numbers of two or three bits, the root mean square error is 1.7e-6 of the results', at 2^-18 and above
// 2e-7 as ever. Entries times 2^10, and sums with one of 64 or more made again in fp32, hold 2e-7 at 2^-22, too, and
// cost every call 3 to 10 % (r 64, M = 11008 72.5 and 76.2 us, r 128, M = 4096 69.1 and 75.6): not taken.
// Tokens of another adapter in the tile are rows of zeros; a tile makes a pass for each adapter it
// holds, so prompts (runs of tokens with one adapter) make one. 2048 tokens of 8 adapters of rank 64 (bf16,
// K = 4096, M = 11008): down 22 us, bound by the latency of its loads at 16 warps an SM, up 55 us.
// Full forms of the three kernels (X, Y0 and Y 16-byte aligned; down K a multiple of 512, above 32 ranks r one of
// 64; up r a multiple of 64 and M of 32) have no branch between their loads or between their products.
// 64 requests of 32 adapters of rank 16 (fp16, K = M = 4096): 6.1 us, both launches, in a graph of calls (one by one
// from Python 16 to 19 us: the host).
#include <algorithm>

#include "gq_few.cuh"

namespace gq {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 16;        // tokens of a tile
constexpr int kRanks = 64;       // ranks of a pass over K
constexpr int kNarrow = 32;      // ranks that the narrower kernel takes
constexpr int kMaxParts = 16;

struct LoraParams {
    const uint16_t *A, *B;
    const float* scales;
    const float* X;
    const int32_t* ids;
    const float* Y0;
    float* Y;
    float* part;      // [part][N][r]
    int64_t K, M, N, L;
    int r, parts;
};

// Eight 16-bit floats to fp32, exact.
template <bool BF16>
__device__ __forceinline__ void widen(const uint4& u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (BF16) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        } else {
            f[2 * i] = half_bits_to_float(w[i]);
            f[2 * i + 1] = half_bits_to_float(w[i] >> 16);
        }
    }
}

__device__ __forceinline__ void load8(const float* x, bool vec, float (&v)[8]) {
    if (vec) {
        const float4 a = *reinterpret_cast<const float4*>(x), b = *reinterpret_cast<const float4*>(x + 4);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = x[i];
    }
}

// Two values as a word of fp16 (bf16), the first in the low half; and what a word holds.
template <bool BF16>
__device__ __forceinline__ uint32_t narrow2(float a, float b) {
    uint32_t r;
    if (BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
template <bool BF16>
__device__ __forceinline__ float low_of(uint32_t w) {
    return BF16 ? __uint_as_float(w << 16) : half_bits_to_float(w);
}
template <bool BF16>
__device__ __forceinline__ float high_of(uint32_t w) {
    return BF16 ? __uint_as_float(w & 0xFFFF0000u) : half_bits_to_float(w >> 16);
}

template <bool BF16>
constexpr int kTerms = BF16 ? 3 : 2;

// A float no farther from zero than the largest bf16: the last ones before infinity would round to it. NaN stays NaN.
__device__ __forceinline__ float inside_bf16(float v) {
    float r;
    asm("min.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(r) : "f"(v), "f"(__uint_as_float(0x7F7F0000u)));
    return r;
}

// Terms of eight values, the largest first. (What the first bf16 of a value beyond the largest one leaves is in the
// next; an infinity leaves one. Cutting instead of rounding would do, too: the three terms are exact either way, but
// they have one sign then, and the errors of the sums grow by 3 to 6 %.)
template <bool BF16>
__device__ __forceinline__ void split8(float (&v)[8], uint32_t (&t)[kTerms<BF16>][4]) {
#pragma unroll
    for (int i = 0; i < kTerms<BF16>; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            t[i][j] = BF16 && i == 0 ? narrow2<BF16>(inside_bf16(v[2 * j]), inside_bf16(v[2 * j + 1]))
                                     : narrow2<BF16>(v[2 * j], v[2 * j + 1]);
            v[2 * j] -= low_of<BF16>(t[i][j]);
            v[2 * j + 1] -= high_of<BF16>(t[i][j]);
        }
}

// The power of two that brings a maximum (its bits) to [2^14, 2^15), and back.
struct Power {
    float up, down;
    __device__ __forceinline__ explicit Power(uint32_t amax) {
        const int e = block_exponent(amax);
        up = pow2f(14 - e);
        down = pow2f(e - 14);
    }
};

template <bool BF16>
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
    if (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// c += 16 rows (this lane: eight of 32 k of rows g and g + 8) times 8 columns (the same k of column g).
template <bool BF16>
__device__ __forceinline__ void products32(float (&c)[4], const uint32_t (&x0)[kTerms<BF16>][4],
                                           const uint32_t (&x1)[kTerms<BF16>][4], const uint4& b) {
#pragma unroll
    for (int i = kTerms<BF16> - 1; i >= 0; --i) {
        mma16<BF16>(c, x0[i][0], x1[i][0], x0[i][1], x1[i][1], b.x, b.y);
        mma16<BF16>(c, x0[i][2], x1[i][2], x0[i][3], x1[i][3], b.z, b.w);
    }
}

__device__ __forceinline__ int64_t adapter_of(const LoraParams& p, int64_t n) {
    const int id = n < p.N ? p.ids[n] : -1;
    return id >= 0 && id < p.L ? id : -1;
}

// ---- A few tokens -------------------------------------------------------------------------

// CTA (n, part): a warp has every eighth rank, lanes eight k each.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) lora_down_few_kernel(const __grid_constant__ LoraParams p) {
    griddep_wait();
    griddep_launch_dependents();
    const int64_t n = blockIdx.x, l = adapter_of(p, n);
    if (l < 0) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t steps = (p.K + 255) / 256, per = (steps + p.parts - 1) / p.parts;
    const int64_t k0 = blockIdx.y * per * 256, k1 = min(p.K, k0 + per * 256);
    const bool vec = (reinterpret_cast<uintptr_t>(p.X) & 15) == 0;
    const float* x = p.X + n * p.K;
    const uint16_t* A = p.A + l * p.r * p.K;
    constexpr int kEach = 4;   // ranks whose loads are on their way together
    for (int j0 = warp; j0 < p.r; j0 += 8 * kEach) {
        float sum[kEach] = {};
        for (int64_t k = k0 + 8 * lane; k < k1; k += 256) {
            float xv[8];
            uint4 a[kEach];
#pragma unroll
            for (int i = 0; i < kEach; ++i)
                if (j0 + 8 * i < p.r) a[i] = *reinterpret_cast<const uint4*>(A + (j0 + 8 * i) * p.K + k);
            load8(x + k, vec, xv);
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                if (j0 + 8 * i >= p.r) break;
                float av[8];
                widen<BF16>(a[i], av);
#pragma unroll
                for (int q = 0; q < 8; ++q) sum[i] = fmaf(av[q], xv[q], sum[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            if (j0 + 8 * i >= p.r) break;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum[i] += __shfl_xor_sync(0xFFFFFFFFu, sum[i], o);
            if (lane == 0) p.part[(blockIdx.y * p.N + n) * p.r + j0 + 8 * i] = sum[i];
        }
    }
}

// CTA (n, 256 rows of B): a thread has a row. What does not come from the kernel before is read while
// that runs: it lets this one start only after all that the call reads is there.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) lora_up_few_kernel(const __grid_constant__ LoraParams p) {
    __shared__ float low[256];
    constexpr int kEarly = 4;   // words of a row read early
    const int64_t n = blockIdx.x, l = adapter_of(p, n);
    const int64_t m = static_cast<int64_t>(blockIdx.y) * kThreads + threadIdx.x;
    const bool live = m < p.M;
    const uint4* b = reinterpret_cast<const uint4*>(p.B + (l * p.M + m) * p.r);
    uint4 early[kEarly];
    float y = 0.0f, scale = 1.0f;
    if (live) y = p.Y0[n * p.M + m];
    if (l >= 0 && live) {
#pragma unroll
        for (int i = 0; i < kEarly; ++i)
            if (8 * i < p.r) early[i] = b[i];
        if (p.scales) scale = p.scales[l];
    }
    griddep_wait();
    griddep_launch_dependents();
    if (l < 0 && p.Y == p.Y0) return;
    if (l >= 0 && threadIdx.x < p.r) {
        float t = 0.0f;
#pragma unroll 4
        for (int i = 0; i < p.parts; ++i) t += p.part[(i * p.N + n) * p.r + threadIdx.x];
        low[threadIdx.x] = t;
    }
    __syncthreads();
    if (!live) return;
    if (l >= 0) {
        float sum = 0.0f;
        const auto add = [&](const uint4& word, int j) {
            float bv[8];
            widen<BF16>(word, bv);
#pragma unroll
            for (int q = 0; q < 8; ++q) sum = fmaf(bv[q], low[j + q], sum);
        };
#pragma unroll
        for (int i = 0; i < kEarly; ++i)
            if (8 * i < p.r) add(early[i], 8 * i);
#pragma unroll 4
        for (int j = 8 * kEarly; j < p.r; j += 8) add(b[j / 8], j);
        y = fmaf(scale, sum, y);
    }
    p.Y[n * p.M + m] = y;
}

// ---- More tokens --------------------------------------------------------------------------

// The adapters of a tile one after another; call with all lanes, the same in every warp.
struct Passes {
    int64_t id;        // of token lane % 16
    unsigned todo;
    __device__ __forceinline__ Passes(const LoraParams& p, int64_t n0) {
        id = adapter_of(p, n0 + (threadIdx.x & 15));
        todo = __ballot_sync(0xFFFFFFFFu, id >= 0) & 0xFFFFu;
    }
    // The next adapter's number and its tokens (0: none left).
    __device__ __forceinline__ unsigned next(int64_t& l) {
        if (todo == 0) return 0;
        l = __shfl_sync(0xFFFFFFFFu, id, __ffs(todo) - 1);
        const unsigned rows = __ballot_sync(0xFFFFFFFFu, id == l) & 0xFFFFu;
        todo &= ~rows;
        return rows;
    }
};

// CTA (tile, part), more than 32 ranks: its warps take chunks of 32 k in turn, 64 ranks at a time, and join
// through shared memory in order. (2048 tokens, K = 4096, r 64, with branches and Full, in us: bf16 28.0 and 22.3,
// fp16 25.6 and 19.8.)
template <bool BF16, bool Full>
__global__ void __launch_bounds__(kThreads, 2) lora_down_wide_kernel(const __grid_constant__ LoraParams p) {
    constexpr int kPitch = kRanks + 4;
    __shared__ float sums[8][kTile][kPitch];
    griddep_wait();
    griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * kTile;
    const bool vec = (reinterpret_cast<uintptr_t>(p.X) & 15) == 0;
    const int64_t step = static_cast<int64_t>(p.parts) * 8 * 32;
    Passes passes(p, n0);
    int64_t l = 0;
    while (const unsigned rows = passes.next(l)) {
        // a row of another adapter, whose results are not stored: the first one's again
        const int first = __ffs(rows) - 1;
        const float* x0 = p.X + (n0 + (rows >> g & 1 ? g : first)) * p.K + 8 * t;
        const float* x1 = p.X + (n0 + (rows >> (g + 8) & 1 ? g + 8 : first)) * p.K + 8 * t;
        for (int j0 = 0; j0 < p.r; j0 += kRanks) {
            const uint16_t* A = p.A + (l * p.r + j0 + g) * p.K + 8 * t;
            float sum[kRanks / 8][4] = {};
            for (int64_t k = (static_cast<int64_t>(blockIdx.y) * 8 + warp) * 32; k < p.K; k += step) {
                float v0[8], v1[8];
                uint4 a[kRanks / 8];
                load8(x0 + k, Full || vec, v0);
                load8(x1 + k, Full || vec, v1);
#pragma unroll
                for (int j = 0; j < kRanks / 8; ++j)
                    if (Full || j0 + 8 * j < p.r) a[j] = *reinterpret_cast<const uint4*>(A + 8 * j * p.K + k);
                float f0 = 1.0f, f1 = 1.0f;   // scales of the two rows' 32 k
                if (!BF16) {
                    uint32_t m0 = 0, m1 = 0;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        m0 = max(m0, __float_as_uint(v0[i]) & 0x7FFFFFFFu);
                        m1 = max(m1, __float_as_uint(v1[i]) & 0x7FFFFFFFu);
                    }
#pragma unroll
                    for (int o = 1; o < 4; o <<= 1) {
                        m0 = max(m0, __shfl_xor_sync(0xFFFFFFFFu, m0, o));
                        m1 = max(m1, __shfl_xor_sync(0xFFFFFFFFu, m1, o));
                    }
                    const Power p0(m0), p1(m1);
                    f0 = p0.down;
                    f1 = p1.down;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        v0[i] *= p0.up;
                        v1[i] *= p1.up;
                    }
                }
                uint32_t t0[kTerms<BF16>][4], t1[kTerms<BF16>][4];
                split8<BF16>(v0, t0);
                split8<BF16>(v1, t1);
#pragma unroll
                for (int j = 0; j < kRanks / 8; ++j) {
                    if (!Full && j0 + 8 * j >= p.r) break;
                    float c[4] = {};
                    products32<BF16>(c, t0, t1, a[j]);
                    sum[j][0] = fmaf(c[0], f0, sum[j][0]);
                    sum[j][1] = fmaf(c[1], f0, sum[j][1]);
                    sum[j][2] = fmaf(c[2], f1, sum[j][2]);
                    sum[j][3] = fmaf(c[3], f1, sum[j][3]);
                }
            }
#pragma unroll
            for (int j = 0; j < kRanks / 8; ++j) {
                sums[warp][g][8 * j + 2 * t] = sum[j][0];
                sums[warp][g][8 * j + 2 * t + 1] = sum[j][1];
                sums[warp][g + 8][8 * j + 2 * t] = sum[j][2];
                sums[warp][g + 8][8 * j + 2 * t + 1] = sum[j][3];
            }
            __syncthreads();
            for (int i = threadIdx.x; i < kTile * kRanks; i += kThreads) {
                const int row = i / kRanks, j = i % kRanks;
                if ((rows >> row & 1) && j0 + j < p.r) {
                    float s = 0.0f;
#pragma unroll
                    for (int w = 0; w < 8; ++w) s += sums[w][row][j];
                    p.part[(blockIdx.y * p.N + n0 + row) * p.r + j0 + j] = s;
                }
            }
            __syncthreads();
        }
    }
}

// CTA (tile, part), up to 32 ranks: 512 k at a time, the tile's X goes to shared memory in terms, every
// thread's 32 elements read together; then each warp has 8 ranks and a share of the k (32 / ranks x 2 of
// them, Split), which join through shared memory in order. (2048 tokens, K = M = 4096, both launches, the
// kernel above and this one, in us: r = 8 41.5 and 37.4, 16 44.5 and 39.4, 64 55.4 and 58.9; 512 tokens,
// r = 16 23.6 and 17.5, 32 25.0 and 20.2.)
// Full: r = 16 bf16 15.7 and 14.8 us, fp16 15.0 and 14.5, r = 32 19.7 and 18.1 (this launch).
constexpr int kBlock = 512;
constexpr int kScalePitch = kBlock / 32 + 1;

// Where eight elements of a row begin: odd rows' halves of 64 bytes change places, so that the rows g and
// g + 1 that eight lanes read at once lie on different banks.
__device__ __forceinline__ int in_block(int row, int k) { return row * kBlock + (k ^ ((row & 1) << 5)); }

template <bool BF16, int Split, bool Full>
__global__ void __launch_bounds__(kThreads, 2) lora_down_kernel(const __grid_constant__ LoraParams p) {
    constexpr int kT = kTerms<BF16>, kChunks = kBlock / 32 / Split;   // chunks of 32 k of a warp
    extern __shared__ __align__(16) uint16_t xs[];   // [term][16][kBlock], then fp16's scales
    float* scales = reinterpret_cast<float*>(xs + kT * kTile * kBlock);   // [16][kScalePitch]
    griddep_wait();
    griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * kTile;
    const bool vec = (reinterpret_cast<uintptr_t>(p.X) & 15) == 0;
    const int64_t blocks = (p.K + kBlock - 1) / kBlock, per = (blocks + p.parts - 1) / p.parts;
    const int64_t first = blockIdx.y * per, last = min(blocks, first + per);
    // ranks 8 tile .. 8 tile + 7, every Split-th chunk
    const int tile = warp / Split, share = warp % Split;
    const int chunk = lane >> 2;   // filling: a quarter of a chunk's row a lane, eight chunks a warp at a time
    Passes passes(p, n0);
    int64_t l = 0;
    while (const unsigned rows = passes.next(l)) {
        const bool mine = 8 * tile < p.r;
        const uint16_t* A = p.A + (l * p.r + 8 * tile + g) * p.K + 8 * t + 32 * share;
        float sum[4] = {};
        const int other = __ffs(rows) - 1;   // for a row of another adapter, whose results are not stored
        for (int64_t b = first; b < last; ++b) {
            const int64_t k0 = b * kBlock;
            const int n = static_cast<int>(min(static_cast<int64_t>(kBlock), p.K - k0)) / 32;   // chunks of the block
            // two tokens a warp, 16 chunks each in two steps
            float v[2][kBlock / 256][8];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < kBlock / 256; ++i) {
                    const int row = 2 * warp + h, c = 8 * i + chunk;
#pragma unroll
                    for (int q = 0; q < 8; ++q) v[h][i][q] = 0.0f;
                    if (Full || c < n)
                        load8(p.X + (n0 + (rows >> row & 1 ? row : other)) * p.K + k0 + 32 * c + 8 * t, Full || vec,
                              v[h][i]);
                }
            uint4 a[kChunks];
            if (mine)
#pragma unroll
                for (int c = 0; c < kChunks; ++c)
                    if (Full || c * Split + share < n)
                        a[c] = *reinterpret_cast<const uint4*>(A + k0 + 32 * Split * c);
            __syncthreads();   // the block before has been used
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < kBlock / 256; ++i) {
                    const int row = 2 * warp + h, c = 8 * i + chunk;
                    if (!BF16) {
                        uint32_t top = 0;
#pragma unroll
                        for (int q = 0; q < 8; ++q) top = max(top, __float_as_uint(v[h][i][q]) & 0x7FFFFFFFu);
                        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                        const Power power(top);
#pragma unroll
                        for (int q = 0; q < 8; ++q) v[h][i][q] *= power.up;
                        if (t == 0) scales[row * kScalePitch + c] = power.down;
                    }
                    uint32_t terms[kT][4];
                    split8<BF16>(v[h][i], terms);
#pragma unroll
                    for (int q = 0; q < kT; ++q)
                        *reinterpret_cast<uint4*>(xs + q * kTile * kBlock + in_block(row, 32 * c + 8 * t)) =
                            make_uint4(terms[q][0], terms[q][1], terms[q][2], terms[q][3]);
                }
            __syncthreads();
            if (!mine) continue;
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                const int at = c * Split + share;
                if (!Full && at >= n) break;
                uint32_t x0[kT][4], x1[kT][4];
#pragma unroll
                for (int q = 0; q < kT; ++q) {
                    const uint4 u =
                        *reinterpret_cast<const uint4*>(xs + q * kTile * kBlock + in_block(g, 32 * at + 8 * t));
                    const uint4 w =
                        *reinterpret_cast<const uint4*>(xs + q * kTile * kBlock + in_block(g + 8, 32 * at + 8 * t));
                    x0[q][0] = u.x; x0[q][1] = u.y; x0[q][2] = u.z; x0[q][3] = u.w;
                    x1[q][0] = w.x; x1[q][1] = w.y; x1[q][2] = w.z; x1[q][3] = w.w;
                }
                float part[4] = {};
                products32<BF16>(part, x0, x1, a[c]);
                const float f0 = BF16 ? 1.0f : scales[g * kScalePitch + at];
                const float f1 = BF16 ? 1.0f : scales[(g + 8) * kScalePitch + at];
                sum[0] = fmaf(part[0], f0, sum[0]);
                sum[1] = fmaf(part[1], f0, sum[1]);
                sum[2] = fmaf(part[2], f1, sum[2]);
                sum[3] = fmaf(part[3], f1, sum[3]);
            }
        }
        float4* joined = reinterpret_cast<float4*>(xs);   // the shares, in the terms' place
        __syncthreads();
        joined[threadIdx.x] = make_float4(sum[0], sum[1], sum[2], sum[3]);
        __syncthreads();
        if (share == 0)
#pragma unroll
            for (int i = 1; i < Split; ++i) {
                const float4 o = joined[threadIdx.x + 32 * i];
                sum[0] += o.x;
                sum[1] += o.y;
                sum[2] += o.z;
                sum[3] += o.w;
            }
        if (mine && share == 0) {
            float* to = p.part + (blockIdx.y * p.N + n0 + g) * p.r + 8 * tile + 2 * t;
            if (rows >> g & 1) *reinterpret_cast<float2*>(to) = make_float2(sum[0], sum[1]);
            if (rows >> (g + 8) & 1) *reinterpret_cast<float2*>(to + 8 * p.r) = make_float2(sum[2], sum[3]);
        }
    }
}

// A token's r numbers of a term: an odd number of 64 bytes apart, so that the rows g and g + 1 that eight
// lanes read at once lie on different banks.
__host__ __device__ __forceinline__ int pitch_of(int ranks) { return ranks % 64 ? ranks : ranks + 32; }

// CTA (tile, every gridDim.y-th 256 rows of B): a warp has 32 of them. The columns of the four products
// are dealt out so that a lane has two float4 of a token, and four lanes' lie side by side: whole sectors.
// 2048 tokens, rank 64 bf16, M = 11008: 55 us (with branches 59), 3.3 TB/s of Y0 and Y; what bounds it is the L1,
// 70 % busy with requests of eight lines of 64 bytes each (of Y0, Y and B).
template <bool BF16, bool One, bool Full>   // One: at most 64 ranks
__global__ void __launch_bounds__(kThreads, 2) lora_up_kernel(const __grid_constant__ LoraParams p) {
    extern __shared__ __align__(16) uint16_t low[];   // [term][16][pitch]: the r numbers of each token, then zeros
    __shared__ float back[kTile];       // their scales
    griddep_wait();
    griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * kTile;
    const int ranks = (p.r + 31) & ~31, pitch = pitch_of(ranks), plane = kTile * pitch;
    Passes passes(p, n0);
#pragma unroll
    for (int h = 0; h < 2; ++h) {   // two tokens a warp, eight numbers a lane
        const int row = 2 * warp + h;
        const bool any = __shfl_sync(0xFFFFFFFFu, passes.id, row) >= 0;
        float v[8] = {};
        uint32_t top = 0;
        if (any && 8 * lane < p.r)
            for (int q = 0; q < p.parts; ++q) {
                float w[8];
                load8(p.part + (q * p.N + n0 + row) * p.r + 8 * lane, true, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] += w[i];
            }
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
        const Power power(__reduce_max_sync(0xFFFFFFFFu, top));
        if (!BF16)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= power.up;
        if (lane == 0) back[row] = BF16 ? 1.0f : power.down;
        uint32_t terms[kTerms<BF16>][4];
        split8<BF16>(v, terms);
        if (8 * lane < ranks)
#pragma unroll
            for (int i = 0; i < kTerms<BF16>; ++i)
                *reinterpret_cast<uint4*>(low + i * plane + row * pitch + 8 * lane) =
                    make_uint4(terms[i][0], terms[i][1], terms[i][2], terms[i][3]);
    }
    __syncthreads();
    const float f0 = back[g], f1 = back[g + 8];
    const bool vec = p.M % 4 == 0 && ((reinterpret_cast<uintptr_t>(p.Y0) | reinterpret_cast<uintptr_t>(p.Y)) & 15) == 0;
    for (int64_t m0 = static_cast<int64_t>(blockIdx.y) * 256 + warp * 32; m0 < p.M;
         m0 += static_cast<int64_t>(gridDim.y) * 256) {
        const bool whole = Full || (vec && m0 + 32 <= p.M);
        const int64_t m = m0 + 4 * t;   // this lane's columns: from m and from m + 16
        float y[2][8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t n = n0 + g + 8 * h;
            const float* from = p.Y0 + n * p.M + m;
#pragma unroll
            for (int i = 0; i < 8; ++i) y[h][i] = 0.0f;
            if (n >= p.N) continue;
            if (whole) {
                const float4 a = *reinterpret_cast<const float4*>(from), b = *reinterpret_cast<const float4*>(from + 16);
                y[h][0] = a.x; y[h][1] = a.y; y[h][2] = a.z; y[h][3] = a.w;
                y[h][4] = b.x; y[h][5] = b.y; y[h][6] = b.z; y[h][7] = b.w;
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int at = i < 4 ? i : 12 + i;
                    if (m + at < p.M) y[h][i] = from[at];
                }
            }
        }
        Passes left = passes;
        int64_t l = 0;
        while (const unsigned rows = left.next(l)) {
            const float s = p.scales ? p.scales[l] : 1.0f;
            float sum[4][4] = {};
            const uint16_t* column = p.B + (l * p.M + m0 + 4 * (g >> 1) + (g & 1)) * p.r + 8 * t;
            const auto below = [](int q) { return 16 * (q >> 1) + 2 * (q & 1); };   // product q's rows of B
            const auto ranks32 = [&](int j0, float(&c)[4][4]) {   // from j0 on
                const int j = j0 + 8 * t;
                uint32_t t0[kTerms<BF16>][4], t1[kTerms<BF16>][4];
                uint4 b[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (!Full) b[q] = uint4{};   // past the ranks and the last row
                    if (Full || (j < p.r && m0 + 4 * (g >> 1) + below(q) + (g & 1) < p.M))
                        b[q] = *reinterpret_cast<const uint4*>(column + below(q) * p.r + j0);
                }
#pragma unroll
                for (int i = 0; i < kTerms<BF16>; ++i) {
                    const uint4 u = *reinterpret_cast<const uint4*>(low + i * plane + g * pitch + j);
                    const uint4 w = *reinterpret_cast<const uint4*>(low + i * plane + (g + 8) * pitch + j);
                    t0[i][0] = u.x; t0[i][1] = u.y; t0[i][2] = u.z; t0[i][3] = u.w;
                    t1[i][0] = w.x; t1[i][1] = w.y; t1[i][2] = w.z; t1[i][3] = w.w;
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) products32<BF16>(c[q], t0, t1, b[q]);
            };
            for (int j0 = 0; j0 < (One ? 1 : p.r); j0 += 64) {   // 64 ranks have accumulators of their own
                float more[4][4] = {};
                float(&c)[4][4] = One ? sum : more;
                ranks32(j0, c);
                if (Full || j0 + 32 < p.r) ranks32(j0 + 32, c);
                if (!One)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
#pragma unroll
                        for (int i = 0; i < 4; ++i) sum[q][i] += c[q][i];
            }
            const float s0 = rows >> g & 1 ? s * f0 : 0.0f, s1 = rows >> (g + 8) & 1 ? s * f1 : 0.0f;
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int i = 0; i < 2; ++i) {   // a token of another adapter: + 0 times what may not be finite
                    if (rows >> g & 1) y[0][2 * q + i] = fmaf(s0, sum[q][i], y[0][2 * q + i]);
                    if (rows >> (g + 8) & 1) y[1][2 * q + i] = fmaf(s1, sum[q][2 + i], y[1][2 * q + i]);
                }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t n = n0 + g + 8 * h;
            float* to = p.Y + n * p.M + m;
            if (n >= p.N) continue;
            if (whole) {
                *reinterpret_cast<float4*>(to) = make_float4(y[h][0], y[h][1], y[h][2], y[h][3]);
                *reinterpret_cast<float4*>(to + 16) = make_float4(y[h][4], y[h][5], y[h][6], y[h][7]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int at = i < 4 ? i : 12 + i;
                    if (m + at < p.M) to[at] = y[h][i];
                }
            }
        }
    }
}

// ---- Host side ----------------------------------------------------------------------------

// Tokens by themselves cost what reading an adapter for each from L2 does, tiles some 7 to 10 us of latencies
// and a pass for each adapter in a tile. In us (r 16, K = M = 4096 unless said otherwise), few and many:
// 128 tokens, runs of one adapter each, 8.0 and 11.1, 256 13.3 and 11.3, 512 24.5 and 16.5; 512 with 64
// adapters in no order 26.3 and 66.4; r 64, M = 11008: 32 tokens 17.6 and 18.1, 64 28.2 and 16.6; r 8,
// K = M = 512: 1024 tokens 7.3 and 7.6. The border goes by sizes: what order the tokens are in is on the device.
bool few_tokens(int64_t r, int64_t K, int64_t M, int64_t N) { return N * r * (K + M) <= 50000000; }

// Parts of K: enough CTAs for 152 SMs, whole steps of 256 k (512 where a kernel takes those) each. (Tiles, the
// down kernel of 2048 tokens, K = 4096, with CTAs for 3, 4 and 6 times the SMs, in us: r 64 bf16 24.7 24.7 22.3,
// r 16 fp16 15.7 15.7 14.5, r 128 bf16 42.6 42.8 39.3.)
int64_t ctas_for(bool few) { return (few ? 4 : 6) * 152; }
int parts_of(int64_t r, int64_t K, int64_t M, int64_t N) {
    const bool few = few_tokens(r, K, M, N);
    const int64_t ctas = few ? N : (N + kTile - 1) / kTile;
    const int64_t want = (ctas_for(few) + ctas - 1) / ctas;
    const int64_t unit = few || r > kNarrow ? 256 : kBlock, steps = (K + unit - 1) / unit;
    const int64_t parts = std::max<int64_t>(1, std::min<int64_t>({want, steps, kMaxParts}));
    const int64_t per = (steps + parts - 1) / parts;
    return static_cast<int>((steps + per - 1) / per);   // none empty
}

template <bool BF16>
cudaError_t launch(const LoraParams& p, cudaStream_t s) {
    const unsigned parts = static_cast<unsigned>(p.parts), blocks = static_cast<unsigned>((p.M + 255) / 256);
    if (few_tokens(p.r, p.K, p.M, p.N)) {
        const unsigned n = static_cast<unsigned>(p.N);   // at most 50000000 / (8 * 33)
        const cudaError_t e = launch_after(lora_down_few_kernel<BF16>, dim3(n, parts), kThreads, 0, s, p);
        if (e != cudaSuccess) return e;
        return launch_after(lora_up_few_kernel<BF16>, dim3(n, blocks), kThreads, 0, s, p);
    }
    const unsigned tiles = static_cast<unsigned>((p.N + kTile - 1) / kTile);
    constexpr int smem = kTerms<BF16> * kTile * kBlock * 2 + (BF16 ? 0 : kTile * kScalePitch * 4);
    static_assert(smem <= 48 * 1024, "more would have to be asked for");
    const auto address = [](const void* x) { return reinterpret_cast<uintptr_t>(x); };
    const bool vec = (address(p.X) & 15) == 0, full = vec && p.K % kBlock == 0, wide_full = vec && p.r % kRanks == 0;
    const auto pick = [](bool yes, auto a, auto b) { return yes ? a : b; };
    const auto narrow = p.r <= 8    ? pick(full, lora_down_kernel<BF16, 8, true>, lora_down_kernel<BF16, 8, false>)
                        : p.r <= 16 ? pick(full, lora_down_kernel<BF16, 4, true>, lora_down_kernel<BF16, 4, false>)
                                    : pick(full, lora_down_kernel<BF16, 2, true>, lora_down_kernel<BF16, 2, false>);
    const auto wide = pick(wide_full, lora_down_wide_kernel<BF16, true>, lora_down_wide_kernel<BF16, false>);
    const dim3 grid(tiles, parts);
    const cudaError_t e = p.r <= kNarrow ? launch_after(narrow, grid, kThreads, smem, s, p)
                                         : launch_after(wide, grid, kThreads, 0, s, p);
    if (e != cudaSuccess) return e;
    // About four CTAs for each of 152 SMs: each prepares the r numbers of its tokens once. (2, 4, 6 and 8, the up
    // kernel in us: 2048 tokens, M = 4096, r 16 fp16 23.8 20.9 23.6 24.0; 1024, r 64 bf16 19.4 20.5 24.0 25.5;
    // 2048, M = 11008, r 64 bf16 70.7 55.7 56.1 55.2.)
    const unsigned along = std::min(blocks, std::max(1u, (4u * 152u + tiles - 1) / tiles));
    const bool up_full = p.r % 64 == 0 && p.M % 32 == 0 && ((address(p.Y0) | address(p.Y)) & 15) == 0;
    const auto up = p.r <= 64 ? pick(up_full, lora_up_kernel<BF16, true, true>, lora_up_kernel<BF16, true, false>)
                              : pick(up_full, lora_up_kernel<BF16, false, true>, lora_up_kernel<BF16, false, false>);
    return launch_after(up, dim3(tiles, along), kThreads, kTerms<BF16> * kTile * pitch_of((p.r + 31) & ~31) * 2, s, p);
}

}  // namespace

// Enough for N tokens and for any fewer, which may be in more parts: a token counts once in each of its parts, and
// parts * n <= (ctas_for / ctas + 1) n <= tokens of a CTA * ctas_for + n. Fewer than few tokens are few.
int64_t lora_workspace_bytes(int64_t r, int64_t K, int64_t M, int64_t N) {
    const bool few = few_tokens(r, K, M, N);
    const int64_t parts = std::min<int64_t>(kMaxParts, (K + 255) / 256);
    const int64_t rows = std::min(parts * N, (few ? 1 : kTile) * ctas_for(few) + N);
    return (rows * r * 4 + 255) / 256 * 256;
}

cudaError_t launch_lora(const LoraProblem& m, void* workspace, cudaStream_t s) {
    const LoraParams p{static_cast<const uint16_t*>(m.A), static_cast<const uint16_t*>(m.B), m.scales, m.X, m.ids, m.Y0,
                       m.Y, static_cast<float*>(workspace), m.K, m.M, m.N, m.L, static_cast<int>(m.r),
                       parts_of(m.r, m.K, m.M, m.N)};
    return m.bf16 ? launch<true>(p, s) : launch<false>(p, s);
}

}  // namespace gq
