// gq_grouped.cu -- block-quantized weights of many experts times the rows that chose them, to fp32
// accuracy on the 5th-generation tensor cores: gq_mul_mat_grouped and its SwiGLU form.
//
// Mathematics. Activations are x = 2^e (hi + lo), two fp16 terms under one scale a row (gq_few.cuh).
// A weight row's 128 k (four blocks; Q4_K: a super-block) go under a power of two of their own, 2^f, that
// brings them below 2^15, and are two fp16 terms, too: with c the code, brought into [-1, 1] by a power of two
// that its scale takes over (kLift), and d' = 2^-f d,
//     Wh = fp16(c d'), Wl = c d' - Wh (one multiply and one multiply-add in fp16),
// Q4_K, whose scale d sc has 17 bits: Wl = (c s - Wh) + c t with d' = s + t. (MXFP4 is one term.) All of it is
// exact as long as no scale is far below the largest of the 128 k: what falls below 2^-24 is lost, at most
// 2^-31 (Q8_0), 2^-32 (Q4_K) or 2^-34 of the largest scale in a weight.
// tcgen05.mma adds Wl hi + Wh lo + Wh hi over the 128 k, 128 weight rows (A, from TMEM) by up to 128 tokens
// (B, from shared memory), the small products first: the tensor cores cut a sum off below the last bit of
// its largest part, which only the last eight of the 24 instructions see at full size. Then the 128 k's
// sums, times 2^f, are added in fp32 by warps that hold the tile's results in registers. Wl lo, 2^-22 of
// the product, is left out. Q4_K's mins are two more instructions a super-block: A the mins in two terms,
// B the block sums of x in two terms.
//
// Why not the codes as they are and a scale for each 32 k (two products instead of three): every 32 k of a
// tile are then 128 x 128 sums to read out of TMEM and to hand over, and those hand-overs, some 200
// instructions on each SM sub-partition with nothing else left in, took 648 cycles where the tensor cores
// need 256 (three products: 384). With few rows an expert it is the better way, for unpacking is what
// bounds then and the sums are small: a form of the kernel of its own keeps the four blocks of a stage in
// accumulators of 32 columns each (Q4_K's mins in a fifth) and reads them out together.
//
// What bounds it: see form_of (gq_grouped.cu) and the waits at `finish`. 2048 tokens over 8 Q4_0 experts of
// 11008 x 4096, gate and up, top 2: 1490 us, 496 TFLOP/s of the result's operations, three times that on the
// tensor cores (1170 us at the rate of a library product, without the tiles' padding). 512 tokens over 64
// Q4_K experts, 2048 x 1024: 82 us, 210 TFLOP/s; 16 tokens over 64 Q8_0 experts, gate and up of 704 x 2048:
// 33 us, 3.4 TB/s of the weights of the 36 experts at work. (All in graphs of calls. No pipe is full but in the first:
// each stage's unpacking, MMAs and read-out wait for the others', two stages in flight.)
//
// Work. One persistent CTA an SM takes tiles (128 weight rows, a unit of up to 128 rows of one expert) in
// turn; stages of 128 k, two in TMEM. Warps: one copies activations (bulk copies, as many atoms of 8 rows
// as the unit has), one issues MMAs, one or two copy raw weights, eight unpack them into TMEM (two for each
// quarter of its lanes, the halves of a stage), eight add up.
#include <algorithm>
#include <type_traits>

#include "gq_grouped.cuh"

namespace gq {
namespace {

constexpr int kPrepThreads = 256;

// ---- Preparation ------------------------------------------------------------------------

struct PrepareParams {
    const float* X;
    const int32_t* rows;      // nullptr: row i of X
    const int32_t* offsets;
    int64_t N, R;
    int E, top_k, kb;
    int64_t atoms;            // of 8 rows
    uint8_t* xw;              // [64 k][atom][hi, lo][8 rows x 128 bytes, 128-byte swizzle]
    uint8_t* mins;            // Q4_K: [256 k][atom][8 rows x 128 bytes]: 8 sums hi, hi, lo, lo; unused
    float* xs;                // scale of a padded row
};

// Per threads a row (a warp with many rows, else the CTA), four lanes a block: lane t brings the eight
// elements that a weight row's t-th word of codes unpacks to, in that order. A row that no token stands
// behind (a number outside [0, N)) is zeros. The first elements stay in registers between the search for the
// largest and the split, the rest is read twice: 16376 rows of 2048 29 us (all twice 31, all kept 30), 4096 of
// 1024 8.5 us (10.7, 9.9). Twice the bytes' time; the writes, four bytes an element, are most of it.
template <int T, int Per>
__global__ void __launch_bounds__(kPrepThreads) grouped_prepare_kernel(const __grid_constant__ PrepareParams p) {
    constexpr int kKeep = Per == 32 ? 4 : 1;
    __shared__ uint32_t most[kPrepThreads / 32];
    __shared__ int groups[kPrepThreads / Per];
    const int tid = threadIdx.x % Per;
    int& group = groups[threadIdx.x / Per];
    griddep_wait();                // X, rows, offsets, and the workspace of calls before
    griddep_launch_dependents();   // the product reads offsets and weights before it waits
    const int64_t i = static_cast<int64_t>(blockIdx.x) * (kPrepThreads / Per) + threadIdx.x / Per;
    if (Per == 32 && i >= p.R) return;
    const auto sync = [] {
        if (Per == 32) __syncwarp();
        else __syncthreads();
    };
    if (tid == 0) group = -1;
    sync();
    for (int e = tid; e < p.E; e += Per)
        if (p.offsets[e] <= i && i < p.offsets[e + 1]) group = e;
    int64_t from = i;
    if (p.rows) {
        const int r = p.rows[i];
        from = r < 0 ? -1 : r / p.top_k;
    }
    const bool real = from >= 0 && from < p.N;
    const float* x = p.X + (real ? from : 0) * p.kb * 32;
    const bool vec = (reinterpret_cast<uintptr_t>(p.X) & 15) == 0;
    const int n = real ? p.kb * 4 : 0;
    const auto load = [&](int at, float (&v)[8]) {
        const float* src = x + (at >> 2) * 32 + (T == GQ_TYPE_Q8_0 ? 8 : 4) * (at & 3);
        constexpr int kSecond = T == GQ_TYPE_Q8_0 ? 4 : 16;
        if (vec) {
            const float4 a = *reinterpret_cast<const float4*>(src);
            const float4 b = *reinterpret_cast<const float4*>(src + kSecond);
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[j] = src[j];
                v[4 + j] = src[kSecond + j];
            }
        }
    };
    uint32_t amax = 0;
    const auto largest = [&](const float (&v)[8]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = max(amax, __float_as_uint(v[j]) & 0x7FFFFFFFu);
    };
    float kept[kKeep][8];   // the row's first kKeep * Per * 8 elements
#pragma unroll
    for (int c = 0; c < kKeep; ++c) {
#pragma unroll
        for (int j = 0; j < 8; ++j) kept[c][j] = 0.0f;
        if (tid + c * Per < n) load(tid + c * Per, kept[c]);
    }
#pragma unroll
    for (int c = 0; c < kKeep; ++c) largest(kept[c]);
#pragma unroll 2
    for (int at = tid + kKeep * Per; at < n; at += Per) {
        float v[8];
        load(at, v);
        largest(v);
    }
    amax = __reduce_max_sync(0xFFFFFFFFu, amax);
    if (Per != 32) {
        if ((threadIdx.x & 31) == 0) most[threadIdx.x >> 5] = amax;
        __syncthreads();
        amax = __reduce_max_sync(0xFFFFFFFFu, most[threadIdx.x & (kPrepThreads / 32 - 1)]);
    } else {
        __syncwarp();
    }
    if (group < 0) return;   // behind the last group
    const int ex = block_exponent(amax);
    const int64_t off = max(p.offsets[group], 0), row = padded_start(off, group) + (i - off);
    if (tid == 0) p.xs[row] = pow2f(ex - 14);
    const int r = static_cast<int>(row & 7);
    const int64_t atom = row >> 3;
    const int lanes = (p.kb * 4 + 31) & ~31;   // whole warps: the sums are shuffled
    const auto split = [&](int at, const float (&v)[8]) {
        __half hi[8], lo[8];
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const Split s(v[j], ex);
            const int slot = few_place(T, T == GQ_TYPE_Q8_0 ? j : (j < 4 ? j : 12 + j)) & 7;
            hi[slot] = s.hi;
            lo[slot] = s.lo;
            sum += s.sum();
        }
        if (at < p.kb * 4) {
            uint8_t* to = p.xw + ((static_cast<int64_t>(at >> 3) * p.atoms + atom) << 11) + r * 128 +
                          (((at & 7) ^ r) << 4);
            *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(hi);
            *reinterpret_cast<uint4*>(to + 1024) = *reinterpret_cast<const uint4*>(lo);
        }
        if (T == GQ_TYPE_Q4_K) {
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
            if (at < p.kb * 4 && (at & 3) == 0) {   // at most 2^20: times 2^-5 in two fp16 terms
                const Split s(sum, 14 + 5);
                const int b = at >> 2;
                uint8_t* to = p.mins + ((static_cast<int64_t>(b >> 3) * p.atoms + atom) << 10) + r * 128;
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    *reinterpret_cast<__half*>(to + ((c ^ r) << 4) + 2 * (b & 7)) = c < 2 ? s.hi : s.lo;
            }
        }
    };
#pragma unroll
    for (int c = 0; c < kKeep; ++c)
        if (tid + c * Per < lanes) split(tid + c * Per, kept[c]);
#pragma unroll 2
    for (int at = tid + kKeep * Per; at < lanes; at += Per) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.0f;
        if (at < n) load(at, v);
        split(at, v);
    }
}

// ---- Host side --------------------------------------------------------------------------

struct GroupedSpace {
    int64_t rows;                  // padded
    int64_t x_bytes, min_bytes;    // then the scales
};

GroupedSpace grouped_space(gq_type t, int64_t E, int64_t K, int64_t R) {
    GroupedSpace s{};
    s.rows = ((R + 15) & ~int64_t(15)) + 16 * std::min(E, R) + 16;
    s.x_bytes = (K + 63) / 64 * s.rows * 256;
    s.min_bytes = t == GQ_TYPE_Q4_K ? K / 256 * s.rows * 128 : 0;
    return s;
}

// A row's chunks of raw bytes start on the boundaries that tensor maps need.
bool aligned_rows(const GroupedProblem& m) { return m.K % (m.t == GQ_TYPE_MXFP4 ? 2 * kChunk : kChunk) == 0; }

// The form by the average rows an expert. Gate and up over 64 experts of 1024 x 2048 (down, 2048 x 1024, ends
// the same way), in us, few / some / many rows' form (MXFP4, whose weights are one exact term, has no use for
// the first; Q8_0 is within 2 us of Q4_0):
//   rows an expert    Q4_0                 Q4_K                 MXFP4
//    2                43.8  46.5  50.3     47.3  55.7  58.4     38.4  45.4
//    8                61.4  65.0  70.5     66.8  78.9  84.8     52.8  61.5
//   12                69.1  69.0  75.7     75.4  84.1  91.2     56.0  65.0
//   16                78.3  76.9  85.7     85.7  92.9 102.2     63.5  73.4
//   24                92.4  86.3  94.1    101.4 104.7 112.9     71.2  79.6
//   32               107.2  97.7 103.2    118.2 116.4 124.9     80.7  86.0
//   48               138.7 118.8 125.1    153.6 143.5 147.9     98.2 102.4
//   64               173.6 139.6 140.9    192.0 167.0 172.2    115.2 115.6
//   96               234.9 181.4 173.0    261.3 217.0 219.8    150.4 143.8
//  128               298.0 223.1 211.4    331.1 266.7 257.7    184.3 172.0
// Rows that tensor maps cannot take (1024 x 2080) are copied by warps. Q8_0's two passes over an expert's
// weights cost more then: 16 rows 112.6 115.7 120.5, 32 153.4 137.6 133.6, 64 248.2 191.3 171.7; not so Q4_0's:
// 16 rows 93.9 94.3 106.0, 32 129.6 115.8 122.8, 64 209.5 164.1 161.6 (MXFP4 16 79.6 83.8, 32 96.4 96.4).
Form form_of(const GroupedProblem& m) {
    const int few = m.t == GQ_TYPE_MXFP4 ? 0 : m.t == GQ_TYPE_Q4_K ? 24 : 12;
    const int some = m.t == GQ_TYPE_MXFP4 ? 48 : m.t == GQ_TYPE_Q4_K ? 96
                     : m.t == GQ_TYPE_Q8_0 && !aligned_rows(m) ? 24 : 64;
    return m.R <= few * m.E ? kFewRows : m.R <= some * m.E ? kSomeRows : kManyRows;
}

int tile_tokens(const GroupedProblem& m) {
    switch (form_of(m)) {
        case kFewRows: return Cfg<GQ_TYPE_Q4_0, true, kFewRows>::kBN;
        case kSomeRows: return Cfg<GQ_TYPE_Q4_0, true, kSomeRows>::kBN;
        default: return m.t == GQ_TYPE_Q4_K ? Cfg<GQ_TYPE_Q4_K, true, kManyRows>::kBN
                                            : Cfg<GQ_TYPE_Q4_0, true, kManyRows>::kBN;
    }
}

int64_t most_tiles(const GroupedProblem& m) {
    const int64_t rows = m.W2 ? kBM / 2 : kBM;
    return (m.M + rows - 1) / rows * (m.R / tile_tokens(m) + std::min(m.E, m.R));
}

}  // namespace

bool grouped_in_range(const GroupedProblem& m) {
    return most_tiles(m) < (int64_t(1) << 31) - 4096;   // the tile behind the last one of a CTA is an int, too
}

int64_t grouped_workspace_bytes(const GroupedProblem& m) {
    const GroupedSpace s = grouped_space(m.t, m.E, m.K, m.R);
    return s.x_bytes + s.min_bytes + (s.rows * 4 + 255) / 256 * 256;
}

cudaError_t launch_grouped(const GroupedProblem& m, void* workspace, cudaStream_t s) {
    DeviceInfo* info = nullptr;
    cudaError_t e = current_device_info(&info);
    if (e != cudaSuccess) return e;
    const GroupedSpace at = grouped_space(m.t, m.E, m.K, m.R);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    PrepareParams p{};
    p.X = m.X;
    p.rows = m.rows;
    p.offsets = m.offsets;
    p.N = m.N;
    p.R = m.R;
    p.E = static_cast<int>(m.E);
    p.top_k = m.top_k;
    p.kb = static_cast<int>(m.K / 32);
    p.atoms = at.rows / 8;
    p.xw = ws;
    p.mins = ws + at.x_bytes;
    p.xs = reinterpret_cast<float*>(ws + at.x_bytes + at.min_bytes);
    // A warp a row where there are many short ones, else a CTA. Whole calls with M = 128, in us, warp and CTA:
    // K = 512, 512 rows 7.9 and 8.2, 4096 rows 12.5 and 16.9; K = 2048, 4096 rows 36.5 and 35.3, 16384 rows
    // 66.6 and 75.1; K = 8192, 128 rows 59 and 45, 16384 rows 294 and 256.
    const bool many = m.K <= 2048 && m.R >= 4 * m.K;
    const int per_cta = many ? kPrepThreads / 32 : 1;
    const dim3 ctas(static_cast<unsigned>((m.R + per_cta - 1) / per_cta));
    const auto prepare = [&](auto type) {
        constexpr int T = decltype(type)::value;
        return launch_after(many ? grouped_prepare_kernel<T, 32> : grouped_prepare_kernel<T, kPrepThreads>, ctas,
                            kPrepThreads, 0, s, p);
    };
    switch (m.t) {
        case GQ_TYPE_Q4_0: e = prepare(std::integral_constant<int, GQ_TYPE_Q4_0>()); break;
        case GQ_TYPE_Q8_0: e = prepare(std::integral_constant<int, GQ_TYPE_Q8_0>()); break;
        case GQ_TYPE_Q4_K: e = prepare(std::integral_constant<int, GQ_TYPE_Q4_K>()); break;
        default: e = prepare(std::integral_constant<int, GQ_TYPE_MXFP4>());
    }
    if (e != cudaSuccess) return e;
    GroupedParams g{};
    g.W = m.W;
    g.W2 = m.W2;
    g.row_bytes = m.K / block_weights_of(m.t) * block_bytes_of(m.t);
    g.total_bytes = m.E * m.M * g.row_bytes;
    g.offsets = m.offsets;
    g.R = m.R;
    g.E = p.E;
    g.M = static_cast<int>(m.M);
    g.kb = p.kb;
    const int tile = m.W2 ? kBM / 2 : kBM;
    g.m_tiles = static_cast<int>((m.M + tile - 1) / tile);
    g.inverse = static_cast<unsigned>(std::min<uint64_t>((uint64_t(1) << 32) / g.m_tiles, 0xFFFFFFFFu));
    g.atoms = p.atoms;
    g.xw = p.xw;
    g.mins = p.mins;
    g.xs = p.xs;
    g.Y = m.Y;
    g.status = info->status;
    const int64_t tiles = most_tiles(m);
    const GroupedLaunch launch{tiles, form_of(m), aligned_rows(m), m.W2 != nullptr};
    switch (m.t) {
        case GQ_TYPE_Q4_0: return launch_grouped_q4_0(g, launch, info, s);
        case GQ_TYPE_Q8_0: return launch_grouped_q8_0(g, launch, info, s);
        case GQ_TYPE_Q4_K: return launch_grouped_q4_k(g, launch, info, s);
        default: return launch_grouped_mxfp4(g, launch, info, s);
    }
}

}  // namespace gq
