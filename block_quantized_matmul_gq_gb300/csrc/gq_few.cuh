// gq_few.cuh -- what the few-token kernels (gq_few.cu) and their callers share: the split
// activation format, its element order, and the launchers.
//
// Split activations. One 32-element block of one activation row becomes 2 x 32 fp16, hi and lo,
// with x = 2^(e - 14) (hi + lo): e = floor(log2 max |x|) over the row (of the hidden vector of an
// expert: over the block, which is all that the kernel that makes it sees). The maximum lands in
// [2^14, 2^15), so hi keeps 11 significant bits of every element and lo the next 11, down to
// 2^-39 of the maximum. With them the scale 2^(e - 14) and, where Q4_K's mins multiply them, the
// sums of the blocks (of a row with one scale: before it).
// The weights enter the tensor cores as exact fp16 integers (or E2M1 values), so a product's
// only rounding beside the fp32 sums is that of hi + lo, 2^-23 of the element.
//
// The bound (K / 32 + 160) 2^-24 on a product, in units of 2^-24 of its absolute sum: one for each
// of the K / 32 multiply-adds of the blocks' sums; 7 for the join of up to eight warps; 2 for the
// terms of X; and four chained instructions a block, each of 17 addends (16 products and the sum
// before) that may lose 2^-24 of the largest, and cut to fp32 at the end, 2^-23: 4 (17 + 2) = 76.
// That is 85. Q4_K chains eight instructions, 152, so 161, but adds six times where the others add
// eight times, which saves K / 128, at least 2. (How the instructions cut is not documented: the
// tests hold all results to the bound.) It is a worst case; the root mean square error is 2 to 8
// units.
//
// MXFP4 activations (the microscaled product) use one term: the E2M1 values themselves, and
// one float 2^e per block.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

#include "gq_device.cuh"
#include "gq_internal.h"

namespace gq {


// Place (0..31) of element i of a block in the order in which the four lanes that share a
// weight row hold it: lane t = place / 8 takes the block's bytes 4t..4t+3 (and 16 + 4t.. for
// the types with 32 code bytes), and the shifts and masks that unpack a word of codes yield
// pairs in these orders. The contraction does not depend on the order, so activations are
// stored in the weights' order and no weight is ever moved between lanes.
__host__ __device__ __forceinline__ int few_place(int type, int i) {
    if (type == GQ_TYPE_Q8_0) return i;                     // lane t: bytes 8t..8t+7
    const int t = (i & 15) >> 2, r = i & 3, hi = i >> 4;
    int slot;
    if (type == GQ_TYPE_MXFP4)
        slot = 2 * r + hi;                                  // byte r: (low, high) nibbles
    else if (type == GQ_TYPE_Q4_0)
        slot = 2 * (2 * (r & 1) + hi) + (r >> 1);           // masks 0x000F000F << 0, 4, 8, 12
    else
        slot = 2 * (2 * hi + (r & 1)) + (r >> 1);           // Q4_K: one nibble of each word
    return 8 * t + slot;
}

// Exponent e (clamped so that 2^(14 - e) and 2^(e - 14) are normal) of a block maximum given
// as the bits of a non-negative float.
__device__ __forceinline__ int block_exponent(uint32_t amax_bits) {
    const int e = static_cast<int>(amax_bits >> 23) - 127;
    return e < -110 ? -110 : (e > 127 ? 127 : e);
}

__device__ __forceinline__ float pow2f(int e) {   // e in [-126, 127]
    return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// Two values already divided by their block scale as one byte of E2M1 codes, `lo` in the low
// nibble: nearest value, ties to the even code, beyond 6 saturates, the sign kept.
__device__ __forceinline__ uint32_t e2m1_pair(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\tcvt.u32.u8 %0, b;\n\t}"
        : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// The code bytes 4q..4q+3 of a block from its elements 4q..4q+3 and 16+4q..16+4q+3.
__device__ __forceinline__ uint32_t mx_codes(const float (&v)[8], float inv) {
    uint32_t codes = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) codes |= e2m1_pair(v[i] * inv, v[4 + i] * inv) << (8 * i);
    return codes;
}

// E8M0 scale byte of a block maximum (bits of a non-negative float): floor(log2 amax) - 2 with
// bias 127, 0 for a zero (or smaller) block, 255 (NaN) for a block with an infinity or a NaN.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
    const uint32_t e = amax_bits >> 23;
    return e == 255 ? 255 : (e > 2 ? e - 2 : 0);
}

// 2^(byte - 127), NaN for 255.
__device__ __forceinline__ float mx_scale(uint32_t byte) {
    return __uint_as_float(byte == 0 ? 0x00400000u : (byte == 255 ? 0x7FC00000u : byte << 23));
}

// 2^(127 - byte) for byte <= 254.
__device__ __forceinline__ float mx_inverse_scale(uint32_t byte) {
    return byte == 254 ? __uint_as_float(0x00400000u) : __uint_as_float((254u - byte) << 23);
}

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

// The eight 4-bit codes of a word minus Z (0 or 8), times 2^-S, as fp16 pairs (bits 0 and 16), (4 and 20),
// (8 and 24), (12 and 28).
template <int Z, int S = 0>
__device__ __forceinline__ void nibbles_to_f16(uint32_t w, uint32_t (&h)[4]) {
    constexpr uint32_t kBoth = 0x00010001u;
    constexpr uint32_t kOne = kMagic - kBoth * (S << 10);                            // 1024 2^-S
    constexpr uint32_t kLow = kOne + kBoth * Z;                                      // (1024 + Z) 2^-S
    constexpr uint32_t kHigh = 0xD400D400u - kBoth * (S << 10) + kBoth * (Z << 4);   // -(64 + Z) 2^-S
    constexpr uint32_t kPart = kSixteenth - kBoth * (S << 10);                       // 2^-S / 16
    const uint32_t v = w >> 8;
    h[0] = h2_sub((w & 0x000F000Fu) | kOne, kLow);
    h[1] = h2_fma((w & 0x00F000F0u) | kMagic, kPart, kHigh);
    h[2] = h2_sub((v & 0x000F000Fu) | kOne, kLow);
    h[3] = h2_fma((v & 0x00F000F0u) | kMagic, kPart, kHigh);
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

// A launch that may start while the kernel before it on the stream still runs (it waits with
// griddep_wait).
template <typename... Sig, typename... Args>
cudaError_t launch_after(void (*kernel)(Sig...), dim3 grid, int threads, int smem, cudaStream_t s,
                         const Args&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
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

}  // namespace gq
