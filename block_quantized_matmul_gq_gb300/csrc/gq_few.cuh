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
