// ra_cache8.cuh -- the 8-bit key/value ring: its layout and the conversion of
// its codes to bf16.
//
// Ring of W frames of s tokens for each of B x H heads: codes e4m3
// [B, H, W * s, d], scales fp32 [B, H, W, blocks] with blocks = ceil(s / 64):
// token j of a slot belongs to block j / 64 of it, and stands for code * scale.
// The scale is a power of two, so code * scale is a bf16 number exactly (4
// significant bits): the attention multiplies bf16 operands that carry no
// rounding of their own.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

namespace ra {

constexpr int CACHE8_BLOCK = 64;  // tokens of a frame that share a scale
constexpr long long CACHE8_MAX_ROWS = 1LL << 30;  // of a head: a few rows further still fit an int

inline int cache8_blocks(int s) { return (s + CACHE8_BLOCK - 1) / CACHE8_BLOCK; }

// Two e4m3 codes, in bytes 1 and 3 of y, as bf16 numbers code * 2^-120: the sign
// and the seven bits of a code land on a bf16's sign and on the low exponent and
// high mantissa bits, which reads 2^(e - 127) where the code means 2^(e - 7) (and
// the same factor for e = 0, a subnormal on both sides).  The two codes of NaN
// read as +-480: they are not part of the ring's format.
__device__ __forceinline__ uint32_t e4m3x2_small(uint32_t y)
{
    return ((y >> 4) & 0x07F007F0u) | (y & 0x80008000u);
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b)
{
    const __nv_bfloat162 r =
        __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}

// The factors that take e4m3x2_small to code * scale: 2^120 * scale as one bf16
// for scales up to 2^7 (values up to 57344), else 2^120 and the scale (which is
// where a NaN scale, the mark of a block with a value that was not finite, goes).
struct CodeScale {
    uint32_t first;   // bf16 bits
    uint32_t second;  // bf16 bits, 1.0 when one factor is enough
};

__device__ __forceinline__ uint32_t bf16_bits(float x)
{
    return static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(x)));
}

__device__ __forceinline__ CodeScale code_scale(float scale)
{
    const float up = __uint_as_float((120u + 127u) << 23);  // 2^120
    if (scale <= 128.f)
        return CodeScale{bf16_bits(scale * up), 0x3F80u};
    return CodeScale{bf16_bits(up), bf16_bits(scale)};
}

}  // namespace ra
