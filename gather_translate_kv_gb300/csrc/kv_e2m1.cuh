// 4-bit values with a scale for every 16 of them (KV_FORMAT_E2M1).
//
// A code is a sign, two bits of exponent and one of mantissa (0, .5, 1, 1.5,
// 2, 3, 4, 6). A scale byte is the upper half, sign apart, of an fp16: the
// scale is fp16(byte << 7), five bits of exponent and three of mantissa, at
// most 8192 (0xE0); greater bytes stand for NaN. code * scale then has six
// bits, no less than 2^-18 and no more than 49152, so it is exact in fp16 (and
// in bf16) and one multiplication of 16-bit pairs makes two values.
#pragma once

#include "kv_batch.cuh"

namespace gtkv {

constexpr uint32_t kMaxScaleByte = 0xE0;

// Bytes of the codes of a row's H heads, behind which their scales lie (the whole row: kv_layout.cpp).
__host__ __device__ constexpr int32_t code_bytes(int32_t H, int32_t D) { return H * D / 2; }

// The codes of a word as four pairs of fp16, in order.
__device__ __forceinline__ void codes8(uint32_t w, uint32_t (&y)[4]) {
  asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n cvt.rn.f16x2.e2m1x2 %0, b0;\n"
      " cvt.rn.f16x2.e2m1x2 %1, b1;\n cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}"
      : "=r"(y[0]), "=r"(y[1]), "=r"(y[2]), "=r"(y[3])
      : "r"(w));
}

__device__ __forceinline__ uint32_t mul_h2(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}

// All ones in the bytes of a word of scales that stand for NaN.
__device__ __forceinline__ uint32_t bad_scales(uint32_t w) { return __vcmpgtu4(w, kMaxScaleByte * 0x01010101u); }

// The same in fewer operations: bit 7 of each byte that is above the largest scale, and bit 15 of each half
// that holds such a scale as fp16 bits.
__device__ __forceinline__ uint32_t above_max(uint32_t w) {
  return ((w & 0x7f7f7f7fu) + (0x7f - (kMaxScaleByte & 0x7f)) * 0x01010101u) & w & 0x80808080u;
}
__device__ __forceinline__ uint32_t above_max_pair(uint32_t s) {
  return (s + (0x7fff - (kMaxScaleByte << 7)) * 0x00010001u) & 0x80008000u;
}

// A scale byte (below 256) as a pair of equal fp16.
__device__ __forceinline__ uint32_t scale_pair(uint32_t byte) {
  const uint32_t s = byte > kMaxScaleByte ? 0x7fffu : byte << 7;
  return s | s << 16;
}

__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __half2float(__ushort_as_half(static_cast<uint16_t>(byte > kMaxScaleByte ? 0x7fffu : byte << 7)));
}

// One element of a block: its code (0 to 15) times its scale.
__device__ __forceinline__ float code_value(uint32_t code, uint32_t byte) {
  const uint32_t m = code & 7;
  // codes 0 and 1 are 0 and 0.5, the others 2^(e - 1) * (1 + m / 2)
  const float v = m < 2 ? 0.5f * m : __uint_as_float(((m >> 1) + 126u) << 23 | (m & 1) << 22);
  return (code & 8 ? -v : v) * scale_value(byte);
}

// The scale byte of a block from the bits of its largest magnitude, 0xFF when that is not finite:
// a sixth of it (in 32 bits, at most 8192) in fp16, then to the upper eight bits, each to nearest even.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return 0xff;
  const float sixth = fminf(__fmul_rn(__uint_as_float(amax_bits), 1.0f / 6.0f), 8192.0f);
  const uint32_t h = __half_as_ushort(__float2half_rn(sixth));
  return (h + 63 + (h >> 7 & 1)) >> 7;
}

// What a block's values are multiplied with before they become codes.
__device__ __forceinline__ float scale_inverse(uint32_t byte) { return byte == 0 ? 0.0f : __frcp_rn(scale_value(byte)); }

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// Eight values times inv as codes, to nearest even, at most 6.
__device__ __forceinline__ uint32_t encode8(const float* x, float inv) {
  uint32_t w;
  asm("{\n .reg .b8 b0, b1, b2, b3;\n cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n mov.b32 %0, {b0, b1, b2, b3};\n}"
      : "=r"(w)
      : "f"(__fmul_rn(x[0], inv)), "f"(__fmul_rn(x[1], inv)), "f"(__fmul_rn(x[2], inv)), "f"(__fmul_rn(x[3], inv)),
        "f"(__fmul_rn(x[4], inv)), "f"(__fmul_rn(x[5], inv)), "f"(__fmul_rn(x[6], inv)), "f"(__fmul_rn(x[7], inv)));
  return w;
}

}  // namespace gtkv
