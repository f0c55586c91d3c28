// 8-bit activation checkpoint: the number format and its device helpers.
//
// A row of d bf16 values is cut into blocks of 32 columns.  A block holds
//   e = the least integer with max|x| <= 127 * 2^e, kept in [-126, 121],
//   q = x * 2^-e rounded to the nearest integer (ties to even), |q| <= 127,
// stored as 32 int8 values and the byte e + 127 (the exponent field of 2^e in
// fp32, so the scale is one shift away).  q has at most seven significant
// bits, so q * 2^e is exact in bf16: the only rounding is the one to q, at most
// 2^(e-1), i.e. 1/127 of the block's largest value.  An 8-bit float with a 3-bit
// mantissa would spend the same bytes for a rounding of up to 1/16 of each
// value.  A block with a NaN or an infinity gets byte 255 and q = 0: its scale
// then reads as infinity and 0 * inf makes every value of the block NaN.
#pragma once

#include "sk_internal.cuh"

namespace sk {

constexpr int kCkptBlock = 32;

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }

// Scale byte from the block's largest |x| (bf16 bits without the sign).
__device__ __forceinline__ uint32_t ckpt8_scale_byte(uint32_t amax) {
  if (amax >= 0x7f80u) return 255u;
  // amax = 1.m * 2^E; 127 * 2^e = 1.984375 * 2^(e+6), and the next bf16 mantissa is 1.9921875
  int byte = (int)(amax >> 7) - 6 + ((amax & 0x7fu) == 0x7fu ? 1 : 0);
  byte = byte < 1 ? 1 : byte;
  return (uint32_t)(byte > 248 ? 248 : byte);
}

// Quantise eight consecutive values (four bf16x2 words) of a 32-column block
// whose other values sit in the neighbouring lanes of an aligned group of four.
// Called by whole warps.
__device__ __forceinline__ uint2 ckpt8_quantize8(const uint32_t (&w)[4], uint32_t& byte) {
  uint32_t a = max_u16x2(max_u16x2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu),
                         max_u16x2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
  a = max_u16x2(a, __shfl_xor_sync(0xffffffffu, a, 1));
  a = max_u16x2(a, __shfl_xor_sync(0xffffffffu, a, 2));
  byte = ckpt8_scale_byte(max(a & 0xffffu, a >> 16));
  if (byte == 255u) return make_uint2(0u, 0u);
  const float inv = __uint_as_float((254u - byte) << 23);          // 2^-e
  uint32_t b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = __uint_as_float((i & 1) ? (w[i >> 1] & 0xffff0000u) : (w[i >> 1] << 16));
    // x * 2^-e rounded to an integer in the low bits of the sum (one rounding, ties to even)
    float r = fmaf(x, inv, 12582912.f);
    r = fminf(fmaxf(r, 12582912.f - 127.f), 12582912.f + 127.f);   // only the largest bf16 values reach it
    b[i] = __float_as_uint(r);
  }
  auto four = [](uint32_t b0, uint32_t b1, uint32_t b2, uint32_t b3) {
    return prmt(prmt(b0, b1, 0x0040), prmt(b2, b3, 0x0040), 0x5410);
  };
  return make_uint2(four(b[0], b[1], b[2], b[3]), four(b[4], b[5], b[6], b[7]));
}

// Two int8 values in the low bytes of the halves of `t` -> bf16x2 of the two,
// exactly: 128 + (the low seven bits) has an ulp of one, and what comes off it is
// 128, or 256 for a negative value -- the sign bit sits where those two constants
// differ (the lowest exponent bit), so one logic operation forms each term.
__device__ __forceinline__ uint32_t int8x2_to_bf16x2(uint32_t t) {
  const uint32_t m = (t & 0x007f007fu) | 0x43004300u;
  const uint32_t c = (t & 0x00800080u) | 0xc300c300u;
  const __nv_bfloat162 v = __hadd2(*reinterpret_cast<const __nv_bfloat162*>(&m),
                                   *reinterpret_cast<const __nv_bfloat162*>(&c));
  return *reinterpret_cast<const uint32_t*>(&v);
}

// bf16x2 of a block's scale 2^e from its byte (255 gives infinity)
__device__ __forceinline__ uint32_t ckpt8_scale2(uint32_t byte) { return (byte << 7) | (byte << 23); }

// Four int8 values times 2^e as two bf16x2 words, exactly (q has at most seven
// significant bits; 0 * inf is the NaN of a block that was not finite).
__device__ __forceinline__ void ckpt8_dequant4(uint32_t q4, uint32_t scale2, uint32_t& w0, uint32_t& w1) {
  const uint32_t t = prmt(q4, 0u, 0x3120);                          // bytes 0 2 1 3
  const __nv_bfloat162 s = *reinterpret_cast<const __nv_bfloat162*>(&scale2);
  uint32_t a = int8x2_to_bf16x2(t), b = int8x2_to_bf16x2(t >> 8);
  const __nv_bfloat162 x = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a), s);
  const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&b), s);
  w0 = *reinterpret_cast<const uint32_t*>(&x);
  w1 = *reinterpret_cast<const uint32_t*>(&y);
}

// launchers
cudaError_t launch_ckpt8_quantize(const uint16_t* X, int64_t T, int64_t d, int8_t* q, uint8_t* scale, cudaStream_t s);
cudaError_t launch_ckpt8_dequantize(const int8_t* q, const uint8_t* scale, int64_t T, int64_t d, uint16_t* X,
                                    cudaStream_t s);

}  // namespace sk
