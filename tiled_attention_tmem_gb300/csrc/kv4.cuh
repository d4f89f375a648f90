// 4-bit cache format on the device: e2m1 codes with an e4m3 scale per 16 channels.
//
// A code times a scale has at most six significant bits and is a multiple of
// 2^-10 of magnitude 2880 at most, so f16 holds every product exactly.  The
// kernels keep scales as f16 of 2^-8 times their value, which is the e4m3 byte
// moved into place (both formats have the exponent next to the sign; e4m3's
// subnormals land on f16's), and fold 2^8 into the gain.  Products are then
// multiples of 2^-18, still exact.  The sign bit is cut off, so no byte can give
// an infinity or NaN.
#pragma once
#include <cstdint>
#include <cuda_fp16.h>

#include "common.cuh"

namespace fa {

constexpr int kKKv4 = 7;  // kernel id in the device error word (after those of common.cuh)
constexpr int kKv4Group = 16;
constexpr float kKv4ScaleBias = 256.f;  // 2^8: value = f16 scale * code * 2^8 * gain

// Four bytes (eight codes) to four f16 pairs; the low half of each byte comes first.
__device__ __forceinline__ void kv4_codes(uint32_t w, uint32_t* r) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}

// Scale bytes lo and hi (0..255 each) as an f16 pair, times 2^-8.
__device__ __forceinline__ uint32_t kv4_scale_pair(uint32_t lo, uint32_t hi) {
  return ((lo | (hi << 16)) & 0x007f007fu) << 7;
}
__device__ __forceinline__ uint32_t kv4_scale_both(uint32_t s) { return (s & 0x7fu) * 0x00800080u; }

__device__ __forceinline__ uint32_t h2mul(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// A quotient is taken by a reciprocal and then cut to 12 bits after a push of 2^-13:
// where x has bf16's eight bits and the gain is a power of two, a quotient on the border
// of two results lands on it exactly, and any other is at least 2^-8 of itself away, so
// both scale and code are those of the exact quotient.
constexpr float kKv4Push = 1.f + 1.f / 8192.f;
__device__ __forceinline__ float cut12(float x) { return __uint_as_float(__float_as_uint(x) & 0xfffff000u); }

// Eight bf16 channels (four words), half of a scale's group whose other half is this warp's lane ^ 1:
// returns their codes, and the scale's byte.  All lanes call it together.  (The gain by reference: by value the store of 16384 tokens
// of 8 heads of 128, with their load, took 32.8 us instead of 32.0, in 64 registers instead of 60.)
__device__ __forceinline__ uint32_t kv4_quantise(const uint32_t* w, const float& inv_gain, uint32_t& scale) {
  uint32_t pair = 0;  // (a NaN is passed over)
#pragma unroll
  for (int k = 0; k < 4; ++k) asm("max.bf16x2 %0, %0, %1;" : "+r"(pair) : "r"(w[k] & 0x7fff7fffu));
  float top = fmaxf(__uint_as_float(pair << 16), __uint_as_float(pair & 0xffff0000u));
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
  uint16_t sb;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(sb) : "f"(0.f), "f"(cut12(top * inv_gain * (kKv4Push / 6.f))));
  scale = sb & 0xffu;
  // e4m3 to fp32 by way of f16 (2^-8 of the scale; exact).
  const float sf = __half2float(__ushort_as_half((unsigned short)((scale & 0x7f) << 7))) * kKv4ScaleBias;
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(sf));
  const float mul = sf > 0.f ? inv * inv_gain * kKv4Push : 0.f;
  uint32_t q[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float lo = cut12(__uint_as_float(w[k] << 16) * mul);
    const float hi = cut12(__uint_as_float(w[k] & 0xffff0000u) * mul);
    asm("{\n\t.reg .b8 x;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 x, %1, %2;\n\t"
        "cvt.u32.u8 %0, x;\n\t}"
        : "=r"(q[k])
        : "f"(hi), "f"(lo));
  }
  return q[0] | (q[1] << 8) | (q[2] << 16) | (q[3] << 24);
}

}  // namespace fa
