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

}  // namespace fa
