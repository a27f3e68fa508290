// Decode of 8-bit activation checkpoints, shared by the restore kernel and the
// adapter gradients that read them (the format: act8.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device.hpp"

namespace qnf4 {

constexpr int kActInt8 = 0, kActE4m3 = 1, kActBf16 = 2;   // kActBf16: not a checkpoint, the bf16 values

__host__ __device__ constexpr float act8_top(int fmt) { return fmt == kActInt8 ? 127.0f : 448.0f; }

// s = fp32(top / 127) or fp32(top / 448): the product with the rounded
// reciprocal and one residual step, which is the correctly rounded quotient for
// every constant the packer writes (0 or at least 2^-80; all of them checked)
template <int FMT>
__device__ __forceinline__ float act8_scale(uint32_t top_bits) {
  constexpr float kTop = act8_top(FMT), kInv = 1.0f / act8_top(FMT);
  const float top = bf16_lo(top_bits), q = top * kInv;
  return __builtin_fmaf(__builtin_fmaf(-q, kTop, top), kInv, q);
}

// 8 codes (8 bytes) -> 8 bf16 in order: bf16_rne(fp32(code * s))
template <int FMT>
__device__ __forceinline__ u32x4 act8_decode8(const u32x2& c, float s) {
  float f[8];
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if constexpr (FMT == kActInt8) {
#pragma unroll
      for (int e = 0; e < 4; ++e) f[4 * h + e] = static_cast<float>(static_cast<int8_t>(w[h] >> (8 * e)));
    } else {
      typedef float f32x2 __attribute__((ext_vector_type(2)));
      const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w[h]), false);
      const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w[h]), true);
      f[4 * h] = lo.x, f[4 * h + 1] = lo.y, f[4 * h + 2] = hi.x, f[4 * h + 3] = hi.y;
    }
  }
  u32x4 r;
  r.x = pack_bf16x2(f[0] * s, f[1] * s);
  r.y = pack_bf16x2(f[2] * s, f[3] * s);
  r.z = pack_bf16x2(f[4] * s, f[5] * s);
  r.w = pack_bf16x2(f[6] * s, f[7] * s);
  return r;
}

}  // namespace qnf4
