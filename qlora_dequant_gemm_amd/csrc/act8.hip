// 8-bit activation checkpoints for gfx950: a layer input x [M, K] (bf16) kept
// between the forward and the backward pass as one byte a value and one bf16
// constant per block of 64 (8.25 bits a value instead of 16), and restored.
//
//   top  = max |x| over the block                     (a bf16 value, kept exactly)
//   code = rne(127 x / top)          (INT8)   or   e4m3_rne(448 x / top)   (E4M3)
//   x^   = bf16_rne(fp32(code * s)),  s = fp32(top / 127)  or  fp32(top / 448)
//
// The quotient is meant in exact arithmetic. With 8-bit significands
// 127 x and 448 x are exact in fp32, a quotient that is not a tie is at least
// 2^-14 (relative) away from one, and one residual step makes a tie exact, so
// the fp32 code below decides every code as exact arithmetic would.
//
// Special blocks: one that holds a NaN or an infinity is kept as all-NaN (its
// constant is NaN), so that an overflow in the forward pass stays visible; one
// whose largest magnitude is below 2^-80 is kept as zeros (constant 0).
//
// Both kernels are one pass and bound by HBM: 3.03 bytes a value moved and
// about 9 VALU operations a value.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "act8.hpp"
#include "mm_common.hpp"

namespace qnf4 {

namespace {

constexpr uint32_t kTinyTop = 0x1780u;       // bf16 bits of 2^-80

// largest of 8 lanes (aligned groups): xor 1, xor 2 within a quad, then the
// mirrored half row, whose lane i pairs with 7 - i (quads are uniform by then)
__device__ __forceinline__ uint32_t max8(uint32_t v) {
  uint32_t o = __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xF, 0xF, true);
  v = v > o ? v : o;
  o = __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xF, 0xF, true);
  v = v > o ? v : o;
  o = __builtin_amdgcn_update_dpp(0, v, 0x141, 0xF, 0xF, true);
  return v > o ? v : o;
}

// the 8 codes of 8 consecutive values in a block with constant `top` (bf16 bits)
template <int FMT>
__device__ __forceinline__ u32x2 encode8(const u32x4& v, uint32_t top) {
  // 2^-9 keeps 448 x finite; no value that gets a nonzero code loses bits by it
  const float d = bf16_lo(top) * 0x1p-9f, inv = __builtin_amdgcn_rcpf(d);
  constexpr float kTop = act8_top(FMT);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float q[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float x = (e & 1) ? bf16_hi(w[e >> 1]) : bf16_lo(w[e >> 1]);
    const float n = (x * 0x1p-9f) * kTop;
    const float q0 = n * inv;
    q[e] = __builtin_fmaf(__builtin_fmaf(-q0, d, n), inv, q0);
  }
  u32x2 c;
  if constexpr (FMT == kActInt8) {
    uint32_t b[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) b[e] = static_cast<uint32_t>(static_cast<int>(__builtin_rintf(q[e])));
    // byte 0 of four integers into one word
    c.x = perm(perm(b[3], b[2], 0x0C0C0400u), perm(b[1], b[0], 0x0C0C0400u), 0x05040100u);
    c.y = perm(perm(b[7], b[6], 0x0C0C0400u), perm(b[5], b[4], 0x0C0C0400u), 0x05040100u);
  } else {
    int lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
    int hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], 0, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], hi, true);
    c.x = static_cast<uint32_t>(lo);
    c.y = static_cast<uint32_t>(hi);
  }
  return c;
}

constexpr int kPackPer = 4;        // 16-byte pieces of x per thread
constexpr int kUnpackPer = 2;      // 16-byte pieces of codes per thread

}  // namespace

// eight lanes hold a block (16 bytes of x each); a workgroup takes
// 256 kPackPer consecutive pieces, 256 at a time so that every wave reads and
// writes contiguous memory
template <int FMT>
__global__ __launch_bounds__(256) void k_act8_pack(const uint16_t* __restrict__ x, int64_t pieces,
                                                   uint8_t* __restrict__ codes, uint16_t* __restrict__ absmax) {
  const int64_t p0 = static_cast<int64_t>(blockIdx.x) * (256 * kPackPer) + threadIdx.x;
  u32x4 v[kPackPer];
#pragma unroll
  for (int u = 0; u < kPackPer; ++u) {
    const int64_t p = p0 + 256 * u;
    v[u] = p < pieces ? ld16(x + 8 * p) : u32x4{0u, 0u, 0u, 0u};
  }
#pragma unroll
  for (int u = 0; u < kPackPer; ++u) {
    const int64_t p = p0 + 256 * u;
    uint32_t m = 0;
    const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = w[i] & 0x7FFFu, hi = (w[i] >> 16) & 0x7FFFu;
      m = m > lo ? m : lo;
      m = m > hi ? m : hi;
    }
    m = max8(m);
    const bool bad = m >= 0x7F80u;             // NaN or infinity in the block
    const uint32_t top = bad ? 0x7FFFu : (m < kTinyTop ? 0u : m);
    u32x2 c = {0u, 0u};
    if (!bad && top) c = encode8<FMT>(v[u], top);
    if (p < pieces) {
      *reinterpret_cast<u32x2*>(codes + 8 * p) = c;
      if ((threadIdx.x & 7) == 0) absmax[p >> 3] = static_cast<uint16_t>(top);
    }
  }
}

// four lanes hold a block (16 codes each)
template <int FMT>
__global__ __launch_bounds__(256) void k_act8_unpack(const uint8_t* __restrict__ codes,
                                                     const uint16_t* __restrict__ absmax, int64_t pieces,
                                                     uint16_t* __restrict__ out) {
  const int64_t p0 = static_cast<int64_t>(blockIdx.x) * (256 * kUnpackPer) + threadIdx.x;
  u32x4 v[kUnpackPer];
  float s[kUnpackPer];
#pragma unroll
  for (int u = 0; u < kUnpackPer; ++u) {
    const int64_t p = p0 + 256 * u;
    const int64_t pc = p < pieces ? p : pieces - 1;
    v[u] = ld16(codes + 16 * pc);
    s[u] = act8_scale<FMT>(absmax[pc >> 2]);
  }
#pragma unroll
  for (int u = 0; u < kUnpackPer; ++u) {
    const int64_t p = p0 + 256 * u;
    if (p >= pieces) continue;
    u32x4* o = reinterpret_cast<u32x4*>(out + 16 * p);
    o[0] = act8_decode8<FMT>(u32x2{v[u].x, v[u].y}, s[u]);
    o[1] = act8_decode8<FMT>(u32x2{v[u].z, v[u].w}, s[u]);
  }
}

hipError_t launch_act8_pack(const uint16_t* x, int64_t numel, int fmt, uint8_t* codes, uint16_t* absmax,
                            hipStream_t stream) {
  const int64_t pieces = numel / 8;
  const dim3 grid(static_cast<unsigned>(cdiv(pieces, 256 * kPackPer)));
  if (fmt == kActInt8)
    hipLaunchKernelGGL(HIP_KERNEL_NAME(k_act8_pack<kActInt8>), grid, dim3(256), 0, stream, x, pieces, codes, absmax);
  else
    hipLaunchKernelGGL(HIP_KERNEL_NAME(k_act8_pack<kActE4m3>), grid, dim3(256), 0, stream, x, pieces, codes, absmax);
  return hipGetLastError();
}

hipError_t launch_act8_unpack(const uint8_t* codes, const uint16_t* absmax, int64_t numel, int fmt, uint16_t* out,
                              hipStream_t stream) {
  const int64_t pieces = numel / 16;
  const dim3 grid(static_cast<unsigned>(cdiv(pieces, 256 * kUnpackPer)));
  if (fmt == kActInt8)
    hipLaunchKernelGGL(HIP_KERNEL_NAME(k_act8_unpack<kActInt8>), grid, dim3(256), 0, stream, codes, absmax, pieces,
                       out);
  else
    hipLaunchKernelGGL(HIP_KERNEL_NAME(k_act8_unpack<kActE4m3>), grid, dim3(256), 0, stream, codes, absmax, pieces,
                       out);
  return hipGetLastError();
}

}  // namespace qnf4
