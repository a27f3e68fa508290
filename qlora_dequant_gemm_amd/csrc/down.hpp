// The rank-r product of 16 or 64 rows with one adapter by a workgroup of four
// waves, and the partial sums that workgroups leave for one another; shared by
// the kernels of multi.hip and mstream.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "act8.hpp"
#include "mm_common.hpp"
#include "multi.hpp"

namespace qnf4 {

constexpr int kMdWaves = 4;

// what a rounding leaves of v; nothing once it is infinite (inf - inf would
// turn an infinity into a NaN)
__device__ __forceinline__ float rest_of(float v, float rounded) {
  const float d = v - rounded;
  return __builtin_fabsf(d) < __builtin_inff() ? d : 0.f;
}
__device__ __forceinline__ f32x4 rest_of(const f32x4& v, const f32x4& rounded) {
  return f32x4{rest_of(v[0], rounded[0]), rest_of(v[1], rounded[1]), rest_of(v[2], rounded[2]), rest_of(v[3], rounded[3])};
}

// A wave takes at most four rank tiles of 16 (its registers), so the four waves
// are (4 / groups) shares of the contraction x groups of rank tiles.
template <int RT>
constexpr int md_rtw() { return RT < 4 ? RT : 4; }
template <int RT>
constexpr int md_groups() { return RT / md_rtw<RT>(); }

// The transposed LDS copy of 64 adapter rows (B [Kc][r], the wave's ranks):
// 32-byte pieces (row R, rank tile jt) at (R RTW + jt) ^ swz(R), so that
// 16-byte writes and ds_read_b64_tr_b16 both touch 64 distinct banks (as in
// lora.hip).
template <int RTW>
__device__ __forceinline__ int md_swz(int R) {
  if constexpr (RTW == 1) return ((R >> 4) & 1) << 2;
  else if constexpr (RTW == 2) return (R >> 4) & 1;
  else return ((R >> 1) & 1) | (((R >> 4) & 1) << 1);
}

// 64-deep chunks of a round (all their loads go out together); two rounds are
// in registers
template <int RM, int RTW>
constexpr int md_gs() {
  if constexpr (RM == 1) return RTW == 1 ? 4 : RTW == 2 ? 2 : 1;
  else return RTW == 1 ? 2 : 1;
}
// LDS chunks (16 bytes) of a workgroup: the waves' staged adapter rows, or
// their sums of one rank tile
template <int RM, int RT, bool kBT>
constexpr int md_lds() {
  constexpr int stage = kBT ? md_gs<RM, md_rtw<RT>()>() * 128 * md_rtw<RT>() : 0;
  return kMdWaves * (stage > 64 * RM ? stage : 64 * RM);
}

// This wave's share of the product of 16 RM rows of `in` with the adapter W
// (kBT: B [Kc][r], else A [r][Kc]) over its share of the 64-deep chunks [qb,
// qe). Lane (g, c) supplies 16 elements at 16 g of each chunk of row rows[i] of
// tile i. XF: the format of `in` (kActBf16, or a checkpoint with
// one constant per 64 values in `tops`). An absent row (< 0) repeats row 0 and a
// rank past r repeats the first piece: they end in sums that nobody takes.
// Columns past Kc (Kc % 64 != 0) are cleared on both sides. kVec: the rows of B
// are whole 16-byte pieces (r % 8 == 0); without it they are read value by value.
template <int RM, int RTALL, bool kBT, int XF, bool kVec>
__device__ __forceinline__ void down_acc(const void* in, const uint16_t* tops, const int64_t (&rows)[RM], int Kc, int qb,
                                         int qe, int rot, const uint16_t* W, int r, u32x4* mine,
                                         f32x4 (&acc)[RM][md_rtw<RTALL>()], int wave, int lane) {
  constexpr int RT = md_rtw<RTALL>(), kGroups = md_groups<RTALL>(), kShares = kMdWaves / kGroups;
  constexpr int GS = kVec ? md_gs<RM, RT>() : 1;
  const int w = wave / kGroups, j0 = 16 * RT * (wave % kGroups);   // share of the contraction, first rank
  const int g = lane >> 4, c = lane & 15;
  const u32x4 zero = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < RM; ++i)
#pragma unroll
    for (int jt = 0; jt < RT; ++jt) acc[i][jt] = f32x4{0.f, 0.f, 0.f, 0.f};
  const char* xp[RM];
  const uint16_t* tp[RM];
#pragma unroll
  for (int i = 0; i < RM; ++i) {
    const int64_t row = rows[i] < 0 ? 0 : rows[i];
    xp[i] = static_cast<const char*>(in) + row * Kc * (XF == kActBf16 ? 2 : 1) + 16 * g * (XF == kActBf16 ? 2 : 1);
    tp[i] = XF == kActBf16 ? nullptr : tops + row * (Kc / 64);
  }
  const uint16_t* wp[kBT ? 1 : RT];
  if constexpr (!kBT) {
#pragma unroll
    for (int jt = 0; jt < RT; ++jt) wp[jt] = W + static_cast<int64_t>(j0 + 16 * jt + c < r ? j0 + 16 * jt + c : 0) * Kc + 16 * g;
  }
  // the chunks in an order turned by `rot`: workgroups that run side by side
  // then read different columns of their rows (whose stride is mostly a
  // multiple of what the memory channels interleave)
  const int span = qe - qb;
  rot = span > 0 ? rot % span : 0;
  auto turned = [&](int q) { return q + rot < qe ? q + rot : q + rot - span; };
  struct Round {
    u32x4 x[GS][RM][XF == kActBf16 ? 2 : 1];
    uint32_t top[XF == kActBf16 ? 1 : GS][RM];
    u32x4 wv[GS][2 * RT];
  };
  auto load_round = [&](int q0, Round& R) {
#pragma unroll
    for (int u = 0; u < GS; ++u) {
      const int qq = q0 + kShares * u;         // the chunk's number before the rotation
      // past the end every lane reads the first bytes of its operand instead (one
      // line a load): a branch around the loads would make the waits before
      // the other round's MFMAs drain them all
      const bool dead = qq >= qe;
      const int q = __builtin_amdgcn_readfirstlane(dead ? qb : turned(qq));
      // pieces past Kc read the row's first ones
      const int o0 = q * 64 + 16 * g < Kc ? q * 64 : -16 * g, o1 = q * 64 + 16 * g + 8 < Kc ? q * 64 + 8 : -16 * g;
#pragma unroll
      for (int i = 0; i < RM; ++i) {
        if constexpr (XF == kActBf16) {
          R.x[u][i][0] = ld16(dead ? in : xp[i] + 2 * o0);
          R.x[u][i][1] = ld16(dead ? in : xp[i] + 2 * o1);
        } else {
          R.x[u][i][0] = ld16(dead ? in : xp[i] + q * 64);
          R.top[u][i] = *(dead ? tops : tp[i] + q);
        }
      }
      if constexpr (kBT) {
#pragma unroll
        for (int e = 0; e < 2 * RT; ++e) {
          const int pc = lane + 64 * e, n = q * 64 + (pc >> 1) / RT, col = j0 + 16 * ((pc >> 1) % RT) + 8 * (pc & 1);
          const uint16_t* wr = W + static_cast<int64_t>(n < Kc ? n : 0) * r;
          if constexpr (kVec) R.wv[u][e] = ld16(dead ? W : wr + (col < r ? col : 0));
          else R.wv[u][e] = load_row8(wr, col, r, false);
        }
      } else {
#pragma unroll
        for (int jt = 0; jt < RT; ++jt) {
          R.wv[u][2 * jt] = ld16(dead ? W : wp[jt] + o0);
          R.wv[u][2 * jt + 1] = ld16(dead ? W : wp[jt] + o1);
        }
      }
    }
  };
  auto compute_round = [&](int q0, const Round& R) {
    if constexpr (kBT) {
#pragma unroll
      for (int u = 0; u < GS; ++u)
#pragma unroll
        for (int e = 0; e < 2 * RT; ++e) {
          const int pc = lane + 64 * e, sl = pc >> 1, Rw = sl / RT;
          mine[u * 128 * RT + 2 * (sl ^ md_swz<RT>(Rw)) + (pc & 1)] = R.wv[u][e];
        }
    }
#pragma unroll
    for (int u = 0; u < GS; ++u) {
      if (q0 + kShares * u >= qe) break;       // wave-uniform
      const int q = turned(q0 + kShares * u);
      const bool tail = q * 64 + 64 > Kc;
      const bool live0 = q * 64 + 16 * g < Kc, live1 = q * 64 + 16 * g + 8 < Kc;
      u32x4 wa[RT][2];
#pragma unroll
      for (int jt = 0; jt < RT; ++jt) {
        if constexpr (kBT) {
          s16x4 v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int Rw = 16 * g + 4 * i + (c >> 2);
            v[i] = ds_read_tr(mine + u * 128 * RT, 16 * ((Rw * RT + jt) ^ md_swz<RT>(Rw)) + 4 * (c & 3));
          }
          wa[jt][0] = __builtin_bit_cast(u32x4, __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7));
          wa[jt][1] = __builtin_bit_cast(u32x4, __builtin_shufflevector(v[2], v[3], 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
          wa[jt][0] = R.wv[u][2 * jt];
          wa[jt][1] = R.wv[u][2 * jt + 1];
        }
        if (tail) {
          wa[jt][0] = live0 ? wa[jt][0] : zero;
          wa[jt][1] = live1 ? wa[jt][1] : zero;
        }
      }
#pragma unroll
      for (int i = 0; i < RM; ++i) {
        u32x4 x0, x1;
        if constexpr (XF == kActBf16) {
          x0 = R.x[u][i][0];
          x1 = R.x[u][i][1];
          if (tail) {
            x0 = live0 ? x0 : zero;
            x1 = live1 ? x1 : zero;
          }
        } else {
          const float s = act8_scale<XF>(R.top[u][i]);
          x0 = act8_decode8<XF>(u32x2{R.x[u][i][0].x, R.x[u][i][0].y}, s);
          x1 = act8_decode8<XF>(u32x2{R.x[u][i][0].z, R.x[u][i][0].w}, s);
        }
#pragma unroll
        for (int jt = 0; jt < RT; ++jt) {
          acc[i][jt] = mfma16(as_bf16x8(x0), as_bf16x8(wa[jt][0]), acc[i][jt]);
          acc[i][jt] = mfma16(as_bf16x8(x1), as_bf16x8(wa[jt][1]), acc[i][jt]);
        }
      }
    }
  };
  constexpr int kStep = kShares * GS;
  Round R0;
  if constexpr (kVec) {                          // the next round's loads go out before this one's MFMAs
    Round R1;
    load_round(qb + w, R0);
    for (int q0 = qb + w; q0 < qe; q0 += 2 * kStep) {
      const int q1 = q0 + kStep;
      __builtin_amdgcn_sched_barrier(0);
      load_round(q1, R1);
      __builtin_amdgcn_sched_barrier(0);
      compute_round(q0, R0);
      __builtin_amdgcn_sched_barrier(0);
      load_round(q1 + kStep, R0);
      __builtin_amdgcn_sched_barrier(0);
      compute_round(q1, R1);
    }
  } else {
    for (int q0 = qb + w; q0 < qe; q0 += kStep) {
      load_round(q0, R0);
      compute_round(q0, R0);
    }
  }
}

// Sums the parts of the shares in order and hands them to put(place, row, rank,
// four values of rows row .. row + 3); `place` numbers the groups of four within
// the workgroup's 16 RM x 16 RT values, consecutive threads having consecutive
// places.
template <int RM, int RT, typename Put>
__device__ __forceinline__ void down_sum(f32x4* red, const f32x4 (&acc)[RM][md_rtw<RT>()], int t, int w, int lane,
                                         Put&& put) {
  constexpr int kGroups = md_groups<RT>(), kShares = kMdWaves / kGroups;
#pragma unroll
  for (int jt = 0; jt < md_rtw<RT>(); ++jt) {
    __syncthreads();                             // the staged rows, or the sums of the rank tile before
#pragma unroll
    for (int i = 0; i < RM; ++i) red[(w * RM + i) * 64 + lane] = acc[i][jt];
    __syncthreads();
    for (int e = t; e < RM * 64 * kGroups; e += 64 * kMdWaves) {
      const int l = e % 64, i = e / 64 % RM, grp = e / (64 * RM);
      f32x4 sum = red[(grp * RM + i) * 64 + l];
#pragma unroll
      for (int sh = 1; sh < kShares; ++sh) sum += red[((sh * kGroups + grp) * RM + i) * 64 + l];
      put(jt * (RM * 64 * kGroups) + e, 16 * i + 4 * (l >> 4), 16 * (md_rtw<RT>() * grp + jt) + (l & 15), sum);
    }
  }
}

// Partial sums that another workgroup adds up: 16-byte stores and loads with
// the device-coherence bit, so that they are seen across the XCDs' caches
// without flushing them (4-byte ones cost the kernels a third of their time).
__device__ __forceinline__ void put_part(const __amdgpu_buffer_rsrc_t& rs, int place, const f32x4& v) {
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), rs, static_cast<uint32_t>(place * 16), 0, 16);
}
__device__ __forceinline__ f32x4 get_part(const __amdgpu_buffer_rsrc_t& rs, int place) {
  return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, static_cast<uint32_t>(place * 16), 0, 16));
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t part_rsrc(float* part, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(part, 0, bytes, 0x00020000);
}

// Every wave waits for its own partial sums before the workgroup counts itself
// in. True in the workgroup that arrives last; it takes the counter back to zero.
__device__ __forceinline__ bool arrived_last(unsigned* cnt, unsigned count, int t, int* flag) {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  if (t == 0) {
    const unsigned old = __hip_atomic_fetch_add(cnt, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    *flag = old == count - 1;
    if (old == count - 1) __hip_atomic_store(cnt, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  return *flag;
}
// the partial sums [S][RM RT 64] of a row block, in order, handed on as by down_sum
template <int RM, int RT, typename Put>
__device__ __forceinline__ void sum_partials(const __amdgpu_buffer_rsrc_t& rs, int S, int t, Put&& put) {
  constexpr int kGroups = md_groups<RT>(), kCount = RM * RT * 64;
  for (int p = t; p < kCount; p += 64 * kMdWaves) {
    f32x4 v[kMdMaxSplit];
#pragma unroll
    for (int s = 0; s < kMdMaxSplit; ++s) v[s] = get_part(rs, s * kCount + p);   // past the S parts: out of range, zero
    f32x4 sum = v[0];
#pragma unroll
    for (int s = 1; s < kMdMaxSplit; ++s)
      if (s < S) sum += v[s];
    const int jt = p / (RM * 64 * kGroups), e = p % (RM * 64 * kGroups), l = e % 64;
    put(p, 16 * (e / 64 % RM) + 4 * (l >> 4), 16 * (md_rtw<RT>() * (e / (64 * RM)) + jt) + (l & 15), sum);
  }
}

}  // namespace qnf4
