// A pool of LoRA adapters beside one frozen weight, for gfx950: the rank-r
// products of a batch whose rows use different adapters, and the gradients of
// every adapter of the pool.
//
// Row m of the batch uses adapter a = index[m] of A [n, r, K], B [n, N, r],
// scale [n]; an index outside 0 .. n - 1 means no adapter. The rank-r update is
// the one of a single adapter ("QLoRA and Quantized Training", "In code"; "A
// 65B fine-tune on the GPU you already have", figure 2), row by row:
//     t_m = x_m . A_a^T,  u_m = dY_m . B_a
//     dB_a = s_a sum_m dY_m^T t_m,   dA_a = s_a sum_m u_m^T x_m   (rows m of a)
//
// k_mdown  s_a t or s_a u of a batch in its own order, for the forward and
//          backward GEMMs: 16 rows per workgroup, one pass per adapter among
//          them; beside it, x in MFMA order for the streaming forward.
// The gradients first list each adapter's rows (k_msort: the rows of an adapter in
// batch order, padded to whole 64-row chunks), so that every later product has
// one adapter per chunk and needs no masks:
// k_gdown  t and u over the listed rows, transposed, as three bf16 numbers
//          that sum to the fp32 value (hi + mid + lo: fp32 gradients want more
//          than one bf16 rounding of t and u)
// k_mgrad  G = P^T . Q over the rows of one item (a run of chunks of one
//          adapter), P = dY or x gathered by row, Q = t or u
// k_mfinish sums the items of adapters with more than one, in order; zeroes the
//          gradients of adapters without rows.
// Results do not depend on scheduling: no atomic touches a sum.
//
// What bounds the gradients: x and dY are each read twice (t and u need whole
// rows before any column of dA or dB can use them), the second time mostly from
// the last-level cache.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "act8.hpp"
#include "mm_common.hpp"
#include "multi.hpp"

namespace qnf4 {

namespace {

constexpr int kMdWaves = 8;
constexpr int kSplit = 3;                      // bf16 numbers that carry one fp32 value of t or u

// The transposed LDS copy of 64 adapter rows (B [Kc][r]): 32-byte pieces (row
// R, rank tile jt) at (R RT + jt) ^ swz(R), so that 16-byte writes and
// ds_read_b64_tr_b16 both touch 64 distinct banks (as in lora.hip).
template <int RT>
__device__ __forceinline__ int md_swz(int R) {
  if constexpr (RT == 1) return ((R >> 4) & 1) << 2;
  else if constexpr (RT == 2) return (R >> 4) & 1;
  else if constexpr (RT == 4) return ((R >> 1) & 1) | (((R >> 4) & 1) << 1);
  else return (R & 3) | (((R >> 4) & 1) << 2);
}

// LDS chunks (16 bytes) a wave needs: its staged adapter rows, then its sums
template <int RT, int GS, bool kBT>
constexpr int md_per() {
  constexpr int stage = kBT ? GS * 128 * RT : 0;
  return stage > 64 * RT ? stage : 64 * RT;
}

// 16 rows x 16 RT ranks of (rows of `in`) . W^T, this wave's share of the
// contraction: chunks w, w + 8, ... of 64. Lane (g, c) supplies 16 elements
// of its row (`row`, < 0: zeros) at 16 g of each chunk. kBT: W is B [Kc][r],
// else A [r][Kc]. XF: the format of `in` (kActBf16 or a checkpoint with one
// constant per 64 values in `tops`). Pieces past Kc, ranks past r and absent
// rows are zero on both sides, whatever the memory next to them holds.
template <int RT, int GS, bool kBT, int XF>
__device__ __forceinline__ void down_acc(const void* in, const uint16_t* tops, int64_t row, int Kc,
                                         const uint16_t* W, int r, u32x4* mine, f32x4 (&acc)[RT], int w, int lane) {
  const int g = lane >> 4, c = lane & 15;
  const int nchunk = (Kc + 63) / 64;
  const bool vec = (r & 7) == 0;
  const bool rlive = row >= 0;
  const int64_t rs = rlive ? row : 0;
  const u32x4 zero = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int jt = 0; jt < RT; ++jt) acc[jt] = f32x4{0.f, 0.f, 0.f, 0.f};
  struct Round {
    u32x4 xa[GS][XF == kActBf16 ? 2 : 1];
    uint32_t top[XF == kActBf16 ? 1 : GS];
    u32x4 wv[GS][2 * RT];
  };
  auto load_round = [&](int q0, Round& R) {
#pragma unroll
    for (int u = 0; u < GS; ++u) {
      const int qq = q0 + kMdWaves * u;
      const int q = qq < nchunk ? qq : 0;
      const int k = q * 64 + 16 * g;
      const int k0 = k < Kc ? k : 0, k1 = k + 8 < Kc ? k + 8 : 0;
      if constexpr (XF == kActBf16) {
        const uint16_t* xr = static_cast<const uint16_t*>(in) + rs * Kc;
        R.xa[u][0] = ld16(xr + k0);
        R.xa[u][1] = ld16(xr + k1);
      } else {
        R.xa[u][0] = ld16(static_cast<const uint8_t*>(in) + rs * Kc + k0);
        R.top[u] = tops[rs * (Kc / 64) + q];
      }
      if constexpr (kBT) {
#pragma unroll
        for (int e = 0; e < 2 * RT; ++e) {
          const int pc = lane + 64 * e, Rw = (pc >> 1) / RT, col = 16 * ((pc >> 1) % RT) + 8 * (pc & 1);
          const int n = q * 64 + Rw;
          const uint16_t* wr = W + static_cast<int64_t>(n < Kc ? n : 0) * r;
          if (vec) R.wv[u][e] = ld16(wr + (col < r ? col : 0));   // cleared when it is staged
          else R.wv[u][e] = load_row8(wr, col, r, false);
        }
      } else {
#pragma unroll
        for (int jt = 0; jt < RT; ++jt) {
          const uint16_t* wr = W + static_cast<int64_t>(16 * jt + c < r ? 16 * jt + c : 0) * Kc;
          R.wv[u][2 * jt] = ld16(wr + k0);
          R.wv[u][2 * jt + 1] = ld16(wr + k1);
        }
      }
    }
  };
  auto compute_round = [&](int q0, const Round& R) {
    u32x4 wa[GS][RT][2];
    if constexpr (kBT) {
#pragma unroll
      for (int u = 0; u < GS; ++u)
#pragma unroll
        for (int e = 0; e < 2 * RT; ++e) {
          const int pc = lane + 64 * e, sl = pc >> 1, Rw = sl / RT, col = 16 * (sl % RT) + 8 * (pc & 1);
          const int q = q0 + kMdWaves * u;
          const bool live = col < r && q < nchunk && q * 64 + Rw < Kc;
          mine[u * 128 * RT + 2 * (sl ^ md_swz<RT>(Rw)) + (pc & 1)] = live ? R.wv[u][e] : zero;
        }
#pragma unroll
      for (int u = 0; u < GS; ++u)
#pragma unroll
        for (int jt = 0; jt < RT; ++jt) {
          s16x4 v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int Rw = 16 * g + 4 * i + (c >> 2);
            v[i] = ds_read_tr(mine + u * 128 * RT, 16 * ((Rw * RT + jt) ^ md_swz<RT>(Rw)) + 4 * (c & 3));
          }
          wa[u][jt][0] = __builtin_bit_cast(u32x4, __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7));
          wa[u][jt][1] = __builtin_bit_cast(u32x4, __builtin_shufflevector(v[2], v[3], 0, 1, 2, 3, 4, 5, 6, 7));
        }
    } else {
#pragma unroll
      for (int u = 0; u < GS; ++u)
#pragma unroll
        for (int jt = 0; jt < RT; ++jt) {
          const bool live = 16 * jt + c < r;
          wa[u][jt][0] = live ? R.wv[u][2 * jt] : zero;
          wa[u][jt][1] = live ? R.wv[u][2 * jt + 1] : zero;
        }
    }
#pragma unroll
    for (int u = 0; u < GS; ++u) {
      const int q = q0 + kMdWaves * u;
      const int k = q * 64 + 16 * g;
      const bool live0 = q < nchunk && k < Kc, live1 = q < nchunk && k + 8 < Kc;
      u32x4 x0, x1;
      if constexpr (XF == kActBf16) {
        x0 = R.xa[u][0];
        x1 = R.xa[u][1];
      } else {
        const float s = act8_scale<XF>(R.top[u]);
        x0 = act8_decode8<XF>(u32x2{R.xa[u][0].x, R.xa[u][0].y}, s);
        x1 = act8_decode8<XF>(u32x2{R.xa[u][0].z, R.xa[u][0].w}, s);
      }
      x0 = live0 && rlive ? x0 : zero;
      x1 = live1 && rlive ? x1 : zero;
#pragma unroll
      for (int jt = 0; jt < RT; ++jt) {
        acc[jt] = mfma16(as_bf16x8(x0), as_bf16x8(live0 ? wa[u][jt][0] : zero), acc[jt]);
        acc[jt] = mfma16(as_bf16x8(x1), as_bf16x8(live1 ? wa[u][jt][1] : zero), acc[jt]);
      }
    }
  };
  constexpr int kStep = kMdWaves * GS;
  Round R0;
  if constexpr (RT * GS <= 4) {                // two rounds in registers where they fit
    Round R1;
    load_round(w, R0);
    for (int q0 = w; q0 < nchunk; q0 += 2 * kStep) {
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
    for (int q0 = w; q0 < nchunk; q0 += kStep) {
      load_round(q0, R0);
      compute_round(q0, R0);
    }
  }
}

// sum of the eight waves' parts of (row, rank j), in wave order
template <int RT, int kPer>
__device__ __forceinline__ float md_sum(const f32x4* red, int row, int j) {
  const int l = ((row >> 2) << 4) | (j & 15);
  float sum = 0.f;
#pragma unroll
  for (int ww = 0; ww < kMdWaves; ++ww) sum += red[ww * kPer + (j >> 4) * 64 + l][row & 3];
  return sum;
}

}  // namespace

// s_a t (kBT false: in = x, W = A) or s_a u (kBT true: in = dY, W = B), rounded
// to bf16 once, [M][rp] with the ranks past r zero; rows without an adapter are
// not written. (One bf16 number each, as for a single adapter: the output is
// bf16 itself. The scale goes in before the rounding, so that the GEMMs need
// no scale.) A block of 16 rows takes one pass per adapter among its rows (rows
// of a request follow each other, so mostly one); blockIdx.y deals the passes
// out. Workgroups past `blocks` copy x into MFMA order: fragment (tile, ss, j)
// has, at lane (g, c), columns 256 ss + 64 g + 8 j + (0 2 | 4 6 | 1 3 | 5 7)
// of row 16 tile + c, zero past M and Kc.
template <int RT, int GS, bool kBT>
__global__ __launch_bounds__(64 * kMdWaves) void k_mdown(const uint16_t* in, int64_t M, int Kc, const uint16_t* W,
                                                         MultiLora ml, int r, int rp, uint16_t* __restrict__ out,
                                                         unsigned blocks, u32x4* __restrict__ frags, int64_t nfrag) {
  if (blockIdx.x >= blocks) {
    if (kBT || blockIdx.y) return;
    const int nss = (Kc + 255) / 256;
    const int64_t f = static_cast<int64_t>(blockIdx.x - blocks) * kMdWaves + (threadIdx.x >> 6);
    if (f >= nfrag) return;
    const int lane = threadIdx.x & 63;
    const int64_t tile = f / (8 * nss);
    const int rest = static_cast<int>(f - tile * 8 * nss);
    const int64_t m = 16 * tile + (lane & 15);
    const int k = 256 * (rest >> 3) + 64 * (lane >> 4) + 8 * (rest & 7);
    u32x4 v = {0u, 0u, 0u, 0u};
    if (m < M && k < Kc) v = perm8(ld16(in + m * Kc + k));
    frags[f * 64 + lane] = v;
    return;
  }
  constexpr int kPer = md_per<RT, GS, kBT>();
  __shared__ u32x4 lds[kMdWaves * kPer];
  const int t = threadIdx.x, lane = t & 63;
  const int w = __builtin_amdgcn_readfirstlane(t >> 6);
  const int c = lane & 15;
  const int64_t m0 = static_cast<int64_t>(blockIdx.x) * 16;
  int id = m0 + c < M ? ml.index[m0 + c] : -1;
  if (static_cast<unsigned>(id) >= static_cast<unsigned>(ml.n)) id = -1;
  uint32_t pend = static_cast<uint32_t>(__ballot(id >= 0)) & 0xFFFFu;
  f32x4* const red = reinterpret_cast<f32x4*>(lds);
  for (unsigned ord = 0; pend; ++ord) {
    const int a = __builtin_amdgcn_readlane(id, __builtin_ctz(pend));
    const uint32_t rows = static_cast<uint32_t>(__ballot(id == a)) & 0xFFFFu;
    pend &= ~rows;
    if (ord % gridDim.y != blockIdx.y) continue;
    f32x4 acc[RT];
    down_acc<RT, GS, kBT, kActBf16>(in, nullptr, (rows >> c) & 1 ? m0 + c : -1, Kc,
                                    W + static_cast<int64_t>(a) * r * Kc, r, lds + w * kPer, acc, w, lane);
#pragma unroll
    for (int jt = 0; jt < RT; ++jt) red[w * kPer + jt * 64 + lane] = acc[jt];
    const float scale = ml.scale[a];
    __syncthreads();
    for (int e = t; e < 16 * rp; e += 64 * kMdWaves) {
      const int row = e / rp, j = e - row * rp;
      if (!((rows >> row) & 1)) continue;
      out[(m0 + row) * rp + j] = j < 16 * RT ? bf16_bits(scale * md_sum<RT, kPer>(red, row, j)) : uint16_t{0};
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// gradients
// ---------------------------------------------------------------------------
// Rows of each adapter, one wave per adapter. Every workgroup counts the whole
// batch (n counters in LDS; a wave whose rows agree adds once), then each wave
// places its adapter's chunks, items and rows after those of the adapters
// before it.
__global__ __launch_bounds__(256) void k_msort(const int* __restrict__ index, int64_t M, int n, int ch_per_item,
                                               GradLists L) {
  __shared__ int hist[kMaxAdapters];
  const int t = threadIdx.x, lane = t & 63;
  const int w = __builtin_amdgcn_readfirstlane(t >> 6);
  for (int i = t; i < n; i += 256) hist[i] = 0;
  __syncthreads();
  for (int64_t m = t; m < M; m += 256) {
    const int id = index[m];
    const int first = __builtin_amdgcn_readfirstlane(id);
    const uint64_t live = __ballot(true), same = __ballot(id == first);
    if (same == live) {
      if (static_cast<unsigned>(first) < static_cast<unsigned>(n) && lane == __builtin_ctzll(live))
        atomicAdd(&hist[first], __builtin_popcountll(live));
    } else if (static_cast<unsigned>(id) < static_cast<unsigned>(n)) {
      atomicAdd(&hist[id], 1);
    }
  }
  __syncthreads();
  const int a = blockIdx.x * 4 + w;
  if (a >= n) return;
  int chunks = 0, items = 0, slots = 0;
  for (int b = lane; b < a; b += 64) {
    const int ch = (hist[b] + 63) >> 6, it = (ch + ch_per_item - 1) / ch_per_item;
    chunks += ch;
    items += it;
    slots += it > 1 ? it : 0;
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    chunks += __shfl_xor(chunks, o);
    items += __shfl_xor(items, o);
    slots += __shfl_xor(slots, o);
  }
  const int nch = (hist[a] + 63) >> 6, nit = (nch + ch_per_item - 1) / ch_per_item;
  if (lane == 0) {
    L.adapter[a] = GradAdapter{nit, slots};
    if (a == n - 1) {
      L.total[0] = chunks + nch;
      L.total[1] = items + nit;
    }
  }
  for (int i = lane; i < nit; i += 64) {
    const int c0 = i * ch_per_item, c1 = c0 + ch_per_item;
    L.item[items + i] = GradItem{a, chunks + c0, chunks + (c1 < nch ? c1 : nch), nit > 1 ? slots + i : -1};
  }
  for (int i = lane; i < nch; i += 64) L.chunk_adapter[chunks + i] = a;
  // the rows, in batch order
  int* const rows = L.rows + static_cast<int64_t>(chunks) * 64;
  int pos = 0;
  for (int64_t m = 0; m < M; m += 64 * 8) {
    int id[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int64_t mm = m + 64 * u + lane;
      id[u] = mm < M ? index[mm] : -1;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const uint64_t hit = __ballot(id[u] == a);
      if (id[u] == a) rows[pos + __builtin_popcountll(hit & ((1ull << lane) - 1))] = static_cast<int>(m + 64 * u + lane);
      pos += __builtin_popcountll(hit);
    }
  }
  for (int i = pos + lane; i < nch * 64; i += 64) rows[i] = -1;
}

// the row listed at place p (no list: the batch itself)
__device__ __forceinline__ int64_t grad_row(const GradLists& L, int64_t p, int64_t M) {
  if (L.rows) return L.rows[p];
  return p < M ? p : -1;
}

template <int RT, int kPer>
__device__ __forceinline__ void store_split(const f32x4* red, uint16_t* qt, int64_t Mp, int64_t p0, int t) {
  // 16 rows x 16 RT ranks; consecutive threads take consecutive rows of a rank
  for (int e = t; e < 16 * 16 * RT; e += 64 * kMdWaves) {
    const int row = e & 15, j = e >> 4;
    float v = md_sum<RT, kPer>(red, row, j);
#pragma unroll
    for (int p = 0; p < kSplit; ++p) {
      const uint16_t b = bf16_bits(v);
      qt[(static_cast<int64_t>(p) * 16 * RT + j) * Mp + p0 + row] = b;
      v -= bf16_lo(b);
    }
  }
}

// t^T (even blocks) and u^T (odd blocks) of 16 listed rows: [3][16 RT][Mp] bf16
template <int RT, int GS, int XF>
__global__ __launch_bounds__(64 * kMdWaves) void k_gdown(const void* x, const uint16_t* tops, const uint16_t* dy, int64_t M,
                                                         int N, int K, const uint16_t* A, const uint16_t* B, int r,
                                                         GradLists L, int64_t Mp, uint16_t* __restrict__ tt,
                                                         uint16_t* __restrict__ ut) {
  constexpr int kPerT = md_per<RT, GS, false>(), kPerU = md_per<RT, GS, true>();
  __shared__ u32x4 lds[kMdWaves * (kPerT > kPerU ? kPerT : kPerU)];
  const int t = threadIdx.x, lane = t & 63;
  const int w = __builtin_amdgcn_readfirstlane(t >> 6);
  const int64_t p0 = static_cast<int64_t>(blockIdx.x >> 1) * 16;
  int64_t a = 0;
  if (L.rows) {
    if ((p0 >> 6) >= L.total[0]) return;
    a = L.chunk_adapter[p0 >> 6];
  }
  const int64_t row = grad_row(L, p0 + (lane & 15), M);
  f32x4 acc[RT];
  f32x4* const red = reinterpret_cast<f32x4*>(lds);
  if (blockIdx.x & 1) {
    down_acc<RT, GS, true, kActBf16>(dy, nullptr, row, N, B + a * N * r, r, lds + w * kPerU, acc, w, lane);
#pragma unroll
    for (int jt = 0; jt < RT; ++jt) red[w * kPerU + jt * 64 + lane] = acc[jt];
    __syncthreads();
    store_split<RT, kPerU>(red, ut, Mp, p0, t);
  } else {
    down_acc<RT, GS, false, XF>(x, tops, row, K, A + a * r * K, r, lds + w * kPerT, acc, w, lane);
#pragma unroll
    for (int jt = 0; jt < RT; ++jt) red[w * kPerT + jt * 64 + lane] = acc[jt];
    __syncthreads();
    store_split<RT, kPerT>(red, tt, Mp, p0, t);
  }
}

namespace {

constexpr int kGCols = 128;                    // columns of P per workgroup (32 per wave)

// P tile in LDS: two halves of 64 rows x 64 columns, chunk c of row m at
// c ^ 2 f(m), f(m) = ((m >> 3) & 3) ^ ((m >> 1) & 1), so that a transposed read
// of 4 rows at offsets 8 G + 4 q touches each bank twice (as in grad.hip)
__device__ __forceinline__ int g_swz(int m) { return 2 * (((m >> 3) & 3) ^ ((m >> 1) & 1)); }

// One item of one 128-column tile. kTR: dA (P = x, out [r][C]); else dB
// (P = dY, out [C][r]).
template <int NT, bool kTR, int XF>
__device__ __forceinline__ void grad_item(const void* P, const uint16_t* tops, int64_t M, int C, const uint16_t* Qt,
                                          int64_t Mp, int r, int ct, const GradItem& it, const GradLists& L,
                                          const float* scale, float alpha_r, int accumulate, float* part, float* out,
                                          u32x4* tile, u32x4* qtile) {
  constexpr int kQ = kSplit * 16 * NT * 8;     // 16-byte pieces of Q per chunk
  constexpr int kQPer = kQ / 256 + (kQ % 256 ? 1 : 0);
  const int t = threadIdx.x, lane = t & 63;
  const int w = __builtin_amdgcn_readfirstlane(t >> 6);
  const int G = lane >> 4, j16 = lane & 15;
  const int c0 = ct * kGCols;
  const u32x4 zero = {0u, 0u, 0u, 0u};
  // this thread's pieces of a chunk: columns 8 lc .. of rows lr + 16 i
  const int lr = t >> 4, lc = t & 15;
  const bool cin = c0 + 8 * lc < C;
  const int col = cin ? c0 + 8 * lc : 0;
  struct Regs {
    u32x4 p[4];
    uint32_t top[XF == kActBf16 ? 1 : 4];
    u32x4 q[kQPer];
    bool live[4];
  };
  auto load = [&](int ch, const int64_t (&rows)[4], Regs& R) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      R.live[i] = rows[i] >= 0;
      const int64_t row = R.live[i] ? rows[i] : 0;
      if constexpr (XF == kActBf16) {
        R.p[i] = ld16(static_cast<const uint16_t*>(P) + row * C + col);
      } else {
        const u32x2 v = *reinterpret_cast<const u32x2*>(static_cast<const uint8_t*>(P) + row * C + col);
        R.p[i].x = v.x;
        R.p[i].y = v.y;
        R.top[i] = tops[row * (C / 64) + (col >> 6)];
      }
    }
#pragma unroll
    for (int i = 0; i < kQPer; ++i) {
      const int e = t + 256 * i;
      const int rank = e >> 3;                  // of the 3 x 16 NT
      if (kQ % 256 == 0 || e < kQ)
        R.q[i] = ld16(Qt + static_cast<int64_t>(rank) * Mp + static_cast<int64_t>(ch) * 64 + 8 * (e & 7));
    }
  };
  auto rows_of = [&](int ch, int64_t (&rows)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) rows[i] = grad_row(L, static_cast<int64_t>(ch) * 64 + lr + 16 * i, M);
  };
  auto store = [&](const Regs& R, int buf) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = lr + 16 * i;
      u32x4 v;
      if constexpr (XF == kActBf16) v = R.p[i];
      else v = act8_decode8<XF>(u32x2{R.p[i].x, R.p[i].y}, act8_scale<XF>(R.top[i]));
      tile[buf * 1024 + (lc >> 3) * 512 + m * 8 + ((lc & 7) ^ g_swz(m))] = R.live[i] ? v : zero;
    }
#pragma unroll
    for (int i = 0; i < kQPer; ++i) {
      const int e = t + 256 * i, rank = e >> 3;
      if (kQ % 256 == 0 || e < kQ) qtile[buf * kQ + rank * 8 + ((e & 7) ^ ((rank >> 1) & 7))] = R.q[i];
    }
  };
  f32x4 acc[2][NT];
#pragma unroll
  for (int b = 0; b < 2; ++b)
#pragma unroll
    for (int jt = 0; jt < NT; ++jt) acc[b][jt] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto compute = [&](int buf) {
    const u32x4* T = tile + buf * 1024 + (w >> 1) * 512;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      bf16x8 pa[2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        s16x4 v[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int m = 32 * kk + 8 * G + 4 * q + (j16 >> 2);
          const int cc = 32 * (w & 1) + 16 * b + 4 * (j16 & 3);
          v[q] = ds_read_tr(T, (m * 8 + ((cc >> 3) ^ g_swz(m))) * 8 + (cc & 7));
        }
        pa[b] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7));
      }
#pragma unroll
      for (int p = 0; p < kSplit; ++p)
#pragma unroll
        for (int jt = 0; jt < NT; ++jt) {
          const int rank = p * 16 * NT + 16 * jt + j16;
          const bf16x8 qb = as_bf16x8(qtile[buf * kQ + rank * 8 + ((4 * kk + G) ^ ((rank >> 1) & 7))]);
#pragma unroll
          for (int b = 0; b < 2; ++b) acc[b][jt] = kTR ? mfma16(qb, pa[b], acc[b][jt]) : mfma16(pa[b], qb, acc[b][jt]);
        }
    }
  };
  // chunk ch + 1 is loaded while chunk ch is multiplied; its row numbers one chunk earlier
  Regs R;
  int64_t rows[4];
  const int last = it.c1 - 1;
  rows_of(it.c0, rows);
  load(it.c0, rows, R);
  rows_of(it.c0 + 1 <= last ? it.c0 + 1 : last, rows);
  store(R, 0);
  __syncthreads();
  for (int ch = it.c0; ch < it.c1; ++ch) {
    const int buf = (ch - it.c0) & 1;
    if (ch < last) {
      load(ch + 1, rows, R);
      rows_of(ch + 2 <= last ? ch + 2 : last, rows);
    }
    compute(buf);
    if (ch < last) store(R, buf ^ 1);          // its last readers passed the barrier of the chunk before
    __syncthreads();
  }

  const bool direct = it.slot < 0;
  const float s = direct ? (scale ? scale[it.adapter] : alpha_r) : 1.0f;
  float* dst = direct ? out + static_cast<int64_t>(it.adapter) * C * r : part + static_cast<int64_t>(it.slot) * C * r;
  const bool add = direct && accumulate;
#pragma unroll
  for (int b = 0; b < 2; ++b)
#pragma unroll
    for (int jt = 0; jt < NT; ++jt)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int cc = c0 + 32 * w + 16 * b + (kTR ? j16 : 4 * G + v);
        const int j = 16 * jt + (kTR ? 4 * G + v : j16);
        if (j < r && cc < C) {
          float* o = kTR ? dst + static_cast<int64_t>(j) * C + cc : dst + static_cast<int64_t>(cc) * r + j;
          const float val = s * acc[b][jt][v];
          *o = add ? *o + val : val;
        }
      }
}

}  // namespace

// blockIdx.x: the column tiles of dB (over dY), then those of dA (over x);
// blockIdx.y: the item
template <int NT, int XF>
__global__ __launch_bounds__(256) void k_mgrad(const void* x, const uint16_t* tops, const uint16_t* dy, int64_t M, int N,
                                               int K, int r, const uint16_t* tt, const uint16_t* ut, int64_t Mp, int ctb,
                                               GradLists L, int ch_per_item, int chunks, const float* scale, float alpha_r,
                                               int accumulate, float* partA, float* partB, float* dA, float* dB) {
  __shared__ u32x4 tile[2 * 1024];
  __shared__ u32x4 qtile[2 * kSplit * 16 * NT * 8];
  GradItem it;
  if (L.rows) {
    if (static_cast<int>(blockIdx.y) >= L.total[1]) return;
    it = L.item[blockIdx.y];
  } else {
    const int c0 = blockIdx.y * ch_per_item, c1 = c0 + ch_per_item;
    it = GradItem{0, c0, c1 < chunks ? c1 : chunks, gridDim.y > 1 ? static_cast<int>(blockIdx.y) : -1};
  }
  if (static_cast<int>(blockIdx.x) < ctb)
    grad_item<NT, false, kActBf16>(dy, nullptr, M, N, tt, Mp, r, blockIdx.x, it, L, scale, alpha_r, accumulate, partB, dB,
                                   tile, qtile);
  else
    grad_item<NT, true, XF>(x, tops, M, K, ut, Mp, r, blockIdx.x - ctb, it, L, scale, alpha_r, accumulate, partA, dA, tile,
                            qtile);
}

// out[a] (+)= s_a * sum of the adapter's partials, in item order; adapters
// without rows: zero (nothing when accumulating); those of one item are done.
// nb and na are multiples of 4.
__global__ __launch_bounds__(256) void k_mfinish(GradLists L, int items, const float* __restrict__ scale, float alpha_r,
                                                 int accumulate, int64_t nb, const float* __restrict__ partB,
                                                 float* __restrict__ dB, int64_t na, const float* __restrict__ partA,
                                                 float* __restrict__ dA) {
  const int64_t a = blockIdx.y;
  const GradAdapter ad = L.rows ? L.adapter[a] : GradAdapter{items, 0};
  if (ad.items == 1 || (ad.items == 0 && accumulate)) return;
  int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
  const float* p = partB;
  float* o = dB;
  int64_t n = nb;
  if (i >= nb) {
    i -= nb;
    p = partA, o = dA, n = na;
    if (i >= na) return;
  }
  f32x4 sum = {0.f, 0.f, 0.f, 0.f};
  if (ad.items) {
    p += static_cast<int64_t>(ad.slot) * n + i;
    for (int s = 0; s < ad.items; ++s) sum += *reinterpret_cast<const f32x4*>(p + s * n);
    sum *= scale ? scale[a] : alpha_r;
  }
  f32x4* dst = reinterpret_cast<f32x4*>(o + a * n + i);
  if (accumulate) sum += *dst;
  *dst = sum;
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
hipError_t launch_multi_down(bool wrow, const uint16_t* in, int64_t M, int64_t Kc, const uint16_t* W,
                             const MultiLora& ml, int r, uint16_t* out, hipStream_t stream, u32x4* frags,
                             int64_t mtiles) {
  const int rp = static_cast<int>(rank_pad(r));
  const int64_t blocks = cdiv(M, 16);
  // the passes of a block side by side where that leaves at most one workgroup per CU
  int64_t y = 256 / blocks;
  if (y > ml.n) y = ml.n;
  if (y > M) y = M;
  if (y > 16) y = 16;
  if (y < 1) y = 1;
  const int64_t nfrag = frags ? mtiles * cdiv(Kc, 256) * 8 : 0;
  const dim3 grid(static_cast<unsigned>(blocks + cdiv(nfrag, kMdWaves)), static_cast<unsigned>(y)), block(64 * kMdWaves);
  const int kc = static_cast<int>(Kc);
  const unsigned nb = static_cast<unsigned>(blocks);
#define QNF4_MD1(RTV, GSV, BT)                                                                                         \
  hipLaunchKernelGGL(HIP_KERNEL_NAME(k_mdown<RTV, GSV, BT>), grid, block, 0, stream, in, M, kc, W, ml, r, rp, out, nb, \
                     frags, nfrag)
#define QNF4_MD(RTV, GSV)                 \
  do {                                    \
    if (wrow) QNF4_MD1(RTV, GSV, false);  \
    else QNF4_MD1(RTV, GSV, true);        \
  } while (0)
  switch (down_nt(r)) {
    case 1: QNF4_MD(1, 4); break;
    case 2: QNF4_MD(2, 2); break;
    case 4: QNF4_MD(4, 1); break;
    default: QNF4_MD(8, 1); break;
  }
#undef QNF4_MD
#undef QNF4_MD1
  return hipGetLastError();
}

MultiGradPlan multi_grad_plan(int64_t M, int64_t N, int64_t K, int r, int n, bool listed) {
  MultiGradPlan g;
  g.nt = down_nt(r);
  const int64_t full = cdiv(M, 64);
  const int64_t used = listed ? (M < n ? M : n) : 0;       // adapters that can have rows
  g.chunks = listed ? M / 64 + used : full;                // at most, with each adapter's last chunk partial
  g.Mp = g.chunks * 64;
  // about four workgroups per CU over all column tiles, whole chunks per item
  const int64_t ct = cdiv(N, kGCols) + cdiv(K, kGCols);
  const int64_t want = cdiv(1024, ct);
  g.per_item = cdiv(full, want);
  g.items = listed ? full / g.per_item + used : cdiv(full, g.per_item);
  // slots: an adapter of I >= 2 items has more than (I - 1) per_item full chunks
  g.slots = listed ? 2 * (full / g.per_item) : (g.items > 1 ? g.items : 0);
  size_t off = kWsCounterBytes;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += align256(bytes);
    return o;
  };
  if (listed) {
    g.rows_off = take(static_cast<size_t>(g.Mp) * 4);
    g.chunk_off = take(static_cast<size_t>(g.chunks) * 4);
    g.item_off = take(static_cast<size_t>(g.items) * sizeof(GradItem));
    g.adapter_off = take(static_cast<size_t>(n) * sizeof(GradAdapter));
    g.total_off = take(8);
  }
  const size_t q = static_cast<size_t>(kSplit) * 16 * g.nt * g.Mp * 2;
  g.tt_off = take(q);
  g.ut_off = take(q);
  g.pa_off = take(static_cast<size_t>(g.slots) * K * r * 4);
  g.pb_off = take(static_cast<size_t>(g.slots) * N * r * 4);
  g.total = off;
  return g;
}

hipError_t launch_multi_grad(const void* x, const uint16_t* tops, int xfmt, const uint16_t* dy, int64_t M, int64_t N,
                             int64_t K, const uint16_t* A, const uint16_t* B, const float* scale, float alpha_r, int n,
                             const int* index, int r, float* dA, float* dB, int accumulate, void* ws,
                             hipStream_t stream) {
  const MultiGradPlan g = multi_grad_plan(M, N, K, r, n, index != nullptr);
  char* wsb = static_cast<char*>(ws);
  GradLists L{};
  if (index) {
    L.rows = reinterpret_cast<int*>(wsb + g.rows_off);
    L.chunk_adapter = reinterpret_cast<int*>(wsb + g.chunk_off);
    L.item = reinterpret_cast<GradItem*>(wsb + g.item_off);
    L.adapter = reinterpret_cast<GradAdapter*>(wsb + g.adapter_off);
    L.total = reinterpret_cast<int*>(wsb + g.total_off);
    hipLaunchKernelGGL(k_msort, dim3(static_cast<unsigned>(cdiv(n, 4))), dim3(256), 0, stream, index, M, n,
                       static_cast<int>(g.per_item), L);
  }
  uint16_t* tt = reinterpret_cast<uint16_t*>(wsb + g.tt_off);
  uint16_t* ut = reinterpret_cast<uint16_t*>(wsb + g.ut_off);
  float* pa = reinterpret_cast<float*>(wsb + g.pa_off);
  float* pb = reinterpret_cast<float*>(wsb + g.pb_off);
  const int ni = static_cast<int>(N), ki = static_cast<int>(K), per = static_cast<int>(g.per_item);
  const int ctb = static_cast<int>(cdiv(N, kGCols)), cta = static_cast<int>(cdiv(K, kGCols));
  const dim3 dgrid(static_cast<unsigned>(g.chunks * 8)), dblock(64 * kMdWaves);
  const dim3 ggrid(static_cast<unsigned>(ctb + cta), static_cast<unsigned>(g.items));
#define QNF4_MG(NTV, GSV, XFV)                                                                                       \
  do {                                                                                                               \
    hipLaunchKernelGGL(HIP_KERNEL_NAME(k_gdown<NTV, GSV, XFV>), dgrid, dblock, 0, stream, x, tops, dy, M, ni, ki, A, B, \
                       r, L, g.Mp, tt, ut);                                                                          \
    hipLaunchKernelGGL(HIP_KERNEL_NAME(k_mgrad<NTV, XFV>), ggrid, dim3(256), 0, stream, x, tops, dy, M, ni, ki, r, tt, \
                       ut, g.Mp, ctb, L, per, static_cast<int>(g.chunks), scale, alpha_r, accumulate, pa, pb, dA, dB); \
  } while (0)
#define QNF4_MGX(NTV, GSV)                              \
  do {                                                  \
    if (xfmt == kActBf16) QNF4_MG(NTV, GSV, kActBf16);  \
    else if (xfmt == kActInt8) QNF4_MG(NTV, GSV, kActInt8); \
    else QNF4_MG(NTV, GSV, kActE4m3);                   \
  } while (0)
  switch (g.nt) {
    case 1: QNF4_MGX(1, 4); break;
    case 2: QNF4_MGX(2, 2); break;
    case 4: QNF4_MGX(4, 1); break;
    default: QNF4_MGX(8, 1); break;
  }
#undef QNF4_MGX
#undef QNF4_MG
  // nothing is left to sum or to clear: a single adapter of one item, or a
  // list without slots that is added to
  if (index ? (g.slots == 0 && accumulate) : g.slots == 0) return hipGetLastError();
  const int64_t nb = N * r, na = K * r;
  hipLaunchKernelGGL(k_mfinish, dim3(static_cast<unsigned>(cdiv((nb + na) / 4, 256)), static_cast<unsigned>(n)), dim3(256),
                     0, stream, L, static_cast<int>(g.items), scale, alpha_r, accumulate, nb, pb, dB, na, pa, dA);
  return hipGetLastError();
}

}  // namespace qnf4
