// Forward of a batch of many requests (up to some hundred rows) through one
// NF4 weight with a pool of adapters, for gfx950:
//     y_m = bf16( x_m . W'^T + t_m . B_a^T ),  t_m = bf16(s_a . x_m . A_a^T)
// (rows, adapters and t as in multi.hip). At these sizes the stored weight is
// what has to be read (0.516 bytes a parameter) and the tiled GEMM's 256 x 256
// tiles would leave most of the chip idle, so the weight is streamed by small
// items.
//
// k_mprep (one launch before it): t of every row, and x copied into the order
// in which the MFMAs take it (16 rows x 256 deep = eight 1 KB fragments), rows
// past M and columns past K zero. The main kernel's loads of x are then whole
// 1 KB lines from L2 straight into registers: no LDS, no barrier in its loop.
//
// k_mstream: an item is 64 weight rows x one of S ranges of K x 16 MT rows of
// x. The four waves of a workgroup take every fourth 256-deep super-step of the
// range: lane (g, c) holds block 4 ss + g of weight row c of each of four
// 16-row tiles (32 code bytes, one scale, one magnitude table for 64 weights),
// eight 16x16x32 MFMAs per tile and 16 rows of x. The next super-step's codes
// and the next half's x are in flight while a half is decoded and multiplied.
// The waves' sums meet in LDS; wave w then owns 16 columns, adds their adapter
// term (split s takes the row tiles i with i % S == s; the B rows of up to eight
// adapters in flight at a time, selected row by row after the product so that
// one adapter's NaN stays with its rows), and either writes y or leaves an fp32
// partial, which the last split to arrive adds up in split order.
// Splitting K inside the workgroup first keeps those partials few: S = 2 or 4
// at 4096 deep where one K range per wave row would need 8 to 16.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mm_common.hpp"
#include "multi.hpp"

namespace qnf4 {

namespace {

constexpr int kMsRows = 64;                      // weight rows per item
constexpr int kMsNT = 4;                         // 16-row tiles of them
constexpr int kMsBatch = 8;                      // adapter fragments in flight in the epilogue

struct MsArgs {
  const u32x4* xp;          // [M16][nss][8][64] fragments of x
  const uint16_t* t;        // [M][rp]
  const uint8_t* packed;
  const int8_t* qscale;
  const float* step;
  const uint16_t* B;        // [n][N][r]
  uint16_t* y;
  float* part;              // [item][16 MT][64]
  unsigned* cnt;            // one per (row block of W, block of x rows)
  int M, N, K, r, rp, S, mblocks, items;
};

template <int MT>
__global__ __launch_bounds__(256, MT <= 2 ? 2 : 1) void k_mstream(MsArgs P, MultiLora ml, Codebook cb) {
  __shared__ f32x4 red[4 * kMsNT * MT * 64];
  __shared__ int last_flag;
  const int t = threadIdx.x, lane = t & 63;
  const int w = __builtin_amdgcn_readfirstlane(t >> 6);
  const int g = lane >> 4, c = lane & 15;
  // XCD (blockIdx % 8) gets a contiguous range: the blocks of x rows that
  // share weights, then the splits, run side by side there
  const int item = (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3);
  if (item >= P.items) return;
  const int mb = item % P.mblocks, s = (item / P.mblocks) % P.S, nb = item / (P.mblocks * P.S);
  const int N = P.N, K = P.K, nbr = K / 64, nss = (nbr + 3) / 4;
  const int ss0 = static_cast<int>(static_cast<int64_t>(nss) * s / P.S);
  const int ss1 = static_cast<int>(static_cast<int64_t>(nss) * (s + 1) / P.S);
  const int n0 = nb * kMsRows, mt0 = mb * MT;

  const uint8_t* crow[kMsNT];
  int64_t brow[kMsNT];
#pragma unroll
  for (int nt = 0; nt < kMsNT; ++nt) {
    const int n = n0 + 16 * nt + c < N ? n0 + 16 * nt + c : N - 1;
    crow[nt] = P.packed + static_cast<int64_t>(n) * (K / 2);
    brow[nt] = static_cast<int64_t>(n) * nbr;
  }
  struct Codes {
    u32x4 cw[kMsNT][2];
    int8_t q[kMsNT];
    float d[kMsNT];
  };
  auto load_codes = [&](int ss, Codes& C) {
    const int kb = ss * 4 + g < nbr ? ss * 4 + g : nbr - 1;   // past K: x is zero there
#pragma unroll
    for (int nt = 0; nt < kMsNT; ++nt) {
      C.cw[nt][0] = ld16(crow[nt] + kb * 32);
      C.cw[nt][1] = ld16(crow[nt] + kb * 32 + 16);
    }
#pragma unroll
    for (int nt = 0; nt < kMsNT; ++nt) {
      C.q[nt] = P.qscale[brow[nt] + kb];
      C.d[nt] = P.step[(brow[nt] + kb) >> 8];
    }
  };
  auto load_x = [&](int ss, int h, u32x4 (&x)[4][MT]) {
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const u32x4* xs = P.xp + ((static_cast<int64_t>(mt0 + i) * nss + ss) * 8 + 4 * h) * 64 + lane;
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j][i] = xs[64 * j];
    }
  };
  // the rows' adapters, asked for now and used at the end
  int id[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int m = 16 * (mt0 + i) + c;
    id[i] = m < P.M ? ml.index[m] : -1;
    if (static_cast<unsigned>(id[i]) >= static_cast<unsigned>(ml.n)) id[i] = -1;
  }
  f32x4 acc[kMsNT][MT];
#pragma unroll
  for (int nt = 0; nt < kMsNT; ++nt)
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[nt][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  MagTable tb[kMsNT];
  auto multiply = [&](const Codes& C, int h, const u32x4 (&x)[4][MT]) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int nt = 0; nt < kMsNT; ++nt) {
        const u32x4 cw = C.cw[nt][h];
        const uint32_t d = j == 0 ? cw.x : j == 1 ? cw.y : j == 2 ? cw.z : cw.w;
        const bf16x8 wf = as_bf16x8(decode8_perm(d, tb[nt]));
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[nt][i] = mfma16(as_bf16x8(x[j][i]), wf, acc[nt][i]);
      }
  };
  Codes cc, cn;
  u32x4 x0[4][MT], x1[4][MT];
  int ss = ss0 + w;
  if (ss < ss1) {
    load_codes(ss, cc);
    load_x(ss, 0, x0);
    for (; ss < ss1; ss += 4) {
      const int nx = ss + 4 < ss1 ? ss + 4 : ss;
      __builtin_amdgcn_sched_barrier(0);
      load_x(ss, 1, x1);
      load_codes(nx, cn);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int nt = 0; nt < kMsNT; ++nt) tb[nt] = make_table(cb, block_scale(cc.q[nt], cc.d[nt]));
      multiply(cc, 0, x0);
      __builtin_amdgcn_sched_barrier(0);
      load_x(nx, 0, x0);
      __builtin_amdgcn_sched_barrier(0);
      multiply(cc, 1, x1);
      cc = cn;
    }
  }

  // the waves' sums, in wave order; wave w keeps the 16 columns of tile w
#pragma unroll
  for (int nt = 0; nt < kMsNT; ++nt)
#pragma unroll
    for (int i = 0; i < MT; ++i) red[((w * kMsNT + nt) * MT + i) * 64 + lane] = acc[nt][i];
  __syncthreads();
  f32x4 sum[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    sum[i] = red[(w * MT + i) * 64 + lane];
#pragma unroll
    for (int ww = 1; ww < 4; ++ww) sum[i] += red[((ww * kMsNT + w) * MT + i) * 64 + lane];
  }

  // the adapter term of this wave's 16 columns: lane (g, c) has column n, rows
  // 4 g + v of each tile
  const int n = n0 + 16 * w + c;
  {
    const int64_t nr = n < N ? n : N - 1;
    const int r = P.r, rp = P.rp;
    const bool vec = (r & 7) == 0;
    const u32x4 zero = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      if ((mt0 + i) % P.S != s) continue;
      const int m = 16 * (mt0 + i) + c;
      uint32_t pend = static_cast<uint32_t>(__ballot(id[i] >= 0)) & 0xFFFFu;
      if (!pend) continue;
      const uint16_t* trow = P.t + static_cast<int64_t>(m < P.M ? m : P.M - 1) * rp;
      f32x4 lora = {0.f, 0.f, 0.f, 0.f};
      while (pend) {
        uint32_t rows[kMsBatch];
        int ad[kMsBatch];
#pragma unroll
        for (int u = 0; u < kMsBatch; ++u) {
          ad[u] = __builtin_amdgcn_readlane(id[i], pend ? __builtin_ctz(pend) : 0);
          rows[u] = pend ? static_cast<uint32_t>(__ballot(id[i] == ad[u])) & 0xFFFFu : 0u;
          pend &= ~rows[u];
        }
        f32x4 p[kMsBatch];
#pragma unroll
        for (int u = 0; u < kMsBatch; ++u) p[u] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int j0 = 0; j0 < r; j0 += 32) {
          const int col = j0 + 8 * g;
          const u32x4 tv = ld16(trow + (col < rp ? col : 0));
          u32x4 bf[kMsBatch];
#pragma unroll
          for (int u = 0; u < kMsBatch; ++u) {
            if (!rows[u]) continue;
            const uint16_t* br = P.B + (static_cast<int64_t>(ad[u]) * N + nr) * r;
            if (vec) bf[u] = ld16(br + (col < r ? col : 0));
            else bf[u] = load_row8(br, col, r, false);
          }
#pragma unroll
          for (int u = 0; u < kMsBatch; ++u) {
            if (!rows[u]) continue;
            p[u] = mfma16(as_bf16x8(col < r ? tv : zero), as_bf16x8(col < r ? bf[u] : zero), p[u]);
          }
        }
#pragma unroll
        for (int u = 0; u < kMsBatch; ++u)
#pragma unroll
          for (int v = 0; v < 4; ++v) lora[v] = (rows[u] >> (4 * g + v)) & 1u ? p[u][v] : lora[v];
      }
      sum[i] += lora;
    }
  }

  // y (or, with a split K, first the partial sums): 16 MT rows x 64 columns
  const int mrows = P.M - 16 * mt0 < 16 * MT ? P.M - 16 * mt0 : 16 * MT;
  uint16_t* const yb = P.y + static_cast<int64_t>(16 * mt0) * N + n0;
  const int ncols = N - n0 < kMsRows ? N - n0 : kMsRows;
  if (P.S == 1) {
    __syncthreads();                             // every wave has read its sums
    uint16_t* const tile = reinterpret_cast<uint16_t*>(red);
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) tile[(16 * i + 4 * g + v) * 72 + 16 * w + c] = bf16_bits(sum[i][v]);
    __syncthreads();
    const bool wide = ncols == kMsRows && N % 8 == 0;
    for (int e = t; e < mrows * 8; e += 256) {
      const int row = e >> 3, col = 8 * (e & 7);
      const uint16_t* src = tile + row * 72 + col;
      uint16_t* dst = yb + static_cast<int64_t>(row) * N + col;
      if (wide) {
        *reinterpret_cast<u32x4*>(dst) = *reinterpret_cast<const u32x4*>(src);
      } else {
        for (int q = 0; q < 8; ++q)
          if (col + q < ncols) dst[q] = src[q];
      }
    }
    return;
  }
  // the partials and the counter go through device-scope accesses, coherent
  // across the XCDs' caches without flushing them; every wave waits for its own
  // stores before the workgroup counts itself in
  constexpr int kPart = 16 * MT * kMsRows;
  float* const mine = P.part + (static_cast<int64_t>(nb * P.mblocks + mb) * P.S + s) * kPart;
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int row = 16 * i + 4 * g + v;
      if (row < mrows)
        __hip_atomic_store(mine + row * kMsRows + 16 * w + c, sum[i][v], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  unsigned* const cnt = P.cnt + nb * P.mblocks + mb;
  if (t == 0) {
    const unsigned old = __hip_atomic_fetch_add(cnt, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    last_flag = old == static_cast<unsigned>(P.S - 1);
  }
  __syncthreads();
  if (!last_flag) return;
  const __amdgpu_buffer_rsrc_t prs = __builtin_amdgcn_make_buffer_rsrc(
      P.part + static_cast<int64_t>(nb * P.mblocks + mb) * P.S * kPart, 0, P.S * kPart * 4, 0x00020000);
  for (int e = t; e < mrows * 16; e += 256) {
    const int row = e >> 4, col = 4 * (e & 15);
    f32x4 v[kMsMaxSplit];
#pragma unroll
    for (int u = 0; u < kMsMaxSplit; ++u)
      if (u < P.S)
        v[u] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                             prs, static_cast<uint32_t>((u * kPart + row * kMsRows + col) * 4), 0, 16));
    f32x4 out = v[0];
#pragma unroll
    for (int u = 1; u < kMsMaxSplit; ++u)
      if (u < P.S) out += v[u];
    uint16_t* dst = yb + static_cast<int64_t>(row) * N + col;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (col + q < ncols) dst[q] = bf16_bits(out[q]);
  }
  if (t == 0) __hip_atomic_store(cnt, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

}  // namespace

// Items: blocks of 64 weight rows x blocks of 16 MT rows of x (MT up to 4) x S
// ranges of K. S is the most that keeps every item resident at once (two
// workgroups per CU up to MT = 2, one above; a second round costs a whole item:
// 48 rows at 11008 x 4096 take 21 us with S = 1, 29 with 2, 35 with 3) and
// leaves every wave a super-step.
MsPlan ms_plan(int64_t M, int64_t N, int64_t K, int r, int n) {
  MsPlan p;
  const int64_t mtiles = cdiv(M, 16), nss = cdiv(K, 256);
  p.MT = static_cast<int>(mtiles < 4 ? mtiles : 4);
  p.mblocks = cdiv(mtiles, p.MT);
  const int64_t blocks = cdiv(N, kMsRows) * p.mblocks;
  int64_t S = (p.MT <= 2 ? 512 : 256) / blocks;
  if (S > cdiv(nss, 4)) S = cdiv(nss, 4);
  if (S > kMsMaxSplit) S = kMsMaxSplit;
  p.S = S < 1 ? 1 : S;
  size_t off = kWsCounterBytes;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += align256(bytes);
    return o;
  };
  p.t_off = take(static_cast<size_t>(M * rank_pad(r) * 2));
  p.x_off = take(static_cast<size_t>(p.mblocks * p.MT * nss) * 8192);
  p.down_off = take(multi_down_plan(M, K, r, n).part_bytes);
  p.part_off = take(p.S > 1 ? static_cast<size_t>(blocks * p.S) * 16 * p.MT * kMsRows * 4 : 0);
  p.total = off;
  return p;
}

hipError_t launch_mstream(const MsPlan& p, const uint16_t* x, int64_t M, int64_t N, int64_t K, const uint8_t* packed,
                          const int8_t* qscale, const float* step, const uint16_t* A, const uint16_t* B,
                          const MultiLora& ml, int r, uint16_t* y, void* ws, const Codebook& cb, hipStream_t stream) {
  char* wsb = static_cast<char*>(ws);
  uint16_t* t = reinterpret_cast<uint16_t*>(wsb + p.t_off);
  u32x4* xp = reinterpret_cast<u32x4*>(wsb + p.x_off);
  const hipError_t e = launch_multi_down(true, x, M, K, A, ml, r, t, ws, reinterpret_cast<float*>(wsb + p.down_off), stream,
                                         xp, p.mblocks * p.MT);
  if (e != hipSuccess) return e;
  MsArgs a{};
  a.xp = xp;
  a.t = t;
  a.packed = packed;
  a.qscale = qscale;
  a.step = step;
  a.B = B;
  a.y = y;
  a.part = reinterpret_cast<float*>(wsb + p.part_off);
  a.cnt = reinterpret_cast<unsigned*>(wsb);
  a.M = static_cast<int>(M);
  a.N = static_cast<int>(N);
  a.K = static_cast<int>(K);
  a.r = r;
  a.rp = static_cast<int>(rank_pad(r));
  a.S = static_cast<int>(p.S);
  a.mblocks = static_cast<int>(p.mblocks);
  a.items = static_cast<int>(cdiv(N, kMsRows) * p.mblocks * p.S);
  const dim3 grid(static_cast<unsigned>(round_up(a.items, 8)));
  mark_kernel(0, stream);
  switch (p.MT) {
    case 1: hipLaunchKernelGGL(HIP_KERNEL_NAME(k_mstream<1>), grid, dim3(256), 0, stream, a, ml, cb); break;
    case 2: hipLaunchKernelGGL(HIP_KERNEL_NAME(k_mstream<2>), grid, dim3(256), 0, stream, a, ml, cb); break;
    case 3: hipLaunchKernelGGL(HIP_KERNEL_NAME(k_mstream<3>), grid, dim3(256), 0, stream, a, ml, cb); break;
    default: hipLaunchKernelGGL(HIP_KERNEL_NAME(k_mstream<4>), grid, dim3(256), 0, stream, a, ml, cb); break;
  }
  mark_kernel(1, stream);
  return hipGetLastError();
}

}  // namespace qnf4
