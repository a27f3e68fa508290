// Forward of a batch of many requests (up to some hundred rows) through one
// NF4 weight with a pool of adapters, for gfx950:
//     y_m = bf16( x_m . W'^T + t_m . B_a^T ),  t_m = bf16(s_a . x_m . A_a^T)
// (rows, adapters and t as in multi.hip). At these sizes the stored weight is
// what has to be read (0.516 bytes a parameter) and the tiled GEMM's 256 x 256
// tiles would leave most of the chip idle, so the weight is streamed by small
// items.
//
// k_mdown (one launch before it): t of every row, and x copied into the order
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
// term (split s takes the row tiles i with i % S == s; the B rows of all
// its adapters in flight at once, selected row by row after the product so that
// one adapter's NaN stays with its rows), and either writes y or leaves an fp32
// partial, which the last split to arrive adds up in split order.
// Splitting K inside the workgroup first keeps those partials few: S = 2 or 4
// at 4096 deep where one K range per wave row would need 8 to 16.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "down.hpp"
#include "multi.hpp"

namespace qnf4 {

namespace {

constexpr int kMsRows = 64;                      // weight rows per item
constexpr int kMsNT = 4;                         // 16-row tiles of them
constexpr int kMsBatch = 16;                     // adapter fragments in flight in the epilogue: a whole tile's

struct MsArgs {
  const u32x4* xp;          // [M16][nss][8][64] fragments of x
  const uint16_t* t;        // [M][rp]
  const uint8_t* packed;
  const int8_t* qscale;
  const float* step;
  const uint16_t* B;        // [n][N][r]
  uint16_t* y;
  float* part;              // [row block of W, block of x rows][S][16 MT x 64]
  unsigned* cnt;            // one per (row block of W, block of x rows)
  int M, N, K, r, rp, S, mblocks, items;
};

// The adapter term of a 16 x 16 tile: lane (g, c) gets rows 4 g + v of column n.
// id: the adapter of row c (lanes of all g alike), < 0 for none; tv(col, hi, lo): 8
// values of t of row c from rank col (a multiple of 8), bf16. The B rows of up
// to kBatch adapters are asked for together; a row takes the product with its
// own adapter's, chosen after it (a NaN in one adapter must not reach the rows
// of another).
// kLo: tv(col, hi, lo) gives t as two bf16 numbers.
// kBatch: adapters at once (code that is run once is mostly fetched, not run:
// no more of it than the rows can need).
template <bool kLo, int kBatch, typename T>
__device__ __forceinline__ f32x4 adapter_term(int id, const uint16_t* B, int N, int64_t n, int r, int lane, T&& tv) {
  const int g = lane >> 4;
  const bool vec = (r & 7) == 0;
  const u32x4 zero = {0u, 0u, 0u, 0u};
  f32x4 lora = {0.f, 0.f, 0.f, 0.f};
  uint32_t pend = static_cast<uint32_t>(__ballot(id >= 0)) & 0xFFFFu;
  while (pend) {
    uint32_t rows[kBatch];
    int ad[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      ad[u] = __builtin_amdgcn_readlane(id, pend ? __builtin_ctz(pend) : 0);
      rows[u] = pend ? static_cast<uint32_t>(__ballot(id == ad[u])) & 0xFFFFu : 0u;
      pend &= ~rows[u];
    }
    f32x4 p[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) p[u] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < r; j0 += 32) {
      const int col = j0 + 8 * g;
      u32x4 bf[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (!rows[u]) continue;
        const uint16_t* br = B + (static_cast<int64_t>(ad[u]) * N + n) * r;
        if (vec) bf[u] = ld16(br + (col < r ? col : 0));
        else bf[u] = load_row8(br, col, r, false);
      }
      u32x4 hi, lo;
      tv(col, hi, lo);
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (!rows[u]) continue;
        const bf16x8 b = as_bf16x8(col < r ? bf[u] : zero);
        p[u] = mfma16(as_bf16x8(col < r ? hi : zero), b, p[u]);
        if constexpr (kLo) p[u] = mfma16(as_bf16x8(col < r ? lo : zero), b, p[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
#pragma unroll
      for (int v = 0; v < 4; ++v) lora[v] = (rows[u] >> (4 * g + v)) & 1u ? p[u][v] : lora[v];
  }
  return lora;
}

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
  // 4 g + v of each tile. The loop over the tiles stays rolled (its code is long
  // and run once, so it is fetched for the first tile and run for the others);
  // the terms wait in LDS.
  __syncthreads();                               // every wave has read its sums
  {
    const int n = n0 + 16 * w + c;
    const int64_t nr = n < N ? n : N - 1;
    const int r = P.r, rp = P.rp;
#pragma unroll 1
    for (int i = 0; i < MT; ++i) {
      int row_id = id[0];
#pragma unroll
      for (int k = 1; k < MT; ++k) row_id = i == k ? id[k] : row_id;
      if ((mt0 + i) % P.S != s) row_id = -1;
      const int m = 16 * (mt0 + i) + c;
      const uint16_t* trow = P.t + static_cast<int64_t>(m < P.M ? m : P.M - 1) * rp;
      red[(w * MT + i) * 64 + lane] =
          adapter_term<false, kMsBatch>(row_id, P.B, N, nr, r, lane, [&](int col, u32x4& hi, u32x4&) {
            hi = ld16(trow + (col < rp ? col : 0));
          });
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) sum[i] += red[(w * MT + i) * 64 + lane];
  }

  // with a split K: the partial sums, which the last range to arrive adds in order
  if (P.S > 1) {
    constexpr int kPart = MT * 256;              // groups of four
    const __amdgpu_buffer_rsrc_t part = part_rsrc(
        P.part + static_cast<int64_t>(nb * P.mblocks + mb) * P.S * (kPart * 4), P.S * kPart * 16);
#pragma unroll
    for (int i = 0; i < MT; ++i) put_part(part, s * kPart + i * 256 + t, sum[i]);
    if (!arrived_last(P.cnt + nb * P.mblocks + mb, P.S, t, &last_flag)) return;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      f32x4 v[kMsMaxSplit];
#pragma unroll
      for (int u = 0; u < kMsMaxSplit; ++u) v[u] = get_part(part, u * kPart + i * 256 + t);   // past S: zero
      sum[i] = v[0];
#pragma unroll
      for (int u = 1; u < kMsMaxSplit; ++u)
        if (u < P.S) sum[i] += v[u];
    }
  }
  // y: 16 MT rows x 64 columns, through LDS to whole 16-byte pieces
  const int mrows = P.M - 16 * mt0 < 16 * MT ? P.M - 16 * mt0 : 16 * MT;
  uint16_t* const yb = P.y + static_cast<int64_t>(16 * mt0) * N + n0;
  const int ncols = N - n0 < kMsRows ? N - n0 : kMsRows;
  __syncthreads();                               // every wave has read its terms
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
}

// ---------------------------------------------------------------------------
// k_mone: the forward of up to four rows in one launch. A workgroup has 64
// weight rows x one of S ranges of K, as in k_mstream (x straight from memory:
// four rows are small), and computes t = s_a x . A_a^T over its own range from the
// same x fragments, one pass per adapter among the rows. Its share of t . B^T
// joins its partial sums of y, t as two bf16 numbers (hi + lo, about 16 bits: a
// rounding of each share to one would add S roundings), so nothing waits for
// the whole of t. The last range of a row block to arrive adds them in order.
// The adapters' 2 r bytes a column are read by every row block, from L2 mostly
// (about 6 TB/s: k_mone where they are few, see multi_plan). Two launches (t,
// then k_mstream) take 17.9 us at 4096 x 4096, r 16 and one row, this one 11.0.
// What bounds it there: a chain of one load from HBM, the products, a partial
// sum and an arrival (the base alone takes 8.1).
// ---------------------------------------------------------------------------
struct MoArgs {
  const uint16_t* x;        // [M][K]
  const uint8_t* packed;
  const int8_t* qscale;
  const float* step;
  const uint16_t* A;        // [n][r][K]
  const uint16_t* B;        // [n][N][r]
  uint16_t* y;
  float* part;              // [row block][S][256 lanes x 4]
  unsigned* cnt;            // one per row block
  int M, N, K, r, S, blocks;
};

template <int RT>
__global__ __launch_bounds__(256, 2) void k_mone(MoArgs P, MultiLora ml, Codebook cb) {
  __shared__ f32x4 red[4 * kMsNT * 64];
  __shared__ f32x4 tsum[4 * RT * 64];          // the waves' parts of t, then hi and lo by row and rank
  __shared__ int flag;
  const int t = threadIdx.x, lane = t & 63;
  const int w = __builtin_amdgcn_readfirstlane(t >> 6);
  const int g = lane >> 4, c = lane & 15;
  const int N = P.N, K = P.K, r = P.r;
  // items of a row block on one XCD
  const int item = (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3);
  if (item >= P.blocks * P.S) return;
  int id = c < P.M ? ml.index[c] : -1;           // looked at once the first weights are asked for
  const int s = item % P.S, nb = item / P.S;
  const int nbr = K / 64, nss = (nbr + 3) / 4;
  const int ss0 = static_cast<int>(static_cast<int64_t>(nss) * s / P.S);
  const int ss1 = static_cast<int>(static_cast<int64_t>(nss) * (s + 1) / P.S);
  const __amdgpu_buffer_rsrc_t xr =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(P.x), 0, P.M * K * 2, 0x00020000);
  const uint8_t* crow[kMsNT];
  int64_t brow[kMsNT];
#pragma unroll
  for (int nt = 0; nt < kMsNT; ++nt) {
    const int n = nb * kMsRows + 16 * nt + c < N ? nb * kMsRows + 16 * nt + c : N - 1;
    crow[nt] = P.packed + static_cast<int64_t>(n) * (K / 2);
    brow[nt] = static_cast<int64_t>(n) * nbr;
  }
  struct Step {                                // one super-step's operands
    u32x4 cw[kMsNT][2];
    u32x4 x[8];
    int8_t q[kMsNT];
    float d[kMsNT];
  };
  auto load = [&](int ss, Step& C) {
    const bool live = ss * 4 + g < nbr;          // past K: x reads as zero
    const int kb = live ? ss * 4 + g : nbr - 1;
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
    const uint32_t off = live ? static_cast<uint32_t>((c * K + kb * 64) * 2) : 0x80000000u;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      C.x[j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(xr, off + 16 * j, 0, 0));
  };
  // rank 16 jt + c of adapter a, block 4 ss + g; a rank past r repeats rank 0
  // (its t is not used), a block past K is zero
  auto load_a = [&](int a, int jt, int ss, u32x4 (&f)[8]) {
    const int kb = ss * 4 + g < nbr ? ss * 4 + g : 0, j = 16 * jt + c < r ? 16 * jt + c : 0;
    const uint16_t* p = P.A + (static_cast<int64_t>(a) * r + j) * K + kb * 64;
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = ld16(p + 8 * i);
  };
  f32x4 acc[kMsNT], tacc[RT];
#pragma unroll
  for (int nt = 0; nt < kMsNT; ++nt) acc[nt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int jt = 0; jt < RT; ++jt) tacc[jt] = f32x4{0.f, 0.f, 0.f, 0.f};
  Step cur, nxt;
  int ss = ss0 + w;
  load(ss < ss1 ? ss : ss0, cur);
  __builtin_amdgcn_sched_barrier(0);
  if (static_cast<unsigned>(id) >= static_cast<unsigned>(ml.n)) id = -1;
  const uint32_t any = static_cast<uint32_t>(__ballot(id >= 0)) & 0xFFFFu;
  const int first = any ? __builtin_amdgcn_readlane(id, __builtin_ctz(any)) : 0;
  // the end's operands of the first adapter, brought near: nothing covers
  // their latency there
  const int n = nb * kMsRows + 16 * w + c;
  const float scale0 = ml.scale[first];
  uint32_t near = 0;
  if (any) near = P.B[(static_cast<int64_t>(first) * N + (n < N ? n : N - 1)) * r];
  {
    for (; ss < ss1; ss += 4) {
      const bool more = ss + 4 < ss1;
      const uint32_t kv = ss * 4 + g < nbr ? 0xFFFFFFFFu : 0u;
      const u32x4 live = {kv, kv, kv, kv};
      u32x4 af[8];
      __builtin_amdgcn_sched_barrier(0);
      if (any) load_a(first, 0, ss, af);         // used after the weights
      if (more) load(ss + 4, nxt);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < 8; ++j) cur.x[j] = perm8(cur.x[j]);
#pragma unroll
      for (int nt = 0; nt < kMsNT; ++nt) {
        const MagTable tb = make_table(cb, block_scale(cur.q[nt], cur.d[nt]));
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const u32x4 cw = cur.cw[nt][j >> 2];
          const uint32_t d = (j & 3) == 0 ? cw.x : (j & 3) == 1 ? cw.y : (j & 3) == 2 ? cw.z : cw.w;
          acc[nt] = mfma16(as_bf16x8(cur.x[j]), as_bf16x8(decode8_perm(d, tb)), acc[nt]);
        }
      }
      // t: every adapter's product with all rows; a row takes its own
      // adapter's, after the product
      for (uint32_t pend = any; pend;) {
        const int a = __builtin_amdgcn_readlane(id, __builtin_ctz(pend));
        const uint32_t rows = static_cast<uint32_t>(__ballot(id == a)) & 0xFFFFu;
#pragma unroll
        for (int jt = 0; jt < RT; ++jt) {
          if (jt > 0 || pend != any) load_a(a, jt, ss, af);
          f32x4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < 8; ++j) p = mfma16(as_bf16x8(cur.x[j]), as_bf16x8(perm8(af[j] & live)), p);
#pragma unroll
          for (int v = 0; v < 4; ++v) tacc[jt][v] += (rows >> (4 * g + v)) & 1u ? p[v] : 0.f;
        }
        pend &= ~rows;
      }
      if (more) cur = nxt;
    }
  }
#pragma unroll
  for (int nt = 0; nt < kMsNT; ++nt) red[(w * kMsNT + nt) * 64 + lane] = acc[nt];
#pragma unroll
  for (int jt = 0; jt < RT; ++jt) tsum[(w * RT + jt) * 64 + lane] = tacc[jt];
  __syncthreads();
  f32x4 sum = red[w * 64 + lane];
#pragma unroll
  for (int ww = 1; ww < 4; ++ww) sum += red[(ww * kMsNT + w) * 64 + lane];
  asm volatile("" ::"v"(near));
  if (any) {
    // t of row c from rank col: the waves' parts in order, times the row's scale
    const float scale = id < 0 ? 0.f : id == first ? scale0 : ml.scale[id];
    sum += adapter_term<true, static_cast<int>(kMoMaxM)>(id, P.B, N, n < N ? n : N - 1, r, lane, [&](int col, u32x4& hi, u32x4& lo) {
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int j = col + e;
        float a = 0.f;
        if (j < r) {
          const int at = (j >> 4) * 64 + ((c >> 2) << 4) + (j & 15);
          a = tsum[at][c & 3];
#pragma unroll
          for (int ww = 1; ww < 4; ++ww) a += tsum[ww * RT * 64 + at][c & 3];
          a *= scale;
        }
        v[e] = a;
      }
      hi = u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
      auto low = [&](int e, uint32_t h) {
        return pack_bf16x2(rest_of(v[e], bf16_lo(h)), rest_of(v[e + 1], bf16_hi(h)));
      };
      lo = u32x4{low(0, hi.x), low(2, hi.y), low(4, hi.z), low(6, hi.w)};
    });
  }
  if (P.S > 1) {
    const __amdgpu_buffer_rsrc_t part = part_rsrc(P.part + static_cast<int64_t>(nb) * P.S * 1024, P.S * 4096);
    put_part(part, s * 256 + t, sum);
    if (!arrived_last(P.cnt + nb, P.S, t, &flag)) return;
    f32x4 v[kMsMaxSplit];
#pragma unroll
    for (int u = 0; u < kMsMaxSplit; ++u) v[u] = get_part(part, u * 256 + t);      // past S: out of range, zero
    sum = v[0];
#pragma unroll
    for (int u = 1; u < kMsMaxSplit; ++u)
      if (u < P.S) sum += v[u];
  }
  if (n < N) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (4 * g + q < P.M) P.y[static_cast<int64_t>(4 * g + q) * N + n] = bf16_bits(sum[q]);
  }
}

}  // namespace

// Items: blocks of 64 weight rows x blocks of 16 MT rows of x (MT up to 4) x S
// ranges of K. S is the most that gives every CU at most one item and every
// wave a super-step (11008 x 4096, ranges 1 / 2 / 4: 16 rows 16.9 / 19.2 / 19.5
// us, 48 rows 20.8 / 27.5 / 30.9; 4096 x 4096, 32 rows 16.5 / 13.9 / 12.5).
MsPlan ms_plan(int64_t M, int64_t N, int64_t K, int r, int n) {
  MsPlan p;
  const int64_t mtiles = cdiv(M, 16), nss = cdiv(K, 256);
  p.MT = static_cast<int>(mtiles < 4 ? mtiles : 4);
  p.mblocks = cdiv(mtiles, p.MT);
  const int64_t blocks = cdiv(N, kMsRows) * p.mblocks;
  int64_t S = 256 / blocks;
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

MoPlan mo_plan(int64_t M, int64_t N, int64_t K) {
  MoPlan p;
  const int64_t nss = cdiv(K, 256);
  p.blocks = cdiv(N, kMsRows);
  // as ms_plan, with two items per CU (11008 x 4096: 22.3 us in one range, 21.5 in two)
  p.S = std::max<int64_t>(std::min({512 / p.blocks, cdiv(nss, 4), int64_t{kMsMaxSplit}}), 1);
  if (p.S > 1) p.part_bytes = static_cast<size_t>(p.blocks * p.S) * 4096;
  return p;
}

hipError_t launch_mone(const MoPlan& p, const uint16_t* x, int64_t M, int64_t N, int64_t K, const uint8_t* packed,
                       const int8_t* qscale, const float* step, const uint16_t* A, const uint16_t* B,
                       const MultiLora& ml, int r, uint16_t* y, void* ws, const Codebook& cb, hipStream_t stream) {
  char* wsb = static_cast<char*>(ws);
  MoArgs a{};
  a.x = x;
  a.packed = packed;
  a.qscale = qscale;
  a.step = step;
  a.A = A;
  a.B = B;
  a.y = y;
  a.part = reinterpret_cast<float*>(wsb + kWsCounterBytes);
  a.cnt = reinterpret_cast<unsigned*>(wsb);
  a.M = static_cast<int>(M);
  a.N = static_cast<int>(N);
  a.K = static_cast<int>(K);
  a.r = r;
  a.S = static_cast<int>(p.S);
  a.blocks = static_cast<int>(p.blocks);
  const dim3 grid(static_cast<unsigned>(round_up(p.blocks * p.S, 8)));
  mark_kernel(0, stream);
  switch (down_nt(r)) {
    case 1: hipLaunchKernelGGL(HIP_KERNEL_NAME(k_mone<1>), grid, dim3(256), 0, stream, a, ml, cb); break;
    case 2: hipLaunchKernelGGL(HIP_KERNEL_NAME(k_mone<2>), grid, dim3(256), 0, stream, a, ml, cb); break;
    case 4: hipLaunchKernelGGL(HIP_KERNEL_NAME(k_mone<4>), grid, dim3(256), 0, stream, a, ml, cb); break;
    default: hipLaunchKernelGGL(HIP_KERNEL_NAME(k_mone<8>), grid, dim3(256), 0, stream, a, ml, cb); break;
  }
  mark_kernel(1, stream);
  return hipGetLastError();
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
