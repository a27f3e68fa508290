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
//          backward GEMMs: 16 or 64 rows per workgroup, one pass per adapter
//          among them; beside it, x in MFMA order for the streaming forward.
// The gradients list each adapter's rows (the rows of an adapter in batch order,
// padded to whole chunks of 64 places), so that every product has one adapter
// per chunk and needs no masks:
// k_gdown  t and u over the listed rows, transposed, as three bf16 numbers
//          that sum to the fp32 value (hi + mid + lo: fp32 gradients want more
//          than one bf16 rounding of t and u; two would leave 2e-6). Up to 8192
//          rows each workgroup finds its chunk's rows itself; above, k_msort
//          lists them first.
// k_mgrad  G = P^T . Q over the rows of one item (a run of chunks of one
//          adapter), P = dY or x gathered by row, Q = t or u. An adapter's only
//          item writes its gradient; with more, the last item to arrive sums
//          all of them in order. Workgroups without an item clear the
//          gradients of adapters without rows.
// Results do not depend on scheduling: no atomic touches a sum.
//
// What bounds the gradients: x and dY are each read twice (t and u need whole
// rows before any column of dA or dB can use them), the second time mostly from
// the last-level cache.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "act8.hpp"
#include "down.hpp"
#include "multi.hpp"

namespace qnf4 {

constexpr int kSplit = 3;                      // bf16 numbers that carry one fp32 value of t or u

struct MdArgs {
  const uint16_t* in;       // [M][Kc]
  const uint16_t* W;        // [n][r Kc]
  uint16_t* out;            // [M][rp]
  float* part;              // [blocks][Smax][16 RT x 16 RM]
  unsigned* cnt;
  u32x4* frags;
  int64_t M, nfrag;
  int Kc, r, rp, blocks, Q, Smax;
};

// s_a t (kBT false: in = x, W = A) or s_a u (kBT true: in = dY, W = B), rounded
// to bf16 once, [M][rp] with the ranks past r zero; rows without an adapter are
// not written. (One bf16 number each, as for a single adapter: the output is
// bf16 itself. The scale goes in before the rounding, so that the GEMMs need
// no scale.) A row block of 16 RM rows has Q workgroups. They share its passes,
// one for each of the D adapters among its rows (mostly one: rows of a request
// follow each other), and, where there are more workgroups than passes, split
// the contraction into S = Q / D ranges: those leave partial sums, and the last
// workgroup of the block adds them in order.
// Workgroups past those copy x into MFMA order: fragment (tile, ss, j) has, at
// lane (g, c), columns 256 ss + 64 g + 8 j + (0 2 | 4 6 | 1 3 | 5 7) of row 16
// tile + c, zero past M and Kc.
template <int RM, int RT, bool kBT>
__global__ __launch_bounds__(64 * kMdWaves) void k_mdown(MdArgs P, MultiLora ml) {
  const int t = threadIdx.x, lane = t & 63;
  const int w = __builtin_amdgcn_readfirstlane(t >> 6);
  const int c = lane & 15;
  const int Kc = P.Kc, r = P.r, rp = P.rp;
  const int wgs = P.blocks * P.Q;
  if (static_cast<int>(blockIdx.x) >= wgs) {
    if constexpr (!kBT) {
      const int nss = (Kc + 255) / 256;
      const int64_t f = static_cast<int64_t>(blockIdx.x - wgs) * kMdWaves + w;
      if (f >= P.nfrag) return;
      const int64_t tile = f / (8 * nss);
      const int rest = static_cast<int>(f - tile * 8 * nss);
      const int64_t m = 16 * tile + c;
      const int k = 256 * (rest >> 3) + 64 * (lane >> 4) + 8 * (rest & 7);
      u32x4 v = {0u, 0u, 0u, 0u};
      if (m < P.M && k < Kc) v = perm8(ld16(P.in + m * Kc + k));
      P.frags[f * 64 + lane] = v;
    }
    return;
  }
  __shared__ u32x4 lds[md_lds<RM, RT, kBT>()];
  __shared__ int flag;
  const int block = blockIdx.x / P.Q, q = blockIdx.x % P.Q;
  const int64_t m0 = static_cast<int64_t>(block) * 16 * RM;
  // the rows' adapters: row lane of the block (RM == 1: lanes 0 .. 15)
  int id = lane < 16 * RM && m0 + lane < P.M ? ml.index[m0 + lane] : -1;
  if (static_cast<unsigned>(id) >= static_cast<unsigned>(ml.n)) id = -1;
  const uint64_t any = __ballot(id >= 0);
  if (!any) return;                              // the whole row block: nobody counts
  int D = 0;
  for (uint64_t pend = any; pend; ++D) pend &= ~__ballot(id == __builtin_amdgcn_readlane(id, __builtin_ctzll(pend)));
  int S = P.Q / D < P.Smax ? P.Q / D : P.Smax;
  if (S < 1) S = 1;
  // ranges: workgroup q has range q % S of pass q / S; one range: passes q, q + Q, ...
  const bool direct = S == 1;
  const int y = direct ? q : q / S, step = direct ? P.Q : D, s = direct ? 0 : q % S;
  const int nchunk = (Kc + 63) / 64;
  const int qb = static_cast<int>(static_cast<int64_t>(nchunk) * s / S);
  const int qe = static_cast<int>(static_cast<int64_t>(nchunk) * (s + 1) / S);
  uint64_t pend = any;
  constexpr int kCount = RM * RT * 64;           // groups of four partial sums
  const __amdgpu_buffer_rsrc_t part =
      part_rsrc(P.part + static_cast<int64_t>(block) * P.Smax * kCount * 4, S * kCount * 16);
  f32x4* const red = reinterpret_cast<f32x4*>(lds);
  constexpr int kPerWave = md_lds<RM, RT, kBT>() / kMdWaves;
  for (int ord = 0; pend; ++ord) {
    const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(pend));
    const uint64_t mine = __ballot(id == a);
    pend &= ~mine;
    if (ord % step != y) continue;
    int64_t rows[RM];
#pragma unroll
    for (int i = 0; i < RM; ++i) rows[i] = (mine >> (16 * i + c)) & 1 ? m0 + 16 * i + c : -1;
    f32x4 acc[RM][md_rtw<RT>()];
    const uint16_t* Wa = P.W + static_cast<int64_t>(a) * r * Kc;
    if (!kBT || (r & 7) == 0)
      down_acc<RM, RT, kBT, kActBf16, true>(P.in, nullptr, rows, Kc, qb, qe, 5 * block, Wa, r, lds + w * kPerWave, acc, w, lane);
    else
      down_acc<RM, RT, kBT, kActBf16, false>(P.in, nullptr, rows, Kc, qb, qe, 5 * block, Wa, r, lds + w * kPerWave, acc, w, lane);
    const float scale = ml.scale[a];
    down_sum<RM, RT>(red, acc, t, w, lane, [&](int place, int row, int j, f32x4 v) {
      v *= scale;
      if (!direct) {
        // the block's partials are written once for all its passes: rows of
        // other adapters keep what their pass left
        if (any == mine) put_part(part, s * kCount + place, v);
        else
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if ((mine >> (row + q)) & 1)
              __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, static_cast<float>(v[q])), part,
                                                    static_cast<uint32_t>((s * kCount + place) * 16 + 4 * q), 0, 16);
        return;
      }
      if (j >= rp) return;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if ((mine >> (row + q)) & 1) P.out[(m0 + row + q) * rp + j] = j < r ? bf16_bits(v[q]) : uint16_t{0};
    });
    if (direct && 16 * RT < rp)                  // r <= 16: t has 32 columns
      for (int e = t; e < 16 * RM * (rp - 16 * RT); e += 64 * kMdWaves) {
        const int row = e / (rp - 16 * RT), j = 16 * RT + e % (rp - 16 * RT);
        if ((mine >> row) & 1) P.out[(m0 + row) * rp + j] = 0;
      }
    __syncthreads();
  }
  if (direct) return;
  if (!arrived_last(P.cnt + block, P.Q, t, &flag)) return;
  sum_partials<RM, RT>(part, S, t, [&](int, int row, int j, const f32x4& v) {
    if (j >= rp) return;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if ((any >> (row + q)) & 1) P.out[(m0 + row + q) * rp + j] = j < r ? bf16_bits(v[q]) : uint16_t{0};
  });
  for (int e = t; e < 16 * RM * (rp - 16 * RT); e += 64 * kMdWaves) {
    const int row = e / (rp - 16 * RT), j = 16 * RT + e % (rp - 16 * RT);
    if ((any >> row) & 1) P.out[(m0 + row) * rp + j] = 0;
  }
}

// ---------------------------------------------------------------------------
// gradients
// ---------------------------------------------------------------------------
namespace {

constexpr int kGdThreads = 64 * kMdWaves;
constexpr int kFindPer = kFindMaxM / kGdThreads;           // rows per thread
constexpr int kAdPer = kMaxAdapters / kGdThreads;          // adapters per thread

// counts the rows of every adapter; a wave whose rows agree adds once
__device__ __forceinline__ void count_rows(int id, int n, int lane, int* hist) {
  const int first = __builtin_amdgcn_readfirstlane(id);
  const uint64_t live = __ballot(true);
  if (__ballot(id == first) == live) {
    if (static_cast<unsigned>(first) < static_cast<unsigned>(n) && lane == __builtin_ctzll(live))
      atomicAdd(&hist[first], __builtin_popcountll(live));
  } else if (static_cast<unsigned>(id) < static_cast<unsigned>(n)) {
    atomicAdd(&hist[id], 1);
  }
}

__device__ __forceinline__ int chunks_of(int rows) { return (rows + 63) >> 6; }
__device__ __forceinline__ int items_of(int chunks, int per) { return (chunks + per - 1) / per; }

// the tables of adapter a, whose chunks, items and slots start at the given numbers
__device__ __forceinline__ void put_adapter(const GradLists& L, int a, int rows, int per, int chunk, int item, int slot) {
  const int ch = chunks_of(rows), it = items_of(ch, per);
  L.adapter[a] = GradAdapter{it, slot};
  for (int i = 0; i < it; ++i) {
    const int c0 = i * per, c1 = c0 + per;
    L.item[item + i] = GradItem{a, chunk + c0, chunk + (c1 < ch ? c1 : ch), it > 1 ? slot + i : -1, it, it > 1 ? slot : -1};
  }
}

// Finds chunk `chunk` of the batch: its adapter, and the rows at its 64 places
// in `out` (-1 where there is none). Every workgroup counts the whole batch.
// The workgroup with `tables` also writes the lists that k_mgrad reads. Returns
// the adapter, or -1 past the last chunk. scratch: kMaxAdapters + 64 integers.
__device__ int find_chunk(const int* __restrict__ index, int M, int n, int per, int chunk, bool tables,
                          const GradLists& L, int* scratch, int* out, int t) {
  int* const hist = scratch;
  int* const sums = scratch + kMaxAdapters;                // [3][8] sums of the waves, then the place found
  const int lane = t & 63, w = t >> 6;
  // wave w has rows [w share, (w + 1) share): in order, 64 at a time
  const int share = ((M + kMdWaves - 1) / kMdWaves + 63) & ~63;
  int id[kFindPer];
#pragma unroll
  for (int i = 0; i < kFindPer; ++i) {
    const int m = w * share + 64 * i + lane;
    id[i] = 64 * i < share && m < M ? index[m] : -1;
  }
  for (int i = t; i < n; i += kGdThreads) hist[i] = 0;
  if (t < 64) out[t] = -1;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kFindPer; ++i)
    if (64 * i < share) count_rows(id[i], n, lane, hist);
  __syncthreads();
  // chunks, items and slots before this thread's adapters (kAdPer in a row)
  const int per_thread = (n + kGdThreads - 1) / kGdThreads;
  int own[3] = {0, 0, 0};
#pragma unroll
  for (int i = 0; i < kAdPer; ++i) {
    const int a = t * per_thread + i;
    if (i < per_thread && a < n) {
      const int ch = chunks_of(hist[a]), it = items_of(ch, per);
      own[0] += ch;
      own[1] += it;
      own[2] += it > 1 ? it : 0;
    }
  }
  int pre[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    pre[k] = own[k];
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(pre[k], o);
      if (lane >= o) pre[k] += v;
    }
    if (lane == 63) sums[8 * k + w] = pre[k];
    pre[k] -= own[k];
  }
  if (t == 0) sums[24] = -1;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 3; ++k)
    for (int ww = 0; ww < w; ++ww) pre[k] += sums[8 * k + ww];
  for (int i = 0; i < per_thread; ++i) {
    const int a = t * per_thread + i;
    if (a >= n) break;
    const int ch = chunks_of(hist[a]), it = items_of(ch, per);
    if (chunk >= pre[0] && chunk < pre[0] + ch) {
      sums[24] = a;
      sums[25] = chunk - pre[0];
    }
    if (tables) {
      put_adapter(L, a, hist[a], per, pre[0], pre[1], pre[2]);
      if (a == n - 1) {
        L.total[0] = pre[0] + ch;
        L.total[1] = pre[1] + it;
      }
    }
    pre[0] += ch;
    pre[1] += it;
    pre[2] += it > 1 ? it : 0;
  }
  __syncthreads();
  const int a = sums[24];
  if (a < 0) return -1;
  // the adapter's rows, in batch order: places [64 k, 64 k + 64) of them
  const int first = 64 * sums[25];
  int mine = 0;
#pragma unroll
  for (int i = 0; i < kFindPer; ++i) mine += 64 * i < share ? __builtin_popcountll(__ballot(id[i] == a)) : 0;
  __syncthreads();
  if (lane == 0) sums[w] = mine;
  __syncthreads();
  int pos = -first;
  for (int ww = 0; ww < w; ++ww) pos += sums[ww];
#pragma unroll
  for (int i = 0; i < kFindPer; ++i) {
    if (64 * i >= share) break;
    const uint64_t hit = __ballot(id[i] == a);
    const int p = pos + __builtin_popcountll(hit & ((1ull << lane) - 1));
    if (id[i] == a && p >= 0 && p < 64) out[p] = w * share + 64 * i + lane;
    pos += __builtin_popcountll(hit);
  }
  __syncthreads();
  return a;
}

}  // namespace

// The lists of a batch above kFindMaxM rows, one wave per adapter: every
// workgroup counts the whole batch, then each wave places its adapter's
// chunks, items and rows after those of the adapters before it.
__global__ __launch_bounds__(256) void k_msort(const int* __restrict__ index, int64_t M, int n, int per, GradLists L) {
  __shared__ int hist[kMaxAdapters];
  const int t = threadIdx.x, lane = t & 63;
  const int w = __builtin_amdgcn_readfirstlane(t >> 6);
  for (int i = t; i < n; i += 256) hist[i] = 0;
  __syncthreads();
  for (int64_t m = t; m < M; m += 256) count_rows(index[m], n, lane, hist);
  __syncthreads();
  const int a = blockIdx.x * 4 + w;
  if (a >= n) return;
  int chunks = 0, items = 0, slots = 0;
  for (int b = lane; b < a; b += 64) {
    const int ch = chunks_of(hist[b]), it = items_of(ch, per);
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
  const int nch = chunks_of(hist[a]);
  if (lane == 0) {
    put_adapter(L, a, hist[a], per, chunks, items, slots);
    if (a == n - 1) {
      L.total[0] = chunks + nch;
      L.total[1] = items + items_of(nch, per);
    }
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

// four values of t or u (places row .. row + 3 of a chunk, rank j) as three bf16
// numbers each, the rounded value and what is left of it twice:
// [chunk][3][16 RT][64], a chunk in one piece (ranks at a stride of a whole row
// length would share one memory channel)
template <int RT>
__device__ __forceinline__ void put_split(uint16_t* qt, int64_t chunk, int row, int j, f32x4 v) {
#pragma unroll
  for (int k = 0; k < kSplit; ++k) {
    u32x2 b;
    b.x = pack_bf16x2(v[0], v[1]);
    b.y = pack_bf16x2(v[2], v[3]);
    *reinterpret_cast<u32x2*>(qt + ((chunk * kSplit + k) * 16 * RT + j) * 64 + row) = b;
    v = rest_of(v, f32x4{bf16_lo(b.x), bf16_hi(b.x), bf16_lo(b.y), bf16_hi(b.y)});
  }
}

// how k_gdown knows a chunk's rows: it finds them, k_msort has listed them, or
// there is one adapter and they are the batch's own
constexpr int kGdFind = 0, kGdListed = 1, kGdWhole = 2;

struct GdArgs {
  const void* x;            // [M][K], or its checkpoint's codes
  const uint16_t* tops;
  const uint16_t* dy;       // [M][N]
  const uint16_t* A;        // [n][r][K]
  const uint16_t* B;        // [n][N][r]
  const int* index;         // [M]
  uint16_t *tt, *ut;        // [chunk][3][16 RT][64]
  float* part;              // [chunk][t, u][kMdMaxSplit][16 RT x 64]
  unsigned* cnt;            // [chunk][t, u]
  unsigned* cnt2;           // k_mgrad's, cleared here: ncnt2
  int64_t M;
  int N, K, r, n, per, St, Su, ncnt2;
  int mode;
};

// t^T (the first St workgroups of a chunk) and u^T (the other Su) of its 64
// places, each over one range of the contraction
template <int RT, int XF>
__global__ __launch_bounds__(kGdThreads) void k_gdown(GdArgs P, GradLists L) {
  constexpr int kLds0 = md_lds<4, RT, true>() > md_lds<4, RT, false>() ? md_lds<4, RT, true>() : md_lds<4, RT, false>();
  constexpr int kLds = kLds0 * 4 > kMaxAdapters + 64 ? kLds0 : (kMaxAdapters + 64) / 4;
  __shared__ u32x4 lds[kLds];
  __shared__ int flag;
  __shared__ int place[64];
  const int t = threadIdx.x, lane = t & 63;
  const int w = __builtin_amdgcn_readfirstlane(t >> 6);
  const int per_chunk = P.St + P.Su;
  const int chunk = blockIdx.x / per_chunk, part_no = blockIdx.x - chunk * per_chunk;
  const bool is_u = part_no >= P.St;
  const int s = is_u ? part_no - P.St : part_no, S = is_u ? P.Su : P.St;
  if (blockIdx.x == 0)
    for (int i = t; i < P.ncnt2; i += kGdThreads) P.cnt2[i] = 0;
  const int64_t p0 = static_cast<int64_t>(chunk) * 64;
  int64_t a = 0;
  if (P.mode == kGdFind) {
    a = find_chunk(P.index, static_cast<int>(P.M), P.n, P.per, chunk, blockIdx.x == 0, L, reinterpret_cast<int*>(lds),
                   place, t);
    if (a < 0) return;
  } else if (P.mode == kGdListed) {
    if (chunk >= L.total[0]) return;
    a = L.chunk_adapter[chunk];
    if (t < 64) place[t] = L.rows[p0 + t];
    __syncthreads();
  } else {
    if (t < 64) place[t] = p0 + t < P.M ? static_cast<int>(p0 + t) : -1;
    __syncthreads();
  }
  if (P.mode != kGdListed && part_no == 0 && t < 64) L.rows[p0 + t] = place[t];
  a = __builtin_amdgcn_readfirstlane(static_cast<int>(a));
  int64_t rows[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) rows[i] = place[16 * i + (lane & 15)];
  const uint64_t live = __ballot(place[lane] >= 0);        // the places that hold a row
  const int Kc = is_u ? P.N : P.K, nchunk = (Kc + 63) / 64;
  const int qb = static_cast<int>(static_cast<int64_t>(nchunk) * s / S);
  const int qe = static_cast<int>(static_cast<int64_t>(nchunk) * (s + 1) / S);
  f32x4 acc[4][md_rtw<RT>()];
  f32x4* const red = reinterpret_cast<f32x4*>(lds);
  if (is_u) {
    u32x4* const mine = lds + w * (md_lds<4, RT, true>() / kMdWaves);
    if ((P.r & 7) == 0)
      down_acc<4, RT, true, kActBf16, true>(P.dy, nullptr, rows, P.N, qb, qe, 5 * chunk, P.B + a * P.N * P.r, P.r, mine, acc, w, lane);
    else
      down_acc<4, RT, true, kActBf16, false>(P.dy, nullptr, rows, P.N, qb, qe, 5 * chunk, P.B + a * P.N * P.r, P.r, mine, acc, w, lane);
  } else {
    down_acc<4, RT, false, XF, true>(P.x, P.tops, rows, P.K, qb, qe, 5 * chunk, P.A + a * P.r * P.K, P.r, lds, acc, w, lane);
  }
  uint16_t* const out = is_u ? P.ut : P.tt;
  // places without a row hold zeros
  auto put = [&](int, int row, int j, f32x4 v) {
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = (live >> (row + q)) & 1 ? v[q] : 0.f;
    put_split<RT>(out, chunk, row, j, v);
  };
  if (S == 1) {
    down_sum<4, RT>(red, acc, t, w, lane, put);
    return;
  }
  constexpr int kCount = 4 * RT * 64;
  const int slot = 2 * chunk + (is_u ? 1 : 0);
  const __amdgpu_buffer_rsrc_t part =
      part_rsrc(P.part + static_cast<int64_t>(slot) * kMdMaxSplit * kCount * 4, S * kCount * 16);
  down_sum<4, RT>(red, acc, t, w, lane, [&](int place, int, int, const f32x4& v) { put_part(part, s * kCount + place, v); });
  if (!arrived_last(P.cnt + slot, S, t, &flag)) return;
  sum_partials<4, RT>(part, S, t, put);
}

namespace {

constexpr int kGThreads = 256;
constexpr int kGCols = 256;                    // columns of P per workgroup (64 per wave)

// two LDS buffers of P and Q where one workgroup fills a CU anyway
template <int NT>
constexpr bool mg_two() { return NT >= 4; }

// P tile in LDS: four quarters of 64 rows x 64 columns, chunk c of row m at
// c ^ 2 f(m), f(m) = ((m >> 3) & 3) ^ ((m >> 1) & 1), so that a transposed read
// of 4 rows at offsets 8 G + 4 q touches each bank twice (as in grad.hip)
__device__ __forceinline__ int g_swz(int m) { return 2 * (((m >> 3) & 3) ^ ((m >> 1) & 1)); }

struct MgArgs {
  const void* x;            // [M][K], or its checkpoint's codes
  const uint16_t* tops;
  const uint16_t* dy;       // [M][N]
  const uint16_t *tt, *ut;  // [chunk][3][16 NT][64]
  const float* scale;       // [n], or null: alpha_r
  float* part;              // [slot][column tile][256 columns x 16 NT ranks]
  float *dA, *dB;
  unsigned* cnt2;           // [first slot of an adapter][column tile]
  int64_t M;
  float alpha_r;
  int N, K, r, n, ctb, per, chunks, accumulate;
};

// One item of one 256-column tile. kTR: dA (P = x, out [r][C]); else dB
// (P = dY, out [C][r]). Four waves of 64 columns share the 64 rows of a chunk
// and its Q; the loads of the next two chunks are in flight while one is
// multiplied. At high ranks the LDS reads of Q bound the kernel (three numbers
// a value, read by every wave), so a wave multiplies each fragment with four
// column tiles.
template <int NT, bool kTR, int XF>
__device__ __forceinline__ void grad_item(const MgArgs& A, const GradItem& it, const GradLists& L, int ct, u32x4* tiles,
                                          u32x4* qtiles) {
  constexpr int kQ = kSplit * 16 * NT * 8;     // 16-byte pieces of Q per chunk
  constexpr int kQPer = (kQ + kGThreads - 1) / kGThreads;
  constexpr int kPer = XF == kActBf16 ? 8 : 4; // 16-byte loads of P per thread and chunk
  constexpr int kRow = XF == kActBf16 ? 32 : 16;            // lanes per row
  const int C = kTR ? A.K : A.N, r = A.r;
  const void* const P = kTR ? A.x : static_cast<const void*>(A.dy);
  const uint16_t* const Qt = kTR ? A.ut : A.tt;
  const int t = threadIdx.x, lane = t & 63;
  const int w = __builtin_amdgcn_readfirstlane(t >> 6);
  const int G = lane >> 4, j16 = lane & 15;
  const int c0 = ct * kGCols;
  const u32x4 zero = {0u, 0u, 0u, 0u};
  // this thread's loads of a chunk: rows lr + (256 / kRow) i, from column col
  const int lr = t / kRow, lc = t % kRow;
  constexpr int kCols = XF == kActBf16 ? 8 : 16;
  const int col = c0 + kCols * lc < C ? c0 + kCols * lc : 0;
  struct Regs {
    u32x4 p[kPer];
    uint32_t top[XF == kActBf16 ? 1 : kPer];
    u32x4 q[kQPer];
    uint32_t live;
  };
  auto rows_of = [&](int ch, int (&rows)[kPer]) {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      rows[i] = L.rows[static_cast<int64_t>(ch) * 64 + lr + kGThreads / kRow * i];
  };
  auto load = [&](int ch, const int (&rows)[kPer], Regs& R) {
    R.live = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int64_t row = rows[i] < 0 ? 0 : rows[i];
      R.live |= rows[i] < 0 ? 0u : 1u << i;
      if constexpr (XF == kActBf16) {
        R.p[i] = ld16(static_cast<const uint16_t*>(P) + row * C + col);
      } else {
        R.p[i] = ld16(static_cast<const uint8_t*>(P) + row * C + col);
        R.top[i] = A.tops[row * (C / 64) + (col >> 6)];
      }
    }
#pragma unroll
    for (int i = 0; i < kQPer; ++i) {
      const int e = t + kGThreads * i;
      if (kQ % kGThreads == 0 || e < kQ)
        R.q[i] = ld16(Qt + (static_cast<int64_t>(ch) * kQ + e) * 8);
    }
  };
  constexpr bool kTwo = mg_two<NT>();
  auto store = [&](const Regs& R, int buf) {
    u32x4* const tile = tiles + (kTwo ? buf * 2048 : 0);
    u32x4* const qtile = qtiles + (kTwo ? buf * kQ : 0);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int m = lr + kGThreads / kRow * i;
      const bool live = (R.live >> i) & 1;     // a place without a row: zeros, whatever row 0 holds
      if constexpr (XF == kActBf16) {
        tile[(lc >> 3) * 512 + m * 8 + ((lc & 7) ^ g_swz(m))] = live ? R.p[i] : zero;
      } else {
        const float s = act8_scale<XF>(R.top[i]);
        const int q = lc >> 2, ch = 2 * (lc & 3);
        const u32x4 v0 = act8_decode8<XF>(u32x2{R.p[i].x, R.p[i].y}, s);
        const u32x4 v1 = act8_decode8<XF>(u32x2{R.p[i].z, R.p[i].w}, s);
        tile[q * 512 + m * 8 + (ch ^ g_swz(m))] = live ? v0 : zero;
        tile[q * 512 + m * 8 + ((ch + 1) ^ g_swz(m))] = live ? v1 : zero;
      }
    }
#pragma unroll
    for (int i = 0; i < kQPer; ++i) {
      const int e = t + kGThreads * i, rank = e >> 3;
      if (kQ % kGThreads == 0 || e < kQ) qtile[rank * 8 + ((e & 7) ^ ((rank >> 1) & 7))] = R.q[i];
    }
  };
  f32x4 acc[4][NT];
#pragma unroll
  for (int b = 0; b < 4; ++b)
#pragma unroll
    for (int jt = 0; jt < NT; ++jt) acc[b][jt] = f32x4{0.f, 0.f, 0.f, 0.f};
  // operands of a 32-row half kk of the chunk: four column tiles of P, all of Q
  struct Frags {
    bf16x8 p[4], q[kSplit * NT];
  };
  auto read = [&](int buf, int kk, Frags& F) {
    const u32x4* T = tiles + (kTwo ? buf * 2048 : 0) + w * 512;
    const u32x4* const qtile = qtiles + (kTwo ? buf * kQ : 0);
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      s16x4 v[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int m = 32 * kk + 8 * G + 4 * q + (j16 >> 2);
        const int cc = 16 * b + 4 * (j16 & 3);
        v[q] = ds_read_tr(T, (m * 8 + ((cc >> 3) ^ g_swz(m))) * 8 + (cc & 7));
      }
      F.p[b] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7));
    }
#pragma unroll
    for (int i = 0; i < kSplit * NT; ++i) {
      const int rank = 16 * i + j16;           // of the 3 x 16 NT
      F.q[i] = as_bf16x8(qtile[rank * 8 + ((4 * kk + G) ^ ((rank >> 1) & 7))]);
    }
  };
  auto multiply = [&](const Frags& F) {
#pragma unroll
    for (int i = 0; i < kSplit * NT; ++i)
#pragma unroll
      for (int b = 0; b < 4; ++b)
        acc[b][i % NT] = kTR ? mfma16(F.p[b], F.q[i], acc[b][i % NT]) : mfma16(F.q[i], F.p[b], acc[b][i % NT]);
  };
  auto compute = [&](int buf) {
    if constexpr (NT <= 4) {
      Frags F0, F1;
      read(buf, 0, F0);
      read(buf, 1, F1);
      multiply(F0);
      multiply(F1);
    } else {                                   // the operands of one half fill the registers
      Frags F;
      read(buf, 0, F);
      multiply(F);
      read(buf, 1, F);
      multiply(F);
    }
  };
  // Chunk i of the item is in set i % 2; loads past the end repeat the last
  // chunk. The row numbers of a chunk are asked for before the loads of the
  // chunk before it: waiting for them then leaves those loads in flight (asked
  // for after them, every step waited for all its loads, 2.8 us a chunk).
  Regs R0, R1;
  int ra[kPer], rb[kPer];
  const int last = it.c1 - 1;
  auto at = [&](int ch) { return ch <= last ? ch : last; };
  rows_of(it.c0, ra);
  rows_of(at(it.c0 + 1), rb);
  load(it.c0, ra, R0);
  __builtin_amdgcn_sched_barrier(0);
  rows_of(at(it.c0 + 2), ra);
  __builtin_amdgcn_sched_barrier(0);
  load(at(it.c0 + 1), rb, R1);
  __builtin_amdgcn_sched_barrier(0);
  auto barrier = [&] { lds_barrier_on(tiles, qtiles, tiles, qtiles); };   // LDS done; loads stay in flight
  auto next_loads = [&](int ch, const int (&rows)[kPer], int (&rows_next)[kPer], Regs& R) {
    __builtin_amdgcn_sched_barrier(0);
    rows_of(at(ch + 1), rows_next);
    __builtin_amdgcn_sched_barrier(0);
    load(at(ch), rows, R);
    __builtin_amdgcn_sched_barrier(0);
  };
  if constexpr (kTwo) {
    // one workgroup per CU: chunk ch + 1 is written into the other buffers
    // while chunk ch is multiplied
    store(R0, 0);
    next_loads(it.c0 + 2, ra, rb, R0);
    barrier();
    // a chunk: its first operands; then its products, the reads of the second
    // half and the decode and writes of the next chunk between them (one wave
    // per SIMD: nothing else would cover the LDS latency)
    auto step = [&](int buf, const Regs& next) {
      if constexpr (NT > 4) {
        store(next, buf ^ 1);
        compute(buf);
        return;
      }
      Frags F0, F1;
      read(buf, 0, F0);
      __builtin_amdgcn_sched_barrier(0);
      read(buf, 1, F1);
      multiply(F0);
      store(next, buf ^ 1);
      multiply(F1);
#pragma unroll
      for (int i = 0; i < 8 * kSplit * NT; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);               // MFMA
        if (i < 4 * kSplit * NT) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // LDS read
        __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);               // VALU
        if (i % 4 == 3) __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);            // LDS write
      }
    };
    for (int ch = it.c0; ch < it.c1; ch += 2) {
      step(0, R1);
      next_loads(ch + 3, rb, ra, R1);
      barrier();
      if (ch + 1 < it.c1) {
        step(1, R0);
        next_loads(ch + 4, ra, rb, R0);
        barrier();
      }
    }
  } else {
    for (int ch = it.c0; ch < it.c1; ch += 2) {
      barrier();                               // the reads of the chunk before are done
      store(R0, 0);
      next_loads(ch + 2, ra, rb, R0);
      barrier();
      compute(0);
      if (ch + 1 < it.c1) {
        barrier();
        store(R1, 0);
        next_loads(ch + 3, rb, ra, R1);
        barrier();
        compute(0);
      }
    }
  }

  // with more items than one: the sums go out whole, and the last workgroup
  // of the column tile takes them back in item order
  float* const out = (kTR ? A.dA : A.dB) + static_cast<int64_t>(it.adapter) * C * r;
  const float s = A.scale ? A.scale[it.adapter] : A.alpha_r;
  if (it.slot >= 0) {
    constexpr int kBytes = kGCols * 16 * NT * 4;
    auto part = [&](int slot) {
      return part_rsrc(A.part + (static_cast<int64_t>(__builtin_amdgcn_readfirstlane(slot)) * gridDim.x + blockIdx.x) *
                                    (kBytes / 4), kBytes);
    };
    const __amdgpu_buffer_rsrc_t mine = part(it.slot);
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
      for (int jt = 0; jt < NT; ++jt) put_part(mine, (b * NT + jt) * kGThreads + t, acc[b][jt]);
    if (!arrived_last(A.cnt2 + static_cast<int64_t>(it.slot0) * gridDim.x + blockIdx.x, it.items, t,
                      reinterpret_cast<int*>(tiles)))
      return;
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
      for (int jt = 0; jt < NT; ++jt) acc[b][jt] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int i = 0; i < it.items; ++i) {
      const __amdgpu_buffer_rsrc_t other = part(it.slot0 + i);
#pragma unroll
      for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int jt = 0; jt < NT; ++jt) acc[b][jt] += get_part(other, (b * NT + jt) * kGThreads + t);
    }
  }
  // a lane has four neighbours of one row of the output
  const bool wide = kTR || r % 4 == 0;
#pragma unroll
  for (int b = 0; b < 4; ++b)
#pragma unroll
    for (int jt = 0; jt < NT; ++jt) {
      const int cc = c0 + 64 * w + 16 * b + (kTR ? 4 * G : j16);
      const int j = 16 * jt + (kTR ? j16 : 4 * G);
      if (j >= r || cc >= C) continue;
      float* const o = kTR ? out + static_cast<int64_t>(j) * C + cc : out + static_cast<int64_t>(cc) * r + j;
      const f32x4 v = acc[b][jt] * s;
      if (wide) {
        f32x4* const o4 = reinterpret_cast<f32x4*>(o);
        *o4 = A.accumulate ? *o4 + v : v;
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (j + q < r) o[q] = A.accumulate ? o[q] + v[q] : v[q];
      }
    }
}

}  // namespace

// blockIdx.x: the column tiles of dB (over dY), then those of dA (over x);
// blockIdx.y: the item. Past the items: the gradients of adapters without rows
// are cleared (unless they are added to), every gridDim.y - items'th adapter.
template <int NT, int XF>
__global__ __launch_bounds__(kGThreads) void k_mgrad(MgArgs A, GradLists L) {
  __shared__ u32x4 tile[(mg_two<NT>() ? 2 : 1) * 2048];
  __shared__ u32x4 qtile[(mg_two<NT>() ? 2 : 1) * kSplit * 16 * NT * 8];
  const bool is_b = static_cast<int>(blockIdx.x) < A.ctb;
  GradItem it;
  if (L.total) {
    const int items = L.total[1];
    if (static_cast<int>(blockIdx.y) >= items) {
      if (A.accumulate) return;
      const int C = is_b ? A.N : A.K, c0 = (is_b ? blockIdx.x : blockIdx.x - A.ctb) * kGCols;
      const int cols = C - c0 < kGCols ? C - c0 : kGCols;
      for (int a = blockIdx.y - items; a < A.n; a += gridDim.y - items) {
        if (L.adapter[a].items) continue;
        float* const o = (is_b ? A.dB : A.dA) + static_cast<int64_t>(a) * C * A.r;
        for (int e = 4 * threadIdx.x; e < cols * A.r; e += 4 * kGThreads)
          *reinterpret_cast<f32x4*>(o + (is_b ? static_cast<int64_t>(c0) * A.r + e
                                              : static_cast<int64_t>(e / cols) * C + c0 + e % cols)) =
              f32x4{0.f, 0.f, 0.f, 0.f};
      }
      return;
    }
    it = L.item[blockIdx.y];
  } else {
    const int c0 = blockIdx.y * A.per, c1 = c0 + A.per;
    const bool one = gridDim.y == 1;
    it = GradItem{0, c0, c1 < A.chunks ? c1 : A.chunks, one ? -1 : static_cast<int>(blockIdx.y),
                  static_cast<int>(gridDim.y), one ? -1 : 0};
  }
  if (is_b)
    grad_item<NT, false, kActBf16>(A, it, L, blockIdx.x, tile, qtile);
  else
    grad_item<NT, true, XF>(A, it, L, blockIdx.x - A.ctb, tile, qtile);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// Row blocks of 64 (an adapter's operands are then read once for 64 rows) where
// there are enough of them, else of 16. Q: one workgroup per CU in all with
// blocks of 64 (t of 4096 rows, 4096 deep: 33, 22, 16 and 23 us in 64, 128, 256
// and 512), two with blocks of 16, whose rows may have 16 adapters.
MultiDownPlan multi_down_plan(int64_t M, int64_t Kc, int r, int n) {
  MultiDownPlan p;
  p.RM = M >= 1024 ? 4 : 1;
  p.blocks = cdiv(M, 16 * p.RM);
  // ranges of at least a round of chunks per wave; a workgroup more than
  // passes times ranges has nothing to do
  const int64_t round = p.RM == 1 ? 4 * kMdWaves : 2 * kMdWaves;
  p.Smax = std::max<int64_t>(std::min<int64_t>(cdiv(cdiv(Kc, 64), round), kMdMaxSplit), 1);
  const int64_t passes = std::min<int64_t>({n, M, 16 * p.RM});
  p.Q = std::max<int64_t>(std::min((p.RM == 1 ? 512 : 256) / p.blocks, passes * p.Smax), 1);
  if (p.Smax > p.Q) p.Smax = p.Q;
  if (p.Smax > 1) p.part_bytes = align256(static_cast<size_t>(p.blocks * p.Smax * p.RM * down_nt(r)) * 1024);
  return p;
}

hipError_t launch_multi_down(bool wrow, const uint16_t* in, int64_t M, int64_t Kc, const uint16_t* W,
                             const MultiLora& ml, int r, uint16_t* out, void* ws, float* part, hipStream_t stream,
                             u32x4* frags, int64_t mtiles) {
  const MultiDownPlan p = multi_down_plan(M, Kc, r, ml.n);
  MdArgs a{};
  a.in = in;
  a.W = W;
  a.out = out;
  a.part = part;
  a.cnt = static_cast<unsigned*>(ws);
  a.frags = frags;
  a.M = M;
  a.nfrag = frags ? mtiles * cdiv(Kc, 256) * 8 : 0;
  a.Kc = static_cast<int>(Kc);
  a.r = r;
  a.rp = static_cast<int>(rank_pad(r));
  a.blocks = static_cast<int>(p.blocks);
  a.Q = static_cast<int>(p.Q);
  a.Smax = static_cast<int>(p.Smax);
  const dim3 grid(static_cast<unsigned>(p.blocks * p.Q + cdiv(a.nfrag, kMdWaves))), block(64 * kMdWaves);
#define QNF4_MD2(RMV, RTV, BT) hipLaunchKernelGGL(HIP_KERNEL_NAME(k_mdown<RMV, RTV, BT>), grid, block, 0, stream, a, ml)
#define QNF4_MD(RTV)                                 \
  do {                                               \
    if (wrow && p.RM == 1) QNF4_MD2(1, RTV, false);  \
    else if (wrow) QNF4_MD2(4, RTV, false);          \
    else if (p.RM == 1) QNF4_MD2(1, RTV, true);      \
    else QNF4_MD2(4, RTV, true);                     \
  } while (0)
  switch (down_nt(r)) {
    case 1: QNF4_MD(1); break;
    case 2: QNF4_MD(2); break;
    case 4: QNF4_MD(4); break;
    default: QNF4_MD(8); break;
  }
#undef QNF4_MD
#undef QNF4_MD2
  return hipGetLastError();
}

MultiGradPlan multi_grad_plan(int64_t M, int64_t N, int64_t K, int r, int n, bool listed) {
  MultiGradPlan g;
  g.nt = down_nt(r);
  const int64_t full = cdiv(M, 64);
  const int64_t used = listed ? std::min<int64_t>(M, n) : 0;       // adapters that can have rows
  g.chunks = listed ? M / 64 + used : full;                        // at most, with each adapter's last chunk partial
  g.Mp = g.chunks * 64;
  // t and u: about one workgroup per CU (more splits cost more than they
  // hide: 4096 rows at 11008 x 4096 29 us with 4, 43 with 14), each chunk's split between them by
  // their lengths, two 64-deep pieces and more per wave (513 rows, 4096 deep:
  // 12.5 us in 16 ranges, 10.9 in 8, 11.3 in 4). From 145 chunks on nothing is
  // split: a split chunk needs an arrival counter, of which there are 4096.
  const int64_t nk = cdiv(K, 64), nn = cdiv(N, 64), q = std::max<int64_t>(288 / g.chunks, 1);
  auto splits = [&](int64_t want, int64_t pieces) {
    return std::max<int64_t>(std::min({want, cdiv(pieces, 2 * kMdWaves), int64_t{kMdMaxSplit}}), 1);
  };
  g.St = splits(std::max<int64_t>((q * nk + (nk + nn) / 2) / (nk + nn), 1), nk);
  g.Su = splits(q > 1 ? q - std::min(q - 1, g.St) : 1, nn);
  // items: about two workgroups per CU over all column tiles; an item's
  // partial sums (4 r bytes a column) stay small beside the rows it reads (r 16,
  // 513 rows: 8.6 us with items of two chunks, 10.2 of four; r 64, 4096 rows:
  // 43 us of sixteen, 55 of eight)
  const int64_t ct = cdiv(N, kGCols) + cdiv(K, kGCols);
  g.per_item = std::max<int64_t>({cdiv(full, cdiv(512, ct)), r > 16 ? r / 4 : 2, 2});
  g.items = listed ? full / g.per_item + used : cdiv(full, g.per_item);
  // slots: an adapter of I >= 2 items has more than (I - 1) per_item full chunks
  g.slots = listed ? 2 * (full / g.per_item) : (g.items > 1 ? g.items : 0);
  size_t off = kWsCounterBytes;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += align256(bytes);
    return o;
  };
  g.rows_off = take(static_cast<size_t>(g.Mp) * 4);
  if (listed) {
    g.chunk_off = take(static_cast<size_t>(g.chunks) * 4);
    g.item_off = take(static_cast<size_t>(g.items) * sizeof(GradItem));
    g.adapter_off = take(static_cast<size_t>(n) * sizeof(GradAdapter));
    g.total_off = take(8);
  }
  g.cnt2_off = take(static_cast<size_t>(g.slots * ct) * 4);
  const size_t qb = static_cast<size_t>(kSplit) * 16 * g.nt * g.Mp * 2;
  g.tt_off = take(qb);
  g.ut_off = take(qb);
  g.dp_off = take(g.St > 1 || g.Su > 1 ? static_cast<size_t>(2 * g.chunks * kMdMaxSplit * 4 * g.nt) * 1024 : 0);
  g.part_off = take(static_cast<size_t>(g.slots * ct) * kGCols * 16 * g.nt * 4);
  g.total = off;
  return g;
}

hipError_t launch_multi_grad(const void* x, const uint16_t* tops, int xfmt, const uint16_t* dy, int64_t M, int64_t N,
                             int64_t K, const uint16_t* A, const uint16_t* B, const float* scale, float alpha_r, int n,
                             const int* index, int r, float* dA, float* dB, int accumulate, void* ws,
                             hipStream_t stream) {
  const MultiGradPlan g = multi_grad_plan(M, N, K, r, n, index != nullptr);
  char* wsb = static_cast<char*>(ws);
  const int ctb = static_cast<int>(cdiv(N, kGCols)), cta = static_cast<int>(cdiv(K, kGCols));
  const bool find = index && M <= kFindMaxM;
  GradLists L{};
  L.rows = reinterpret_cast<int*>(wsb + g.rows_off);
  if (index) {
    L.chunk_adapter = reinterpret_cast<int*>(wsb + g.chunk_off);
    L.item = reinterpret_cast<GradItem*>(wsb + g.item_off);
    L.adapter = reinterpret_cast<GradAdapter*>(wsb + g.adapter_off);
    L.total = reinterpret_cast<int*>(wsb + g.total_off);
    if (!find)
      hipLaunchKernelGGL(k_msort, dim3(static_cast<unsigned>(cdiv(n, 4))), dim3(256), 0, stream, index, M, n,
                         static_cast<int>(g.per_item), L);
  }
  GdArgs d{};
  d.x = x;
  d.tops = tops;
  d.dy = dy;
  d.A = A;
  d.B = B;
  d.index = index;
  d.tt = reinterpret_cast<uint16_t*>(wsb + g.tt_off);
  d.ut = reinterpret_cast<uint16_t*>(wsb + g.ut_off);
  d.part = reinterpret_cast<float*>(wsb + g.dp_off);
  d.cnt = reinterpret_cast<unsigned*>(wsb);
  d.cnt2 = reinterpret_cast<unsigned*>(wsb + g.cnt2_off);
  d.M = M;
  d.N = static_cast<int>(N);
  d.K = static_cast<int>(K);
  d.r = r;
  d.n = n;
  d.per = static_cast<int>(g.per_item);
  d.St = static_cast<int>(g.St);
  d.Su = static_cast<int>(g.Su);
  d.ncnt2 = static_cast<int>(g.slots * (ctb + cta));
  d.mode = find ? kGdFind : index ? kGdListed : kGdWhole;
  MgArgs m{};
  m.x = x;
  m.tops = tops;
  m.dy = dy;
  m.tt = d.tt;
  m.ut = d.ut;
  m.scale = scale;
  m.part = reinterpret_cast<float*>(wsb + g.part_off);
  m.dA = dA;
  m.dB = dB;
  m.cnt2 = d.cnt2;
  m.M = M;
  m.alpha_r = alpha_r;
  m.N = d.N;
  m.K = d.K;
  m.r = r;
  m.n = n;
  m.ctb = ctb;
  m.per = d.per;
  m.chunks = static_cast<int>(g.chunks);
  m.accumulate = accumulate;
  const dim3 dgrid(static_cast<unsigned>(g.chunks * (g.St + g.Su)));
  // a few workgroups without an item for adapters without rows
  const int64_t clear = index && !accumulate ? std::min<int64_t>(n, 8) : 0;
  const dim3 ggrid(static_cast<unsigned>(ctb + cta), static_cast<unsigned>(g.items + clear));
#define QNF4_MG(NTV, XFV)                                                                                    \
  do {                                                                                                       \
    hipLaunchKernelGGL(HIP_KERNEL_NAME(k_gdown<NTV, XFV>), dgrid, dim3(kGdThreads), 0, stream, d, L);        \
    hipLaunchKernelGGL(HIP_KERNEL_NAME(k_mgrad<NTV, XFV>), ggrid, dim3(kGThreads), 0, stream, m, L);         \
  } while (0)
#define QNF4_MGX(NTV)                                  \
  do {                                                 \
    if (xfmt == kActBf16) QNF4_MG(NTV, kActBf16);      \
    else if (xfmt == kActInt8) QNF4_MG(NTV, kActInt8); \
    else QNF4_MG(NTV, kActE4m3);                       \
  } while (0)
  switch (g.nt) {
    case 1: QNF4_MGX(1); break;
    case 2: QNF4_MGX(2); break;
    case 4: QNF4_MGX(4); break;
    default: QNF4_MGX(8); break;
  }
#undef QNF4_MGX
#undef QNF4_MG
  return hipGetLastError();
}

}  // namespace qnf4
