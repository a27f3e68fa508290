// Fused NF4-dequant matmuls for gfx950 (MI355X).
//
// Forward  y  = bf16( x . W'^T + (alpha/r) . t . B^T ),  t = bf16(x . A^T)
// Backward dX = bf16( dY . W'  + (alpha/r) . u . A   ),  u = bf16(dY . B)
// with W' the bf16 dequantization of the NF4 weight, done block by block
// right before the multiply ("A 65B fine-tune on the GPU you already have",
// figure 2; "QLoRA Explained", "What is QLoRA?").
//
// Kernels (M > 16; the decode shapes have their own kernels)
//   k_gemm_fwd    M > 16: 256x256 output tile, 4 waves each owning 64 output
//                 columns; each lane dequantizes its MFMA B operands straight
//                 into registers, x goes through double-buffered LDS; 32x32x16
//                 bf16 MFMA with fp32 accumulation; LoRA as a rank-r MFMA in
//                 the epilogue. MFMA-bound.
//   k_gemm_bwd    M > 16: same tiling over dX [M, K]; the contraction runs over
//                 W's rows, so the dequantized tile is stored row-major and
//                 read transposed with ds_read_b64_tr_b16.
// The rank-r down projections t and u come from k_down_rows (lora.hip).
// Both kernels also have a form (kMulti) for a batch whose rows use different
// adapters of a pool, with a contraction that can be split (t and u from
// k_mdown, multi.hip; partial sums added by k_split_sum), and the backward one
// for fewer rows per tile. 4096 rows at 11008 x 4096, r 16, eight adapters: 348
// and 356 us with t and u, against 314 at the rate of a large library product.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "mm_common.hpp"
#include "multi.hpp"

namespace qnf4 {

// ---------------------------------------------------------------------------
// Tiled MFMA GEMMs (M > 16)
// ---------------------------------------------------------------------------
constexpr int kTile = 256;
constexpr int kChunks = 2048;                // 16-byte chunks in one 256x64 bf16 tile

// Workgroup id -> output tile. Consecutive ids land on different XCDs (round
// robin over 8), so each XCD is first given a contiguous range of the tile
// order; that order then sweeps groups of 4 tile-rows across all tile-columns
// so co-resident workgroups share operand tiles in their XCD's L2 (the 32
// workgroups an XCD runs at once cover 4 x 8 tiles: a quarter less L2 fill
// than 8 x 4, since an x tile row is four times the bytes of a code column).
__device__ __forceinline__ void tile_of(int pid, int ntm, int ntn, int& tm, int& tn) {
  const int total = ntm * ntn;
  int p = pid;
  if ((total & 7) == 0) p = (pid & 7) * (total >> 3) + (pid >> 3);
  const int G = 4;
  const int group = p / (G * ntn);
  const int first_m = group * G;
  const int gsz = (ntm - first_m) < G ? (ntm - first_m) : G;
  const int within = p - group * G * ntn;
  tm = first_m + within % gsz;
  tn = within / gsz;
}

// The adapters of the 256 rows of a tile: lane l has those of rows 64 q + l.
struct TileRows {
  int id[4];
  __device__ __forceinline__ void init(const MultiLora& ml, int64_t m0, int64_t M, int lane) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t m = m0 + 64 * q + lane;
      id[q] = m < M ? ml.index[m] : -1;
      if (static_cast<unsigned>(id[q]) >= static_cast<unsigned>(ml.n)) id[q] = -1;
    }
  }
};

// rows of a 32 x 32 block that `rm` names (bit = row) from p, the others as
// they are: a NaN in one adapter must not reach the rows of another, so the
// choice is made after the product
__device__ __forceinline__ void take_rows(f32x16& tmp, const f32x16& p, uint32_t rm, int h) {
  const uint32_t mine = rm >> (4 * h);
#pragma unroll
  for (int v = 0; v < 16; ++v) tmp[v] = (mine >> (8 * (v >> 2) + (v & 3))) & 1u ? p[v] : tmp[v];
}

// A tile (256 rows x 64 deep, bf16) in LDS: row-major, 8 chunks of 16 bytes
// per row. The LDS has 64 four-byte banks and serves a 16-byte-per-lane read
// 16 lanes at a time; a 128-byte row covers half the banks, so rows of one
// parity share a half. Logical chunk c of row r sits at physical chunk
// c ^ ((r >> 1) & 7): 16 consecutive rows reading the same logical chunk then
// land on 8 distinct chunks in each half, i.e. on all 64 banks once.
__device__ __forceinline__ int a_swz(int row) { return (row >> 1) & 7; }
__device__ __forceinline__ int a_slot(int row, int ch) { return row * 8 + (ch ^ a_swz(row)); }

// ---------------------------------------------------------------------------
// k_gemm_fwd: y [M, N] = x . W'^T (+ LoRA), M > 16.
//
// Workgroup tile 256 (M) x 256 (N), 4 waves; wave w owns output columns
// [64w, 64w + 64) for all 256 rows: 8 x 2 blocks of 32x32x16 bf16 MFMA with
// fp32 accumulators. In this NT layout one packed dword (8 codes of one
// weight row) is exactly one MFMA B operand, so each lane dequantizes its own
// B operands straight into registers and every weight is decoded once.
//
// Memory traffic is what limits this kernel, so every stream is moved in
// whole 128-byte lines:
//   x      global -> LDS by DMA (buffer_load ... lds), a ring of four 256x64
//          tiles; the tile of step k+3 is requested at the start of step k.
//   codes  each wave DMAs the codes of its own 64 weight rows for a super-step
//          of four K steps (64 rows x 128 bytes = 8 KB) into a private LDS
//          slab; lanes then read their 16-byte code words from LDS. The slab
//          of super-step S+1 is requested in step 4S+2, right after that
//          step has read the last codes of super-step S.
//   scales q and d of step k+2 are loaded at the start of step k.
// In step k the MFMAs of step k run while the codes of step k+1 are decoded.
// LDS: 4 x 32 KB of x + 4 x 8 KB of codes = 160 KB, one workgroup per CU.
//
// K permutation: within a step, lane half h holds k in [32h, 32h + 32) and
// MFMA sub-step s uses k = 32h + 8s + (0..7) on both operands (the sum over k
// is order-free), so a lane's codes for a step are one 16-byte word.
// ---------------------------------------------------------------------------
constexpr int kBufferDword3 = 0x00020000;    // raw buffer descriptor word 3 on gfx9-family parts

struct BScale {
  float d[2];      // second-level steps of this lane's weight rows (N-blocks j)
  int8_t q[2];     // block scale codes
  float live;      // 1 for a real K step, 0 for a step past the end
};
struct BScale4 {   // the same for the four steps of a super-step
  float d[2];
  uint32_t q[2];   // byte u = scale code of step 4S + u
};


// kQuad: K is a multiple of 256, so the four block-scale codes of a
// super-step are one aligned 4-byte word of qscale and share one second-level
// step (a 256-block group never splits 4-aligned blocks); scales are then
// loaded once per super-step. Otherwise they are loaded per step.
// RSN: chunks of 16 ranks in the LoRA epilogue (1 for r <= 16: t's padding
// columns 16 .. 31 are zero and skipped; else rank_pad(r) / 16), 0 for none.
// kMulti: tab (one weight) has a pool B [n][N][r]; row m uses adapter
// ml.index[m] of it; t carries the scale (`scale` is not used).
// kMulti also splits K (ml.S > 1): workgroup p has tile p % tiles and range p /
// tiles of the super-steps, adds the adapter term of the row blocks i with i %
// S == range, and leaves fp32 partial sums (ml.part [S][M][N]) for k_split_sum.
template <bool kQuad, int RSN, bool kMulti = false>
__global__ __launch_bounds__(256, 1) void k_gemm_fwd(FwdTable tab, int64_t M, int rp, int r, float scale,
                                                     Codebook cb, MultiLora ml) {
  // ring of four x tiles (32 KB each) and the per-wave code slabs (8 KB each),
  // distinct objects so that the compiler can tell a DMA into one from reads
  // of another
  __shared__ u32x4 As0[kChunks];
  __shared__ u32x4 As1[kChunks];
  __shared__ u32x4 As2[kChunks];
  __shared__ u32x4 As3[kChunks];
  __shared__ u32x4 Bs[4 * 512];
  const int t = threadIdx.x, lane = t & 63;
  const int w = __builtin_amdgcn_readfirstlane(t >> 6);   // wave index, provably uniform (SGPR)
  const int h = lane >> 5, l32 = lane & 31;
  // The weights' tile columns are numbered one after another, so the tile
  // order sweeps groups of tile-rows across every weight of the table (x
  // rows shared by weights with the same input stay in L2 across them).
  const int ntm = static_cast<int>(cdiv(M, kTile));
  int tm, tnv;
  const int ntiles = ntm * tab.col0[tab.count];
  const int split = kMulti ? __builtin_amdgcn_readfirstlane(static_cast<int>(blockIdx.x) / ntiles) : 0;
  tile_of(blockIdx.x - split * ntiles, ntm, tab.col0[tab.count], tm, tnv);
  tm = __builtin_amdgcn_readfirstlane(tm);     // uniform already; this keeps the
  tnv = __builtin_amdgcn_readfirstlane(tnv);   // buffer descriptors in SGPRs
  int g = 0;
#pragma unroll
  for (int i = 1; i < kFwdMaxWeights; ++i)
    if (i < tab.count && tnv >= tab.col0[i]) g = i;
  g = __builtin_amdgcn_readfirstlane(g);
  const int tn = tnv - tab.col0[g];
  const uint16_t* __restrict__ x = tab.x[g];
  const uint8_t* __restrict__ packed = tab.packed[g];
  const int8_t* __restrict__ qscale = tab.qscale[g];
  const float* __restrict__ step = tab.step[g];
  const uint16_t* __restrict__ tl = tab.tl[g];
  const uint16_t* __restrict__ Bl = tab.B[g];
  uint16_t* __restrict__ y = tab.y[g];
  const int64_t N = tab.N[g], K = tab.K[g];
  const int64_t m0 = static_cast<int64_t>(tm) * kTile, n0 = static_cast<int64_t>(tn) * kTile;
  const int64_t nk = K / 64;
  const int64_t nsup = (nk + 3) / 4;           // super-steps of four K steps
  const int64_t sup0 = kMulti ? nsup * split / ml.S : 0, sup1 = kMulti ? nsup * (split + 1) / ml.S : nsup;
  const int64_t kt0 = 4 * sup0;

  // x tile DMA (rows past M read as zero through the descriptor's range
  // check). Instruction i of wave w fills LDS rows 64w + 8i + (lane >> 3),
  // physical chunk lane & 7, i.e. logical chunk (lane & 7) ^ a_swz(row); the
  // K step goes in soffset.
  const int64_t rows_valid = imin(static_cast<int64_t>(kTile), M - m0);
  const __amdgpu_buffer_rsrc_t xr = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint16_t*>(x + m0 * K), 0, static_cast<int>(rows_valid * K * 2), kBufferDword3);
  uint32_t voff[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = 64 * w + 8 * i + (lane >> 3);
    voff[i] = static_cast<uint32_t>(row * K * 2 + 16 * ((lane & 7) ^ a_swz(row)));
  }
  auto dma_a = [&](int64_t kt, u32x4* Ab) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lds_void* dst = (lds_void*)(&Ab[(64 * w + 8 * i) * 8]);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(xr, dst, 16, voff[i], static_cast<uint32_t>(kt * 128), 0, 0);
    }
  };
  // code slab DMA: wave w's rows n0 + 64w + r, r = 8i + (lane >> 3), bytes
  // [128 S, 128 S + 128) of each packed row, same chunk swizzle as x. A
  // super-step past the end re-reads the last one (its steps are dead).
  const int64_t nrows_valid = imin(static_cast<int64_t>(kTile), N - n0);
  const __amdgpu_buffer_rsrc_t wr = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(packed + n0 * (K / 2)), 0, static_cast<int>(nrows_valid * (K / 2)), kBufferDword3);
  uint32_t boff[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r8 = 8 * i + (lane >> 3);
    boff[i] = static_cast<uint32_t>((64 * w + r8) * (K / 2) + 16 * ((lane & 7) ^ a_swz(r8)));
  }
  u32x4* const Bw = Bs + 512 * w;              // this wave's slab: 64 rows x 8 chunks
  auto dma_b = [&](int64_t S) {
    const uint32_t so = static_cast<uint32_t>(imin(S, nsup - 1) * 128);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lds_void* dst = (lds_void*)(&Bw[64 * i]);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(wr, dst, 16, boff[i], so, 0, 0);
    }
  };
  // the 16-byte code words of K step kt for this lane (N-blocks j = 0, 1)
  auto read_codes = [&](int64_t kt, u32x4 (&c)[2]) {
    const int ch = (2 * static_cast<int>(kt & 3) + h) ^ a_swz(l32);   // a_swz(32 j + l32) == a_swz(l32)
#pragma unroll
    for (int j = 0; j < 2; ++j) c[j] = Bw[(32 * j + l32) * 8 + ch];
  };
  int64_t bblk[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) bblk[j] = imin(n0 + 64 * w + 32 * j + l32, N - 1) * nk;
  // block scales of K step kt; a step past the end (the loop runs whole
  // super-steps) re-reads the last one and is marked dead, which makes its
  // block scale, and so every decoded weight, zero
  auto load_s = [&](int64_t kt, BScale& P) {
    const int64_t kc = imin(kt, nk - 1);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      P.q[j] = qscale[bblk[j] + kc];
      P.d[j] = step[(bblk[j] + kc) >> 8];
    }
    P.live = kt < nk ? 1.0f : 0.0f;
  };
  auto load_s4 = [&](int64_t S, BScale4& P) {
    const int64_t kc = 4 * imin(S, nsup - 1);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      P.q[j] = *reinterpret_cast<const uint32_t*>(qscale + bblk[j] + kc);
      P.d[j] = step[(bblk[j] + kc) >> 8];
    }
  };
  // scales of step kt (position u in its super-step) from a quad
  auto scale_of = [&](const BScale4& P, int u, int64_t kt, int j) {
    const int8_t q = static_cast<int8_t>((P.q[j] >> (8 * u)) & 0xFFu);
    return block_scale(q, P.d[j]) * (kt < nk ? 1.0f : 0.0f);
  };
  f32x16 acc[8][2];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
  bf16x8 B0_[2][4], B1[2][4];                  // decoded B of the current / next step

  // One K step k (position u = k % 4 in its super-step): reads x tile Ab,
  // multiplies with the decoded B `bo`, decodes the codes of step k+1 (read
  // here from the slab) with the block scales scales_next(j) into `bn`,
  // requests x tile k+3 into An, issues this step's scale loads
  // (issue_scales) and, at u == 2, the next super-step's code slab.
  auto step_k = [&](auto u_c, const u32x4* Ab, u32x4* An, const bf16x8 (&bo)[2][4], bf16x8 (&bn)[2][4],
                    auto&& issue_scales, auto&& scales_next, int64_t k) {
    constexpr int u = decltype(u_c)::value;
    u32x4 cw[2];
    read_codes(k + 1, cw);
    if constexpr (u == 2) {
      // the slab's last reads have landed: refill it first, so that waiting
      // for it (end of this step) leaves this step's x-tile and scale loads
      // in flight
      wait_lgkm0();
      asm volatile("" ::: "memory");
      dma_b(k / 4 + 1);
      __builtin_amdgcn_sched_barrier(0);
    }
    dma_a(imin(k + 3, nk - 1), An);
    __builtin_amdgcn_sched_barrier(0);
    issue_scales();
    __builtin_amdgcn_sched_barrier(0);
    MagTable tb[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) tb[j] = make_table(cb, scales_next(j));
    // A fragments double-buffered across sub-steps: those of s+1 are read
    // while the MFMAs of s issue
    bf16x8 afr[2][8];
    auto read_frags = [&](int s, bf16x8 (&af)[8]) {
      const int sw = (4 * h + s) ^ a_swz(l32);     // a_swz(32 i + l32) == a_swz(l32)
#pragma unroll
      for (int i = 0; i < 8; ++i) af[i] = as_bf16x8(Ab[(32 * i + l32) * 8 + sw]);
    };
    read_frags(0, afr[0]);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      if (s < 3) read_frags(s + 1, afr[(s + 1) & 1]);
      const bf16x8 (&af)[8] = afr[s & 1];
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = mfma32(af[i], bo[j][s], acc[i][j]);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t pw = s == 0 ? cw[j].x : s == 1 ? cw[j].y : s == 2 ? cw[j].z : cw[j].w;
        bn[j][s] = as_bf16x8(decode8(pw, tb[j]));
      }
    }
    // issue order after the loads: the A fragments of sub-step 0, then each
    // MFMA followed by four VALU ops (the decode of the next step) and, every
    // other MFMA, one LDS read of the next sub-step's A fragments
    __builtin_amdgcn_sched_group_barrier(0x100, 8, 0);
#pragma unroll
    for (int m = 0; m < 64; ++m) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      if ((m & 1) == 0 && m < 48) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
    }
  };
  using U0 = std::integral_constant<int, 0>;
  using U1 = std::integral_constant<int, 1>;
  using U2 = std::integral_constant<int, 2>;
  using U3 = std::integral_constant<int, 3>;
  auto decode_step0 = [&](auto&& scale0) {
    u32x4 c0[2];
    read_codes(kt0, c0);
    bf16x8 (&bo)[2][4] = B0_;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const MagTable tb = make_table(cb, scale0(j));
      bo[j][0] = as_bf16x8(decode8(c0[j].x, tb));
      bo[j][1] = as_bf16x8(decode8(c0[j].y, tb));
      bo[j][2] = as_bf16x8(decode8(c0[j].z, tb));
      bo[j][3] = as_bf16x8(decode8(c0[j].w, tb));
    }
  };
  bf16x8 (&B0)[2][4] = B0_;
  auto nothing = [] {};

  // Prologue: the loads of "steps -2 and -1" in the order the loop issues
  // them, so that the loop's wait counts hold from step 0 on.
  // Vector-memory loads per step, in order: at u == 2 the code slab (8), then
  // x tile k+3 (8), then the scale loads (quad path: 4 at u == 1 for the next
  // super-step; per-step path: 4 for step k+2). The end of step k waits for x
  // tile k+1, issued in step k-2; whatever was issued after it may stay in
  // flight, and that count is the argument of each wait_vm below. Step u == 2
  // waits instead for the code slab it requested first (so only its own
  // x-tile and scale loads stay in flight): the next step reads that slab
  // right after the barrier. These explicit waits are what order the slab
  // DMA before its reads: the compiler's own LDS-DMA tracking cannot be
  // relied on to cover reads at other offsets of the slab.
  if constexpr (kQuad) {
    BScale4 Qc, Qn;
    load_s4(sup0, Qc);
    __builtin_amdgcn_sched_barrier(0);
    dma_a(kt0, As0);
    __builtin_amdgcn_sched_barrier(0);
    dma_b(sup0);
    __builtin_amdgcn_sched_barrier(0);
    dma_a(imin(kt0 + 1, nk - 1), As1);
    __builtin_amdgcn_sched_barrier(0);
    dma_a(imin(kt0 + 2, nk - 1), As2);
    __builtin_amdgcn_sched_barrier(0);
    wait_vm<16>();                             // scales of super-step 0, x tile 0, code slab 0
    decode_step0([&](int j) { return scale_of(Qc, 0, kt0, j); });
    lds_barrier();
    for (int64_t S = sup0; S < sup1; ++S) {
      const int64_t k = 4 * S;
      step_k(U0{}, As0, As3, B0, B1, nothing, [&](int j) { return scale_of(Qc, 1, k + 1, j); }, k);
      wait_vm<16>();
      lds_barrier();
      step_k(U1{}, As1, As0, B1, B0, [&] { load_s4(S + 1, Qn); },
             [&](int j) { return scale_of(Qc, 2, k + 2, j); }, k + 1);
      wait_vm<20>();
      lds_barrier();
      step_k(U2{}, As2, As1, B0, B1, nothing, [&](int j) { return scale_of(Qc, 3, k + 3, j); }, k + 2);
      wait_vm<8>();                            // also the code slab requested first in this step
      lds_barrier();
      step_k(U3{}, As3, As2, B1, B0, nothing, [&](int j) { return scale_of(Qn, 0, k + 4, j); }, k + 3);
      wait_vm<28>();
      lds_barrier();
      Qc = Qn;
    }
  } else {
    BScale P0, P1;
    dma_a(kt0, As0);
    __builtin_amdgcn_sched_barrier(0);
    dma_b(sup0);
    __builtin_amdgcn_sched_barrier(0);
    dma_a(imin(kt0 + 1, nk - 1), As1);
    __builtin_amdgcn_sched_barrier(0);
    load_s(kt0, P0);
    __builtin_amdgcn_sched_barrier(0);
    dma_a(imin(kt0 + 2, nk - 1), As2);
    __builtin_amdgcn_sched_barrier(0);
    load_s(kt0 + 1, P1);
    __builtin_amdgcn_sched_barrier(0);
    wait_vm<12>();                             // everything up to the scales of step 0
    // pin step 1's scales here: left alone, the (read-only) loads get sunk
    // into the loop entry, and the loop head would then drain every later load
    asm volatile("" ::"v"(static_cast<int>(P1.q[0])), "v"(static_cast<int>(P1.q[1])), "v"(P1.d[0]), "v"(P1.d[1]));
    decode_step0([&](int j) { return block_scale(P0.q[j], P0.d[j]) * P0.live; });
    lds_barrier();
    auto sc = [](const BScale& P, int j) { return block_scale(P.q[j], P.d[j]) * P.live; };
    for (int64_t S = sup0; S < sup1; ++S) {
      const int64_t k = 4 * S;
      step_k(U0{}, As0, As3, B0, B1, [&] { load_s(k + 2, P0); }, [&](int j) { return sc(P1, j); }, k);
      wait_vm<28>();
      lds_barrier();
      step_k(U1{}, As1, As0, B1, B0, [&] { load_s(k + 3, P1); }, [&](int j) { return sc(P0, j); }, k + 1);
      wait_vm<28>();
      lds_barrier();
      step_k(U2{}, As2, As1, B0, B1, [&] { load_s(k + 4, P0); }, [&](int j) { return sc(P1, j); }, k + 2);
      wait_vm<12>();                           // also the code slab requested first in this step
      lds_barrier();
      step_k(U3{}, As3, As2, B1, B0, [&] { load_s(k + 5, P1); }, [&](int j) { return sc(P0, j); }, k + 3);
      wait_vm<36>();
      lds_barrier();
    }
  }
  wait_vm<0>();

  // epilogue: LoRA up-projection as a rank-r MFMA (RSN chunks of 16 ranks),
  // then bf16 stores
  if constexpr (RSN > 0) {
    const bool vec_ok = (r & 7) == 0;
    // All fragment loads of a group of row blocks go out before its MFMAs,
    // so their latency is paid once, not once per MFMA.
    auto lora = [&](auto rsn_c) {
      constexpr int RS = decltype(rsn_c)::value;
      constexpr int IG = RS <= 2 ? 8 : RS <= 4 ? 4 : 2;   // row blocks per group (registers)
      u32x4 bfr[2][RS];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int64_t nrow = imin(n0 + 64 * w + 32 * j + l32, N - 1);
#pragma unroll
        for (int rs = 0; rs < RS; ++rs) bfr[j][rs] = load_row8(Bl + nrow * r, 16 * rs + 8 * h, r, vec_ok);
      }
#pragma unroll
      for (int i0 = 0; i0 < 8; i0 += IG) {
        u32x4 tf[IG][RS];
#pragma unroll
        for (int ii = 0; ii < IG; ++ii) {
          const int64_t mrow = imin(m0 + 32 * (i0 + ii) + l32, M - 1);
#pragma unroll
          for (int rs = 0; rs < RS; ++rs) tf[ii][rs] = ld16(tl + mrow * rp + 16 * rs + 8 * h);
        }
#pragma unroll
        for (int ii = 0; ii < IG; ++ii)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            f32x16 tmp;
#pragma unroll
            for (int v = 0; v < 16; ++v) tmp[v] = 0.f;
#pragma unroll
            for (int rs = 0; rs < RS; ++rs) tmp = mfma32(as_bf16x8(tf[ii][rs]), as_bf16x8(bfr[j][rs]), tmp);
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i0 + ii][j][v] += scale * tmp[v];
          }
      }
    };
    if constexpr (!kMulti) lora(std::integral_constant<int, RSN>{});
  }
  // A pool of adapters: block by block of 32 rows, the adapters among them
  // (mostly one: rows of a request follow each other), then the block's
  // stores. The loop stays rolled: unrolled over the eight blocks, its branches
  // cost 230 to 740 bytes of spills a lane and 70 to 130 KB of code, twice the
  // instruction cache. An adapter's B fragments are kept until another one is
  // needed; t carries the scale. Rows are chosen after the product.
  if constexpr (kMulti) {
    constexpr int RS = RSN;
    const bool vec_ok = (r & 7) == 0;
    TileRows tr;
    tr.init(ml, m0, M, lane);
    u32x4 bfr[2][RS], tf[RS], tn[RS];
    auto load_t = [&](int i, u32x4 (&f)[RS]) {
      const int64_t mrow = imin(m0 + 32 * i + l32, M - 1);
#pragma unroll
      for (int rs = 0; rs < RS; ++rs) f[rs] = ld16(tl + mrow * rp + 16 * rs + 8 * h);
    };
    load_t(0, tn);
    int have = -1;
    const bool wide = n0 + kTile <= N && N % 8 == 0;
    uint16_t* const yl = reinterpret_cast<uint16_t*>(Bw);      // the wave's slab: 32 rows x 64 columns, chunks swizzled by row
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {
#pragma unroll
      for (int rs = 0; rs < RS; ++rs) tf[rs] = tn[rs];
      load_t(i < 7 ? i + 1 : 7, tn);
      f32x16 cur[2];
      switch (i) {
        case 0: cur[0] = acc[0][0], cur[1] = acc[0][1]; break;
        case 1: cur[0] = acc[1][0], cur[1] = acc[1][1]; break;
        case 2: cur[0] = acc[2][0], cur[1] = acc[2][1]; break;
        case 3: cur[0] = acc[3][0], cur[1] = acc[3][1]; break;
        case 4: cur[0] = acc[4][0], cur[1] = acc[4][1]; break;
        case 5: cur[0] = acc[5][0], cur[1] = acc[5][1]; break;
        case 6: cur[0] = acc[6][0], cur[1] = acc[6][1]; break;
        default: cur[0] = acc[7][0], cur[1] = acc[7][1]; break;
      }
      const int id = i < 2 ? tr.id[0] : i < 4 ? tr.id[1] : i < 6 ? tr.id[2] : tr.id[3];
      const int up = 32 * (i & 1);
      uint32_t pend = i % ml.S == split ? static_cast<uint32_t>(__ballot(id >= 0) >> up) : 0u;
      if (pend) {
        f32x16 tmp[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int v = 0; v < 16; ++v) tmp[j][v] = 0.f;
        while (pend) {
          const int a = __builtin_amdgcn_readlane(id, up + __builtin_ctz(pend));
          const uint32_t rows = static_cast<uint32_t>(__ballot(id == a) >> up);
          pend &= ~rows;
          if (a != have) {
            have = a;
            const uint16_t* Ba = Bl + static_cast<int64_t>(a) * N * r;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint16_t* Br = Ba + imin(n0 + 64 * w + 32 * j + l32, N - 1) * r;
#pragma unroll
              for (int rs = 0; rs < RS; ++rs) bfr[j][rs] = load_row8(Br, 16 * rs + 8 * h, r, vec_ok);
            }
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            f32x16 p;
#pragma unroll
            for (int v = 0; v < 16; ++v) p[v] = 0.f;
#pragma unroll
            for (int rs = 0; rs < RS; ++rs) p = mfma32(as_bf16x8(tf[rs]), as_bf16x8(bfr[j][rs]), p);
            take_rows(tmp[j], p, rows, h);
          }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int v = 0; v < 16; ++v) cur[j][v] += tmp[j][v];
      }
      const int64_t mb = m0 + 32 * i;
      if (ml.S > 1) {
        float* const pt = ml.part + (split * M + mb) * N + n0 + 64 * w + l32;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int v = 0; v < 16; ++v) {
            const int row = 8 * (v >> 2) + 4 * h + (v & 3);
            if (mb + row < M && n0 + 64 * w + 32 * j + l32 < N) pt[row * N + 32 * j] = cur[j][v];
          }
      } else if (wide) {
        // through the wave's slab to whole 128-byte rows
        wait_lgkm0();
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int v = 0; v < 16; ++v) {
            const int row = 8 * (v >> 2) + 4 * h + (v & 3), col = 32 * j + l32;
            yl[row * 64 + 8 * ((col >> 3) ^ (row & 7)) + (col & 7)] = bf16_bits(cur[j][v]);
          }
        wait_lgkm0();
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = 8 * e + (lane >> 3), ch = lane & 7;
          const u32x4 o = Bw[row * 8 + (ch ^ (row & 7))];
          if (mb + row < M) *reinterpret_cast<u32x4*>(y + (mb + row) * N + n0 + 64 * w + 8 * ch) = o;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int v = 0; v < 16; ++v) {
            const int64_t mm = mb + 8 * (v >> 2) + 4 * h + (v & 3), nn = n0 + 64 * w + 32 * j + l32;
            if (mm < M && nn < N) y[mm * N + nn] = bf16_bits(cur[j][v]);
          }
      }
    }
    return;
  }
  // bf16 stores: for fixed (i, j, v) the 32 lanes of a half-wave write 64
  // contiguous bytes of one row; interior tiles skip the bounds checks
  if (m0 + kTile <= M && n0 + kTile <= N) {
    uint16_t* yt = y + (m0 + 4 * h) * N + n0 + 64 * w + l32;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v)
          yt[(32 * i + 8 * (v >> 2) + (v & 3)) * N + 32 * j] = bf16_bits(acc[i][j][v]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int64_t nn = n0 + 64 * w + 32 * j + l32;
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const int64_t mm = m0 + 32 * i + 8 * (v >> 2) + 4 * h + (v & 3);
          if (mm < M && nn < N) y[mm * N + nn] = bf16_bits(acc[i][j][v]);
        }
      }
  }
}

// ---------------------------------------------------------------------------
// k_gemm_bwd: dX [M, K] = dY . W' (+ LoRA), M > 16.
//
// Workgroup tile 256 (M) x 256 (K), eight waves (two per SIMD) as 2 x 4, each
// 128 x 64: 4 x 2 blocks of 32x32x16 bf16 MFMA. The contraction runs over W's
// rows (N) in steps of 64, so the weights are needed transposed: each step
// the workgroup decodes the 64 x 256 slice of W' (half a 64-block per thread,
// every weight once) into LDS, row-major, and the waves read their B operands
// with ds_read_b64_tr_b16. Two waves per SIMD let one wave's MFMAs issue
// while the other waits on its LDS reads, its decode or the step barrier.
// Per step k:
//   dY    tile k+1 (256 x 64) loaded into registers and written into the
//         other slot of a two-slot LDS ring at the end of the step (rows past
//         M read as zero);
//   codes of step k+2 loaded into registers (16 bytes per thread: eight
//         threads per weight row);
//   the MFMAs of step k run while the codes of step k+1 are decoded and
//         written into the other W' buffer.
// LDS: 2 x 32 KB (dY) + 2 x 36 KB (W', rows padded to 576 bytes so that a
// transposed read of 4 rows x 64 bytes covers all 64 banks once).
// ---------------------------------------------------------------------------
constexpr int kBwRow = 36;                     // 16-byte chunks per LDS row of the W' tile (32 + pad)
constexpr int kBwChunks = 64 * kBwRow;
constexpr int kBwThreads = 512;

struct BCodes {
  u32x4 p;         // this thread's 16 code bytes (half a 64-block)
  float d;
  int8_t q;
  float live;      // 1 for a real weight row, 0 past N
};

// RSN: rank chunks of 16 in the LoRA epilogue (1 for r <= 16, else rank_pad(r) / 16), 0 for none.
// kMulti: Al is a pool [n][r][K]; row m uses adapter ml.index[m]; u carries the
// scale. It also splits the contraction (ml.S > 1) as k_gemm_fwd does, in ranges
// of whole step pairs; the o-th adapter of a tile is added by range o % S.
// MB: 32-row blocks per wave; the tile has 64 MB rows (fewer than 256 where the
// batch is short and the decode, not the MFMAs, bounds a step).
template <int RSN, bool kMulti = false, int MB = 4>
__global__ __launch_bounds__(kBwThreads, 1) void k_gemm_bwd(const uint16_t* __restrict__ dy, int64_t M, int64_t N,
                                                            int64_t K, const uint8_t* __restrict__ packed,
                                                            const int8_t* __restrict__ qscale,
                                                            const float* __restrict__ step,
                                                            const uint16_t* __restrict__ ul, int rp,
                                                            const uint16_t* __restrict__ Al, int r, float scale,
                                                            uint16_t* __restrict__ dx, Codebook cb,
                                                            MultiLora ml) {
  // the two W' buffers are one array: after the main loop it holds A's
  // slice for the LoRA epilogue (up to 128 ranks x 256 columns)
  constexpr int kRows = 64 * MB;               // rows of the tile
  __shared__ u32x4 As0[8 * kRows];
  __shared__ u32x4 As1[8 * kRows];
  __shared__ u32x4 Ws[2 * kBwChunks];
  u32x4* const Ws0 = Ws;
  u32x4* const Ws1 = Ws + kBwChunks;
  const int t = threadIdx.x, lane = t & 63;
  const int w = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = w >> 2, wn = w & 3;
  const int h = lane >> 5, l32 = lane & 31;
  const int ntm = static_cast<int>(cdiv(M, kRows)), ntk = static_cast<int>(cdiv(K, kTile));
  int tm, tk;
  const int split = kMulti ? __builtin_amdgcn_readfirstlane(static_cast<int>(blockIdx.x) / (ntm * ntk)) : 0;
  tile_of(blockIdx.x - split * ntm * ntk, ntm, ntk, tm, tk);
  tm = __builtin_amdgcn_readfirstlane(tm);
  tk = __builtin_amdgcn_readfirstlane(tk);
  const int64_t m0 = static_cast<int64_t>(tm) * kRows, k0 = static_cast<int64_t>(tk) * kTile;
  const int64_t nbr = K / 64;
  const int64_t nsteps = cdiv(N, 64), npairs = (nsteps + 1) / 2;
  const int64_t st0 = kMulti ? 2 * (npairs * split / ml.S) : 0;
  const int64_t st1 = kMulti ? 2 * (npairs * (split + 1) / ml.S) : nsteps;

  // dY tile staging through registers (not LDS DMA: the transposed LDS reads
  // of W' carry no alias information, so any LDS DMA in flight would make the
  // compiler wait for it before each of them). Thread t moves 16-byte chunk
  // t & 7 of rows (t >> 3) + 64 i: eight lanes cover a row's 128 bytes.
  // Buffer loads through a descriptor over this tile's dY rows: rows past M
  // read as zero without a branch. (Columns past N in the last step read the
  // next row; the matching weight rows are dead, so they contribute zero, except
  // with a pool, below.)
  const int ach = t & 7, arow0 = t >> 3;
  const int64_t rows_valid = imin(static_cast<int64_t>(kRows), M - m0);
  const __amdgpu_buffer_rsrc_t yr = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint16_t*>(dy + m0 * N), 0, static_cast<int>(rows_valid * N * 2), kBufferDword3);
  uint32_t aoff[MB];
#pragma unroll
  for (int i = 0; i < MB; ++i) aoff[i] = static_cast<uint32_t>((arow0 + 64 * i) * N * 2 + 16 * ach);
  const int alive = static_cast<int>(2 * N) - 16 * ach;      // bytes of a row from this thread's first chunk
  u32x4 areg[MB];
  auto load_a = [&](int64_t st) {
    const uint32_t so = static_cast<uint32_t>(imin(st, nsteps - 1) * 128);
    // a pool's rows are kept apart: columns past N read as zero (out of range),
    // or a NaN at the start of the next row would meet the zero weights
    const uint32_t dead = kMulti && static_cast<int>(so) >= alive ? 0x80000000u : 0u;
#pragma unroll
    for (int i = 0; i < MB; ++i)
      areg[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(yr, aoff[i] | dead, so, 0));
  };
  auto store_a = [&](u32x4* Ab) {
#pragma unroll
    for (int i = 0; i < MB; ++i) Ab[a_slot(arow0 + 64 * i, ach)] = areg[i];
  };
  // this thread decodes half bh = t >> 8 (columns 32 bh .. 32 bh + 31) of
  // 64-column block t & 3 of weight row (t >> 2) & 63 of the step
  const int brow = (t >> 2) & 63, bkb = t & 3, bh = t >> 8;
  const int64_t bkbi = imin(k0 / 64 + bkb, nbr - 1);
  auto load_codes = [&](int64_t st, BCodes& P) {
    const int64_t n = st * 64 + brow;
    const int64_t nc = imin(n, N - 1);
    P.p = ld16(packed + nc * (K / 2) + bkbi * 32 + 16 * bh);
    const int64_t blk = nc * nbr + bkbi;
    P.q = qscale[blk];
    P.d = step[blk >> 8];
    P.live = n < N ? 1.0f : 0.0f;
  };
  // W' tile slot of (row, 16-byte chunk c of the 256 columns). Within each
  // 8-chunk block the chunk is xor-ed with the block index: a decode write
  // phase (4 rows x the 4 blocks, same chunk) then covers all 64 banks once,
  // and a transposed read phase (4 rows x 4 aligned chunks of one block) still does.
  auto w_slot = [](int row, int c) { return row * kBwRow + (c ^ ((c >> 3) & 3)); };

  f32x16 acc[MB][2];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;

  // B-operand reads (ds_read_b64_tr_b16): lane group G = lane / 16 reads rows
  // 16 s + 8 (G >> 1) + 4 q + (j16 >> 2), 4 columns at 4 (j16 & 3) of the
  // 16-column half (G & 1) of the wave's 32-column block j
  const int G = lane >> 4, j16 = lane & 15;
  const int hh = G >> 1, cbh = G & 1;
  auto read_bj = [&](const u32x4* Wb, int s, int j) {
    const int col = 64 * wn + 32 * j + 16 * cbh + 4 * (j16 & 3);
    s16x4 v[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int row = 16 * s + 8 * hh + 4 * q + (j16 >> 2);
      v[q] = ds_read_tr(Wb, w_slot(row, col >> 3) * 8 + (col & 4));
    }
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7));
  };
  auto read_b = [&](const u32x4* Wb, int s, bf16x8 (&bf)[2]) {
#pragma unroll
    for (int j = 0; j < 2; ++j) bf[j] = read_bj(Wb, s, j);
  };
  auto read_a = [&](const u32x4* Ab, int s, bf16x8 (&af)[MB]) {
    const int sw = (2 * s + h) ^ a_swz(l32);       // a_swz(32 (MB wm + i) + l32) == a_swz(l32)
#pragma unroll
    for (int i = 0; i < MB; ++i) af[i] = as_bf16x8(Ab[(32 * (MB * wm + i) + l32) * 8 + sw]);
  };

  // one step: MFMAs on (Ab, Wb); decode `nx` into Wn; load dY tile st+1 and
  // write it into An in the last sub-step; load the codes of step st+2 into `ld`
  auto step_b = [&](const u32x4* Ab, u32x4* An, const u32x4* Wb, u32x4* Wn, const BCodes& nx, BCodes& ld,
                    int64_t st) {
    load_a(st + 1);
    __builtin_amdgcn_sched_barrier(0);
    load_codes(st + 2, ld);
    __builtin_amdgcn_sched_barrier(0);
    const MagTable tb = make_table(cb, block_scale(nx.q, nx.d) * nx.live);
    const uint32_t pw[4] = {nx.p.x, nx.p.y, nx.p.z, nx.p.w};
    bf16x8 af[2][MB], bf[2][2];
    read_a(Ab, 0, af[0]);
    read_b(Wb, 0, bf[0]);
    __builtin_amdgcn_sched_barrier(0);
    // Each sub-step is its own scheduling region, issued in this order: its
    // first MFMA (operands read during the previous sub-step), then per MFMA
    // one fragment read of the next sub-step and a share of the decode, then
    // its W' write (and in the last one the dY writes).
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      if (s < 3) {
        read_a(Ab, s + 1, af[(s + 1) & 1]);
        read_b(Wb, s + 1, bf[(s + 1) & 1]);
      }
#pragma unroll
      for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = mfma32(af[s & 1][i], bf[s & 1][j], acc[i][j]);
      Wn[w_slot(brow, 8 * bkb + 4 * bh + s)] = decode8(pw[s], tb);
      if (s == 3) store_a(An);
#pragma unroll
      for (int m = 0; m < 2 * MB; ++m) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        if (s < 3) __builtin_amdgcn_sched_group_barrier(0x100, MB == 4 ? 1 : MB == 2 ? 2 : 3, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, 12 / MB, 0);
      }
      if (s == 3)
        __builtin_amdgcn_sched_group_barrier(0x200, 1 + MB, 0);
      else
        __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // a pool's rows: asked for here, used in the epilogue
  TileRows tr;
  if constexpr (kMulti) tr.init(ml, m0, M < m0 + kRows ? M : m0 + kRows, lane);

  // prologue: dY tile 0, codes of steps 0 and 1; decode step 0
  BCodes P0, P1;
  load_a(st0);
  __builtin_amdgcn_sched_barrier(0);
  load_codes(st0, P0);
  __builtin_amdgcn_sched_barrier(0);
  load_codes(st0 + 1, P1);
  __builtin_amdgcn_sched_barrier(0);
  store_a(As0);
  asm volatile("" ::"v"(P1.p), "v"(static_cast<int>(P1.q)), "v"(P1.d));
  {
    const MagTable tb = make_table(cb, block_scale(P0.q, P0.d) * P0.live);
    const uint32_t pw[4] = {P0.p.x, P0.p.y, P0.p.z, P0.p.w};
#pragma unroll
    for (int c = 0; c < 4; ++c) Ws0[w_slot(brow, 8 * bkb + 4 * bh + c)] = decode8(pw[c], tb);
  }
  __syncthreads();
  // The end of step st waits for this wave's LDS writes (W' and dY of step
  // st+1), then the barrier publishes them; the code loads of step st+2 stay
  // in flight.
  for (int64_t st = st0; st < st1; st += 2) {
    step_b(As0, As1, Ws0, Ws1, P1, P0, st);
    __builtin_amdgcn_s_waitcnt(0xC07F);        // lgkmcnt(0)
    lds_barrier();
    step_b(As1, As0, Ws1, Ws0, P0, P1, st + 1);
    __builtin_amdgcn_s_waitcnt(0xC07F);
    lds_barrier();
  }
  wait_vm<0>();

  if constexpr (RSN > 0) {
    // The up-projection contracts over the ranks: its B operand is the r x 256
    // slice of A under this tile, staged row-major in the W' buffers (free
    // after the main loop; the same padded, swizzled rows) and read with the
    // main loop's transposed reads, rank chunk rs in place of sub-step s.
    // Ranks past r and columns past K are zero. RSN counts the rank chunks
    // of 16 that are used (1 for r <= 16: u's padding columns 16 .. 31 are
    // zero and skipped).
    static_assert(16 * 8 * kBwRow <= 2 * kBwChunks, "A's slice does not fit the W' buffers");
    auto stage_a = [&](const uint16_t* Aa) {
      // 16 RSN rows x 32 chunks of 8 columns (K % 64 == 0, so a chunk is
      // wholly inside or past K), all loads before the LDS writes
      constexpr int kPer = 16 * RSN * 32 / kBwThreads;
      u32x4 av[kPer];
#pragma unroll
      for (int u = 0; u < kPer; ++u) {
        const int e = t + kBwThreads * u, j = e >> 5, ch = e & 31;
        const int64_t kc = k0 + 8 * ch;
        av[u] = (j < r && kc < K) ? ld16(Aa + static_cast<int64_t>(j) * K + kc) : u32x4{0u, 0u, 0u, 0u};
      }
#pragma unroll
      for (int u = 0; u < kPer; ++u) {
        const int e = t + kBwThreads * u;
        Ws[w_slot(e >> 5, e & 31)] = av[u];
      }
    };
    // groups of IG row blocks: their u fragments are loaded before their
    // MFMAs; A's fragments read per column block
    auto lora = [&](auto rsn_c) {
      constexpr int RS = decltype(rsn_c)::value;
      constexpr int IG = RS <= 2 ? 4 : RS <= 4 ? 2 : 1;
#pragma unroll
      for (int i0 = 0; i0 < 4; i0 += IG) {
        u32x4 uf[IG][RS];
#pragma unroll
        for (int ii = 0; ii < IG; ++ii) {
          const int64_t mrow = imin(m0 + 128 * wm + 32 * (i0 + ii) + l32, M - 1);
#pragma unroll
          for (int rs = 0; rs < RS; ++rs) uf[ii][rs] = ld16(ul + mrow * rp + 16 * rs + 8 * h);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          bf16x8 bl[RS];
#pragma unroll
          for (int rs = 0; rs < RS; ++rs) bl[rs] = read_bj(Ws, rs, j);
#pragma unroll
          for (int ii = 0; ii < IG; ++ii) {
            f32x16 tmp;
#pragma unroll
            for (int v = 0; v < 16; ++v) tmp[v] = 0.f;
#pragma unroll
            for (int rs = 0; rs < RS; ++rs) tmp = mfma32(as_bf16x8(uf[ii][rs]), bl[rs], tmp);
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i0 + ii][j][v] += scale * tmp[v];
          }
        }
      }
    };
    // a pool of adapters: every adapter among the tile's rows in turn (the
    // same order in every wave), its slice of A staged by the whole workgroup;
    // straight-line code over the wave's blocks, so that the accumulators
    // stay where they are. u carries the scale.
    auto lora_multi = [&](auto rsn_c) {
      constexpr int RS = decltype(rsn_c)::value;
      uint64_t pend[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) pend[q] = __ballot(tr.id[q] >= 0);
      // u of the wave's rows once, where it fits the registers
      constexpr bool kKeep = RS <= 2;
      u32x4 uf[kKeep ? MB : 1][RS];
      auto load_u = [&](int i, u32x4 (&f)[RS]) {
        const int64_t mrow = imin(m0 + 32 * (MB * wm + i) + l32, M - 1);
#pragma unroll
        for (int rs = 0; rs < RS; ++rs) f[rs] = ld16(ul + mrow * rp + 16 * rs + 8 * h);
      };
      if constexpr (kKeep) {
#pragma unroll
        for (int i = 0; i < MB; ++i) load_u(i, uf[i]);
      }
      for (int ord = 0; pend[0] | pend[1] | pend[2] | pend[3]; ++ord) {
        const int a = pend[0]   ? __builtin_amdgcn_readlane(tr.id[0], __builtin_ctzll(pend[0]))
                      : pend[1] ? __builtin_amdgcn_readlane(tr.id[1], __builtin_ctzll(pend[1]))
                      : pend[2] ? __builtin_amdgcn_readlane(tr.id[2], __builtin_ctzll(pend[2]))
                                : __builtin_amdgcn_readlane(tr.id[3], __builtin_ctzll(pend[3]));
        uint64_t rows[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          rows[q] = __ballot(tr.id[q] == a);
          pend[q] &= ~rows[q];
        }
        if (ord % ml.S != split) continue;
        __syncthreads();                       // the reads of the slice before (or of the last W' tile)
        stage_a(Al + static_cast<int64_t>(a) * r * K);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < MB; ++i) {
          // block MB wm + i of the tile
          const uint64_t two = rows[i >> 1], two1 = rows[(MB + i) >> 1];
          const uint32_t rm = static_cast<uint32_t>(wm ? two1 >> (32 * ((MB + i) & 1)) : two >> (32 * (i & 1)));
          if constexpr (!kKeep) load_u(i, uf[0]);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            f32x16 p, tmp;
#pragma unroll
            for (int v = 0; v < 16; ++v) p[v] = tmp[v] = 0.f;
#pragma unroll
            for (int rs = 0; rs < RS; ++rs) p = mfma32(as_bf16x8(uf[kKeep ? i : 0][rs]), read_bj(Ws, rs, j), p);
            take_rows(tmp, p, rm, h);
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] += tmp[v];
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    };
    if constexpr (kMulti) {
      lora_multi(std::integral_constant<int, RSN>{});
    } else {
      __syncthreads();
      stage_a(Al);
      __syncthreads();
      lora(std::integral_constant<int, RSN>{});
    }
  }
  if constexpr (kMulti) {
    if (ml.S > 1) {
      float* const pt = ml.part + (split * M + m0 + 32 * MB * wm) * K + k0 + 64 * wn + l32;
#pragma unroll
      for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int v = 0; v < 16; ++v) {
            const int row = 32 * i + 8 * (v >> 2) + 4 * h + (v & 3);
            if (m0 + 32 * MB * wm + row < M && k0 + 64 * wn + 32 * j + l32 < K) pt[row * K + 32 * j] = acc[i][j][v];
          }
      return;
    }
  }
  if (m0 + kRows <= M && k0 + kTile <= K) {
    uint16_t* dt = dx + (m0 + 32 * MB * wm + 4 * h) * K + k0 + 64 * wn + l32;
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v)
          dt[(32 * i + 8 * (v >> 2) + (v & 3)) * K + 32 * j] = bf16_bits(acc[i][j][v]);
  } else {
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int64_t kk = k0 + 64 * wn + 32 * j + l32;
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const int64_t mm = m0 + 32 * (MB * wm + i) + 8 * (v >> 2) + 4 * h + (v & 3);
          if (mm < M && kk < K) dx[mm * K + kk] = bf16_bits(acc[i][j][v]);
        }
      }
  }
}

// ---------------------------------------------------------------------------
// dispatch: LoRA down-projection, then the small-M or the tiled kernel
// ---------------------------------------------------------------------------
// The tiled forward over a table of up to kFwdMaxWeights weights at one M:
// the LoRA down-projection of each weight into its own workspace slice (one
// launch each), then one launch of k_gemm_fwd for all of them. Weight i's
// workspace is ws + i * ws_stride (its layout ws_layout(0, M, N[i], K[i], r)).
static hipError_t launch_fwd_tiled(int64_t M, int G, const uint16_t* const* x, const int64_t* N, const int64_t* K,
                                   const uint8_t* const* packed, const int8_t* const* qscale,
                                   const float* const* step, const uint16_t* const* A, const uint16_t* const* B,
                                   int r, float alpha, uint16_t* const* y, void* ws, size_t ws_stride,
                                   const Codebook& cb, hipStream_t stream) {
  const float scale = r > 0 ? alpha / static_cast<float>(r) : 0.0f;
  const int rp = r > 0 ? static_cast<int>(rank_pad(r)) : 0;
  FwdTable tab{};
  tab.count = G;
  bool quad = true;
  int cols = 0;
  for (int i = 0; i < G; ++i) {
    const WsLayout L = ws_layout(0, M, N[i], K[i], r);
    char* wsb = static_cast<char*>(ws) + static_cast<size_t>(i) * ws_stride;
    void* lora = r > 0 ? static_cast<void*>(wsb + L.lora_off) : nullptr;
    if (r > 0) {
      const hipError_t e = launch_lora_down(true, x[i], M, K[i], A[i], r, lora, stream, nullptr,
                                            reinterpret_cast<float*>(wsb + L.dp_off));
      if (e != hipSuccess) return e;
    }
    tab.x[i] = x[i];
    tab.packed[i] = packed[i];
    tab.qscale[i] = qscale[i];
    tab.step[i] = step[i];
    tab.tl[i] = static_cast<const uint16_t*>(lora);
    tab.B[i] = r > 0 ? B[i] : nullptr;
    tab.y[i] = y[i];
    tab.N[i] = static_cast<int>(N[i]);
    tab.K[i] = static_cast<int>(K[i]);
    tab.col0[i] = cols;
    cols += static_cast<int>(cdiv(N[i], kTile));
    quad = quad && K[i] % 256 == 0;
  }
  tab.col0[G] = cols;
  const int64_t tiles = cdiv(M, kTile) * cols;
#define QNF4_FWD(RSNV)                                                                                          \
  do {                                                                                                         \
    if (quad)                                                                                                  \
      hipLaunchKernelGGL(HIP_KERNEL_NAME(k_gemm_fwd<true, RSNV>), dim3(static_cast<unsigned>(tiles)), dim3(256), \
                         0, stream, tab, M, rp, r, scale, cb, MultiLora{});                                                 \
    else                                                                                                       \
      hipLaunchKernelGGL(HIP_KERNEL_NAME(k_gemm_fwd<false, RSNV>), dim3(static_cast<unsigned>(tiles)),          \
                         dim3(256), 0, stream, tab, M, rp, r, scale, cb, MultiLora{});                                      \
  } while (0)
  mark_kernel(0, stream);
  switch (r == 0 ? 0 : r <= 16 ? 1 : rp / 16) {
    case 0: QNF4_FWD(0); break;
    case 1: QNF4_FWD(1); break;
    case 2: QNF4_FWD(2); break;
    case 4: QNF4_FWD(4); break;
    case 6: QNF4_FWD(6); break;
    default: QNF4_FWD(8); break;
  }
#undef QNF4_FWD
  mark_kernel(1, stream);
  return hipGetLastError();
}

hipError_t launch_lora_fwd(const uint16_t* x, int64_t M, int64_t N, int64_t K, const uint8_t* packed,
                           const int8_t* qscale, const float* step, const uint16_t* A, const uint16_t* B,
                           int r, float alpha, uint16_t* y, void* ws, const Codebook& cb,
                           hipStream_t stream) {
  if (M <= kSmallM)
    return launch_dec_fwd(M, 1, &x, &N, &K, &packed, &qscale, &step, &A, &B, r, alpha, &y, ws, cb, stream);
  return launch_fwd_tiled(M, 1, &x, &N, &K, &packed, &qscale, &step, &A, &B, r, alpha, &y, ws, 0, cb, stream);
}

// Tiled batches go in chunks of kFwdMaxWeights, each weight with a workspace
// slice of the largest single-weight size in the batch.
static size_t tiled_stride(int64_t M, int G, const int64_t* N, const int64_t* K, int r) {
  size_t need = 0;
  for (int i = 0; i < G; ++i) {
    const size_t b = align256(ws_layout(0, M, N[i], K[i], r).total);
    need = b > need ? b : need;
  }
  return need;
}

size_t batched_ws_bytes(int64_t M, int G, const int64_t* N, const int64_t* K, int r) {
  if (M <= kSmallM) return dec_workspace_bytes(M, G, N, K);
  const int per_launch = G < kFwdMaxWeights ? G : kFwdMaxWeights;
  return tiled_stride(M, G, N, K, r) * static_cast<size_t>(per_launch);
}

hipError_t launch_lora_fwd_batched(int64_t M, int G, const uint16_t* const* x, const int64_t* N, const int64_t* K,
                                   const uint8_t* const* packed, const int8_t* const* qscale,
                                   const float* const* step, const uint16_t* const* A, const uint16_t* const* B,
                                   int r, float alpha, uint16_t* const* y, void* ws, const Codebook& cb,
                                   hipStream_t stream) {
  if (M <= kSmallM) return launch_dec_fwd(M, G, x, N, K, packed, qscale, step, A, B, r, alpha, y, ws, cb, stream);
  const size_t stride = tiled_stride(M, G, N, K, r);
  for (int c0 = 0; c0 < G; c0 += kFwdMaxWeights) {
    const int cn = G - c0 < kFwdMaxWeights ? G - c0 : kFwdMaxWeights;
    const hipError_t e = launch_fwd_tiled(M, cn, x + c0, N + c0, K + c0, packed + c0, qscale + c0, step + c0,
                                          r ? A + c0 : nullptr, r ? B + c0 : nullptr, r, alpha, y + c0, ws, stride,
                                          cb, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_bwd_dx(const uint16_t* dy, int64_t M, int64_t N, int64_t K, const uint8_t* packed,
                         const int8_t* qscale, const float* step, const uint16_t* A, const uint16_t* B,
                         int r, float alpha, uint16_t* dx, void* ws, const Codebook& cb,
                         hipStream_t stream) {
  // small M: the down-projection u = dY . B is computed inside k_dec_bwd
  if (M <= kSmallM)
    return launch_dec_bwd(M, 1, &dy, &N, &K, &packed, &qscale, &step, &A, &B, r, alpha, &dx, ws, cb, stream);
  const WsLayout L = ws_layout(1, M, N, K, r);
  char* wsb = static_cast<char*>(ws);
  const float scale = r > 0 ? alpha / static_cast<float>(r) : 0.0f;
  const int rp = r > 0 ? static_cast<int>(rank_pad(r)) : 0;
  void* lora = r > 0 ? static_cast<void*>(wsb + L.lora_off) : nullptr;
  if (r > 0) {
    const hipError_t e = launch_lora_down(false, dy, M, N, B, r, lora, stream,
                                          reinterpret_cast<uint16_t*>(wsb + L.bt_off),
                                          reinterpret_cast<float*>(wsb + L.dp_off));
    if (e != hipSuccess) return e;
  }
  const int64_t tiles = cdiv(M, kTile) * cdiv(K, kTile);
#define QNF4_BWD(RSNV)                                                                                         \
  hipLaunchKernelGGL(HIP_KERNEL_NAME(k_gemm_bwd<RSNV>), dim3(static_cast<unsigned>(tiles)), dim3(kBwThreads), 0, \
                     stream,                                                                                  \
                     dy, M, N, K, packed, qscale, step, static_cast<const uint16_t*>(lora), rp, A, r, scale, dx, cb, \
                     MultiLora{})
  mark_kernel(0, stream);
  switch (r == 0 ? 0 : r <= 16 ? 1 : rp / 16) {
    case 0: QNF4_BWD(0); break;
    case 1: QNF4_BWD(1); break;
    case 2: QNF4_BWD(2); break;
    case 4: QNF4_BWD(4); break;
    case 6: QNF4_BWD(6); break;
    default: QNF4_BWD(8); break;
  }
#undef QNF4_BWD
  mark_kernel(1, stream);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// a pool of adapters: t or u of every row (launch_multi_down), then the
// streaming forward, or the tiled GEMM with the row-by-row epilogue
// ---------------------------------------------------------------------------
// out[i] = bf16(sum of the S partials of element i, in order), 8 per thread;
// count is a multiple of 8 or the rest goes one by one
__global__ __launch_bounds__(256) void k_split_sum(const float* __restrict__ part, int S, int64_t count,
                                                   uint16_t* __restrict__ out) {
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 8;
  if (i >= count) return;
  if (i + 8 <= count && count % 4 == 0) {
    f32x4 a = *reinterpret_cast<const f32x4*>(part + i), b = *reinterpret_cast<const f32x4*>(part + i + 4);
    for (int s = 1; s < S; ++s) {
      a += *reinterpret_cast<const f32x4*>(part + s * count + i);
      b += *reinterpret_cast<const f32x4*>(part + s * count + i + 4);
    }
    *reinterpret_cast<u32x4*>(out + i) = u32x4{pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]),
                                               pack_bf16x2(b[0], b[1]), pack_bf16x2(b[2], b[3])};
    return;
  }
  for (int64_t e = i; e < i + 8 && e < count; ++e) {
    float sum = part[e];
    for (int s = 1; s < S; ++s) sum += part[s * count + e];
    out[e] = bf16_bits(sum);
  }
}

// How a call of op 0 (forward, contraction over K) or 1 (backward, over N) runs.
// The contraction of the tiled kernels is split while the tiles leave CUs
// idle, into S ranges of at least two super-steps (forward, 256 deep) or 2 MB
// steps (backward, 64 deep); the backward's tile has 256, 128 or 64 rows (MB 4,
// 2, 1). The time of each way, in us, from the shapes measured:
//   tiled      ranges of 64-deep steps (forward 1.4 each; backward 1.3, 0.75,
//              0.55 by tile), 8 to start and end, and the partial sums written and
//              read at 4 TB/s and another launch
//   streaming  rounds of items; an item is 9 and 2.8 per super-step of a wave
// e.g. forward, 700 rows at 4096 x 11008: streaming 127 (3 rounds), tiled in five
// ranges 88; 256 rows at 4096 x 4096: streaming 24, tiled 38. Backward at 4096 x
// 4096, tiles of 256 / 128 / 64 rows at their best S: 64 rows 28.5 / 23.5 / 21.4,
// 128 rows 32.8 / 25.2 / 25.5, 321 rows 35.6 / 32.1 / 98, 600 rows 47 / 60 / 100:
// hence 64-row tiles up to 64 rows, 128-row ones up to 384.
struct MultiPlan {
  bool one = false, stream = false;
  int MB = 4;                                   // backward: 32-row blocks per wave, 64 MB rows per tile
  int64_t S = 1;
  size_t t_off = 0, down_off = 0, part_off = 0, total = 0;   // the tiled kernels' workspace
};
static MultiPlan multi_plan(int op, int64_t M, int64_t N, int64_t K, int r, int n) {
  MultiPlan p;
  const int64_t Kc = op == 0 ? K : N, cols = op == 0 ? N : K;
  const int64_t steps = cdiv(Kc, 64);
  // One launch for up to four rows, while the adapters that every block of 64
  // weight rows reads again (min(n, M) of them at most: the index is on the
  // device) cost less than the second launch: one row r 16 / 64 at 4096 x 4096
  // (8 / 34 MB) 11.0 / 15.2 us against 17.9 / 22.3 in two launches, r 16 at 11008 x
  // 4096 (23 MB) 21.9 against 24.3; four rows of four adapters there (90 MB) 32.9
  // against 24.9, at r 64 (361 MB) 75 against 30.
  if (op == 0 && M <= kMoMaxM && cdiv(N, 64) * std::min<int64_t>(n, M) * 16 * down_nt(r) * K * 2 <= 72000000) {
    p.one = true;
    p.total = kWsCounterBytes + mo_plan(M, N, K).part_bytes;
    return p;
  }
  p.MB = op == 0 || M > 384 ? 4 : M > 64 ? 2 : 1;
  const int64_t tiles = cdiv(M, 64 * p.MB) * cdiv(cols, kTile);
  const double step_us = op == 0 ? 1.4 : p.MB == 4 ? 1.3 : p.MB == 2 ? 0.75 : 0.55;
  double best = 0;
  for (int64_t S = 1; S <= kMultiMaxSplit && (S == 1 || (S * tiles <= 256 && steps / S >= 2 * p.MB)); ++S) {
    double us = static_cast<double>(cdiv(S * tiles, 256)) * (step_us * 4 * cdiv(cdiv(steps, 4), S) + 8);
    if (S > 1) us += 4 + 8e-6 * static_cast<double>(S * M * cols) / 4;
    if (S == 1 || us < best) best = us, p.S = S;
  }
  if (op == 0 && M <= kMsMaxM) {
    const MsPlan m = ms_plan(M, N, K, r, n);
    const int64_t items = cdiv(N, 64) * m.mblocks * m.S;
    const double us = static_cast<double>(cdiv(items, 256)) * (9 + 2.8 * cdiv(cdiv(K, 256), 4 * m.S));
    if (us <= best) {
      p.stream = true;
      p.total = m.total;
      return p;
    }
  }
  p.t_off = kWsCounterBytes;
  p.down_off = p.t_off + align256(static_cast<size_t>(M * rank_pad(r) * 2));
  p.part_off = p.down_off + multi_down_plan(M, Kc, r, n).part_bytes;
  p.total = p.part_off + (p.S > 1 ? align256(static_cast<size_t>(p.S * M * cols) * 4) : 0);
  return p;
}

size_t multi_ws_bytes(int op, int64_t M, int64_t N, int64_t K, int r, int n) {
  return op == 2 ? multi_grad_plan(M, N, K, r, n, true).total : multi_plan(op, M, N, K, r, n).total;
}

static hipError_t launch_split_sum(const MultiLora& ml, int64_t count, uint16_t* out, hipStream_t stream) {
  if (ml.S > 1)
    hipLaunchKernelGGL(k_split_sum, dim3(static_cast<unsigned>(cdiv(count, 2048))), dim3(256), 0, stream, ml.part, ml.S,
                       count, out);
  return hipGetLastError();
}

hipError_t launch_multi_fwd(const uint16_t* x, int64_t M, int64_t N, int64_t K, const uint8_t* packed,
                            const int8_t* qscale, const float* step, const uint16_t* A, const uint16_t* B,
                            const int* index, const float* scale, int n, int r, uint16_t* y, void* ws,
                            const Codebook& cb, hipStream_t stream) {
  const MultiPlan p = multi_plan(0, M, N, K, r, n);
  char* wsb = static_cast<char*>(ws);
  const MultiLora ml{index, scale, n, static_cast<int>(p.S), reinterpret_cast<float*>(wsb + p.part_off)};
  if (p.one)
    return launch_mone(mo_plan(M, N, K), x, M, N, K, packed, qscale, step, A, B, ml, r, y, ws, cb, stream);
  if (p.stream)
    return launch_mstream(ms_plan(M, N, K, r, n), x, M, N, K, packed, qscale, step, A, B, ml, r, y, ws, cb, stream);
  uint16_t* tl = reinterpret_cast<uint16_t*>(wsb + p.t_off);
  const hipError_t e = launch_multi_down(true, x, M, K, A, ml, r, tl, ws, reinterpret_cast<float*>(wsb + p.down_off),
                                         stream);
  if (e != hipSuccess) return e;
  const int rp = static_cast<int>(rank_pad(r));
  FwdTable tab{};
  tab.count = 1;
  tab.x[0] = x;
  tab.packed[0] = packed;
  tab.qscale[0] = qscale;
  tab.step[0] = step;
  tab.tl[0] = tl;
  tab.B[0] = B;
  tab.y[0] = y;
  tab.N[0] = static_cast<int>(N);
  tab.K[0] = static_cast<int>(K);
  tab.col0[1] = static_cast<int>(cdiv(N, kTile));
  const dim3 grid(static_cast<unsigned>(cdiv(M, kTile) * cdiv(N, kTile) * p.S));
#define QNF4_MFWD(RSNV)                                                                                        \
  do {                                                                                                         \
    if (K % 256 == 0)                                                                                          \
      hipLaunchKernelGGL(HIP_KERNEL_NAME(k_gemm_fwd<true, RSNV, true>), grid, dim3(256), 0, stream, tab, M, rp, r, \
                         0.0f, cb, ml);                                                                        \
    else                                                                                                       \
      hipLaunchKernelGGL(HIP_KERNEL_NAME(k_gemm_fwd<false, RSNV, true>), grid, dim3(256), 0, stream, tab, M, rp, r, \
                         0.0f, cb, ml);                                                                        \
  } while (0)
  mark_kernel(0, stream);
  switch (r <= 16 ? 1 : rp / 16) {
    case 1: QNF4_MFWD(1); break;
    case 2: QNF4_MFWD(2); break;
    case 4: QNF4_MFWD(4); break;
    case 6: QNF4_MFWD(6); break;
    default: QNF4_MFWD(8); break;
  }
#undef QNF4_MFWD
  mark_kernel(1, stream);
  return launch_split_sum(ml, M * N, y, stream);
}

hipError_t launch_multi_bwd(const uint16_t* dy, int64_t M, int64_t N, int64_t K, const uint8_t* packed,
                            const int8_t* qscale, const float* step, const uint16_t* A, const uint16_t* B,
                            const int* index, const float* scale, int n, int r, uint16_t* dx, void* ws,
                            const Codebook& cb, hipStream_t stream) {
  const MultiPlan p = multi_plan(1, M, N, K, r, n);
  char* wsb = static_cast<char*>(ws);
  const MultiLora ml{index, scale, n, static_cast<int>(p.S), reinterpret_cast<float*>(wsb + p.part_off)};
  uint16_t* ul = reinterpret_cast<uint16_t*>(wsb + p.t_off);
  const hipError_t e = launch_multi_down(false, dy, M, N, B, ml, r, ul, ws, reinterpret_cast<float*>(wsb + p.down_off),
                                         stream);
  if (e != hipSuccess) return e;
  const int rp = static_cast<int>(rank_pad(r));
  const dim3 grid(static_cast<unsigned>(cdiv(M, 64 * p.MB) * cdiv(K, kTile) * p.S));
#define QNF4_MBWD1(RSNV, MBV)                                                                                 \
  hipLaunchKernelGGL(HIP_KERNEL_NAME(k_gemm_bwd<RSNV, true, MBV>), grid, dim3(kBwThreads), 0, stream, dy, M, N, K, packed, \
                     qscale, step, static_cast<const uint16_t*>(ul), rp, A, r, 0.0f, dx, cb, ml)
#define QNF4_MBWD(RSNV)                     \
  do {                                      \
    if (p.MB == 4) QNF4_MBWD1(RSNV, 4);     \
    else if (p.MB == 2) QNF4_MBWD1(RSNV, 2); \
    else QNF4_MBWD1(RSNV, 1);               \
  } while (0)
  mark_kernel(0, stream);
  switch (r <= 16 ? 1 : rp / 16) {
    case 1: QNF4_MBWD(1); break;
    case 2: QNF4_MBWD(2); break;
    case 4: QNF4_MBWD(4); break;
    case 6: QNF4_MBWD(6); break;
    default: QNF4_MBWD(8); break;
  }
#undef QNF4_MBWD
#undef QNF4_MBWD1
  mark_kernel(1, stream);
  return launch_split_sum(ml, M * K, dx, stream);
}

size_t bwd_batched_ws_bytes(int64_t M, int G, const int64_t* N, const int64_t* K, int r) {
  if (M <= kSmallM) return dec_bwd_workspace_bytes(M, G, N, K);
  size_t most = 0;                           // the tiled calls run one after another on one workspace
  for (int i = 0; i < G; ++i) {
    const size_t b = ws_layout(1, M, N[i], K[i], r).total;
    if (b > most) most = b;
  }
  return most;
}

hipError_t launch_bwd_dx_batched(int64_t M, int G, const uint16_t* const* dy, const int64_t* N, const int64_t* K,
                                 const uint8_t* const* packed, const int8_t* const* qscale,
                                 const float* const* step, const uint16_t* const* A, const uint16_t* const* B,
                                 int r, float alpha, uint16_t* const* dx, void* ws, const Codebook& cb,
                                 hipStream_t stream) {
  if (M <= kSmallM) return launch_dec_bwd(M, G, dy, N, K, packed, qscale, step, A, B, r, alpha, dx, ws, cb, stream);
  for (int i = 0; i < G; ++i) {
    const hipError_t e = launch_bwd_dx(dy[i], M, N[i], K[i], packed[i], qscale[i], step[i], r ? A[i] : nullptr,
                                       r ? B[i] : nullptr, r, alpha, dx[i], ws, cb, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace qnf4
