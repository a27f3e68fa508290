// The streaming forward of a pool of adapters (mstream.hip) and what it shares
// with the products before it (multi.hip).
#pragma once

#include "device.hpp"
#include "kernels.hpp"

namespace qnf4 {

constexpr int64_t kMsMaxM = 1024;                // rows the streaming forward takes
constexpr int64_t kMultiMaxSplit = 16;          // ranges of a split contraction at most (tiled kernels)
constexpr int kMsMaxSplit = 4;                   // ranges of K at most

struct MsPlan {
  int MT = 1;                                    // 16-row tiles of x per item
  int64_t mblocks = 1, S = 1;
  size_t t_off = 0, x_off = 0, down_off = 0, part_off = 0, total = 0;
};
constexpr int64_t kMoMaxM = 4;                   // rows the one-launch forward takes
struct MoPlan {
  int64_t blocks = 1, S = 1;                     // blocks of 64 weight rows, ranges of K
  size_t part_bytes = 0;
};
MoPlan mo_plan(int64_t M, int64_t N, int64_t K);
hipError_t launch_mone(const MoPlan& p, const uint16_t* x, int64_t M, int64_t N, int64_t K, const uint8_t* packed,
                       const int8_t* qscale, const float* step, const uint16_t* A, const uint16_t* B,
                       const MultiLora& ml, int r, uint16_t* y, void* ws, const Codebook& cb, hipStream_t stream);
MsPlan ms_plan(int64_t M, int64_t N, int64_t K, int r, int n);
hipError_t launch_mstream(const MsPlan& p, const uint16_t* x, int64_t M, int64_t N, int64_t K, const uint8_t* packed,
                          const int8_t* qscale, const float* step, const uint16_t* A, const uint16_t* B,
                          const MultiLora& ml, int r, uint16_t* y, void* ws, const Codebook& cb, hipStream_t stream);

// t = bf16(s_a x . A_a^T) (wrow: in = x, Kc = K, W = A) or u = bf16(s_a dY . B_a)
// (in = dY, Kc = N, W = B) of every row with an adapter: bf16 [M][rank_pad(r)].
// ws: the workspace (its counters); part: multi_down_plan().part_bytes of it.
// frags (wrow): `in` copied into MFMA order too, `mtiles` tiles of 16 rows.
constexpr int kMdMaxSplit = 16;
struct MultiDownPlan {
  int64_t RM = 1, blocks = 0, Q = 1, Smax = 1;   // 16-row tiles per block, blocks, workgroups of a block, ranges at most
  size_t part_bytes = 0;
};
MultiDownPlan multi_down_plan(int64_t M, int64_t Kc, int r, int n);
hipError_t launch_multi_down(bool wrow, const uint16_t* in, int64_t M, int64_t Kc, const uint16_t* W,
                             const MultiLora& ml, int r, uint16_t* out, void* ws, float* part, hipStream_t stream,
                             u32x4* frags = nullptr, int64_t mtiles = 0);

}  // namespace qnf4
