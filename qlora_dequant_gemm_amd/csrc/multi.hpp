// The streaming forward of a pool of adapters (mstream.hip) and what it shares
// with the products before it (multi.hip).
#pragma once

#include "device.hpp"
#include "kernels.hpp"

namespace qnf4 {

constexpr int64_t kMsMaxM = 1024;                // rows the streaming forward takes
constexpr int kMsMaxSplit = 4;                   // ranges of K at most

struct MsPlan {
  int MT = 1;                                    // 16-row tiles of x per item
  int64_t mblocks = 1, S = 1;
  size_t t_off = 0, x_off = 0, part_off = 0, total = 0;
};
MsPlan ms_plan(int64_t M, int64_t N, int64_t K, int r);
hipError_t launch_mstream(const MsPlan& p, const uint16_t* x, int64_t M, int64_t N, int64_t K, const uint8_t* packed,
                          const int8_t* qscale, const float* step, const uint16_t* A, const uint16_t* B,
                          const MultiLora& ml, int r, uint16_t* y, void* ws, const Codebook& cb, hipStream_t stream);

// t = bf16(s_a x . A_a^T) (wrow: in = x, Kc = K, W = A) or u = bf16(s_a dY . B_a)
// (in = dY, Kc = N, W = B) of every row with an adapter: bf16 [M][rank_pad(r)].
// frags (wrow): `in` copied into MFMA order too, `mtiles` tiles of 16 rows.
hipError_t launch_multi_down(bool wrow, const uint16_t* in, int64_t M, int64_t Kc, const uint16_t* W,
                             const MultiLora& ml, int r, uint16_t* out, hipStream_t stream, u32x4* frags = nullptr,
                             int64_t mtiles = 0);

}  // namespace qnf4
