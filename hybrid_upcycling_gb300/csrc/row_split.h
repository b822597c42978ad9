// How a row of logits is shared out over the CTAs of a cluster: plain arithmetic, for the host and the device.
//
// A row is `blocks` blocks of 32 vectors. Its groups (whose maxima are kept for the alternatives) are 2^vec_shift vectors
// each. A CTA takes `span` consecutive blocks: whole groups and whole warp loads of four blocks, so that no word and no group
// belongs to two CTAs. The last CTAs may have no blocks at all.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define HYLO_HD __host__ __device__ __forceinline__
#else
#define HYLO_HD inline
#endif

namespace hylo {

struct RowPart {
  int blk0, blk1;  // its blocks
  int g0, g1;      // its groups
};

HYLO_HD int row_span(int64_t blocks, int ctas, int vec_shift) {
  const int64_t unit = vec_shift > 7 ? int64_t(1) << (vec_shift - 5) : 4;
  return static_cast<int>(((blocks + ctas - 1) / ctas + unit - 1) / unit * unit);
}

// CTA q's part of a row of `blocks` blocks. A CTA without blocks has no groups: the row's end may lie inside a group, which is
// the CTA's that has its first block.
HYLO_HD RowPart row_part(int blocks, int span, int q, int vec_shift) {
  RowPart r;
  const int64_t first = static_cast<int64_t>(q) * span;
  r.blk0 = first < blocks ? static_cast<int>(first) : blocks;
  r.blk1 = blocks - r.blk0 < span ? blocks : r.blk0 + span;
  const int per = vec_shift < 5 ? 5 - vec_shift : 0, down = vec_shift > 5 ? vec_shift - 5 : 0;
  r.g0 = (r.blk0 << per) >> down;
  r.g1 = r.blk0 < r.blk1 ? ((r.blk1 << per) + (1 << down) - 1) >> down : r.g0;
  return r;
}

}  // namespace hylo
