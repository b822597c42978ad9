// Shared by the host side and the kernels of the orthogonalised updates (muon.cu, muon_pipe.cu): the layout of a group of
// matrices in the workspace.
//
// A group's matrices live in the workspace as fp16 in panels of 64 columns: element (r, c) of a matrix whose panels have `mp`
// rows, with `base` its first row of 128 bytes, lies in row base + (c / 64) mp + r, column c % 64. So the whole workspace is
// one tensor of 64 columns for the TMA loads, and a block of 64 rows and 64 columns, 8 KiB in one piece, serves as an operand
// whose rows are summed over as well as one whose columns are. X has at most as many rows as columns (a tall matrix is
// transposed) and is padded with zeros to multiples of 64, which stay zero in every product. Tiles reach to multiples of 256; what
// lies there is neither written nor has a part in any other row or column.
#pragma once

#include <cstdint>

#include "hylo_internal.h"

namespace hylo {

constexpr int kMuonMats = 64;     // matrices of a group at most
constexpr int kMuonParts = 1024;  // partial sums of squares of a matrix at most
constexpr int kMuonSums = 3;      // of magnitudes near 2^-80, 1 and 2^80

constexpr int kMuonStepsMax = 32;

// X's second term lies in the order in which the epilogue's lanes take it: [256 x 256 tile][CTA of the pair: 128 rows][warp: 32
// rows (warp % 4) and 128 columns (warp / 4)][32 columns][16 columns][row], in sectors of 32 bytes (16 columns).
constexpr int kMuonLoUnits = 4;
__host__ __device__ constexpr int64_t muon_lo_sector(int tile, int rank, int warp) {
  return ((static_cast<int64_t>(tile) * 2 + rank) * 8 + warp) * (kMuonLoUnits * 2 * 32);
}

// One matrix of a group.
struct MuonMat {
  const void* src;  // the matrix (orthogonalize) or the gradient
  int64_t ld;       // its row stride
  float* mom;       // momentum
  void* dst;        // the result, or the parameter
  float* master;
  uint64_t pos;     // position of element 0 in the list (random bits)
  float decay, step;  // w <- decay w - step O
  int rows, cols;
  int mt, nt;       // X is [m, n], m <= n (the matrix, or its transpose if tall): 256-row and 256-column tiles
  int kn, km;       // 64-deep k-blocks of n and m
  int tall, src_vec, dst_vec;
  uint32_t x[2], lo, a, b;  // first 128-byte rows of X before even and odd steps, its second term, A and B
  uint32_t sum0, parts;     // first partial sum, and how many
  uint32_t fill0;           // first thread block of the kernel that fills X
  int item0[3];             // first work items, among the group's, of each product (before they are halved)
  int splits, split0, part0;  // parts of the sum of an item of Gram; its first tile, and part, among the group's split ones
};
struct MuonTable {
  MuonMat t[kMuonMats];
  int count;
};

// Products are summed by the tensor cores over at most this many 64-deep k-blocks at a time.
constexpr int kMuonDepth = 128;
constexpr int64_t kMuonScratch = int64_t(128) * 256 * 4;  // bytes of a CTA's fp32 sums in between

enum : int { kMuonGram = 0, kMuonPoly = 1, kMuonApply = 2 };
enum : int { kMuonOutBf16 = 0, kMuonOutF16, kMuonParamF32, kMuonParamBf16, kMuonParamMaster };  // what the last product writes
struct MuonPipe {
  int steps;
  int items[3];             // work items of the group for each product: 256 x 256 tiles, of Gram times its splits
  int half[3];              // 1: work items of 256 x 128, so that there are twice as many
  float acc[kMuonStepsMax][3], add[kMuonStepsMax][3];  // factors on the sum of products, and on A (Poly) or X (Apply)
  unsigned* ctrl;           // [0] work queue, [1 + matrix] work done, then [split tile][16 warps] parts done; zero at launch
  uint8_t* parts;           // sums of split items [split items][2 CTAs][8 warps][16 KiB], as fp32 in the order of the lanes
  uint8_t* scratch;         // kMuonScratch bytes for each CTA, where some sum is longer than kMuonDepth
  WaitCtl ctl;
};
constexpr int kMuonCtrlWords = 1 + kMuonMats;  // before the split tiles'

struct MuonHyper {
  int muon;        // momentum and parameters, not just the matrices
  int nesterov;
  float mu, one_minus_mu;
  float grad_scale;
  const float* norm;  // or null
  float max_norm;
  float eps;
  float scale_in;  // X's scale of the first step, a power of two
  float unscale;   // 1 / that of the last X
  uint32_t seed;
  int fill_blocks;
  uint8_t* ws;
  float* sums;     // [parts][kMuonSums] of the group
  unsigned* ctrl;  // MuonPipe's, cleared on the way
  int ctrl_words;
};
// Thread blocks of the kernel that fills X, for one matrix, if each fills up to `blocks` blocks of 64 x 64.
uint32_t muon_fill_ctas(const MuonMat& t, int blocks);
cudaError_t launch_muon_sums(const MuonTable& t, const MuonHyper& h, int dtype, uint32_t ctas, cudaStream_t stream);
cudaError_t launch_muon_fill(const MuonTable& t, const MuonHyper& h, int dtype, uint32_t ctas, cudaStream_t stream);
// All products of all steps; the last one writes the results or steps the parameters (`out`). load: boxes of 64 columns and 64
// rows of the workspace.
cudaError_t muon_pipe_prepare(int* max_clusters);
cudaError_t launch_muon_pipe(const CUtensorMap& load, const MuonTable& t, const MuonPipe& p, const MuonHyper& h,
                             int out, bool split, int clusters, cudaStream_t stream);

}  // namespace hylo
