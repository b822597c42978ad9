// Host-side helpers shared by the files that implement the C ABI: error text, the per-device
// state, tensor maps. Defined in hylo_kl_api.cu.
#pragma once

#include <string>

#include "../../include/hylo_kl.h"
#include "hylo_internal.h"
#include "hylo_ops_internal.h"

namespace hylo {

struct DeviceState {
  bool init = false;
  bool sm103 = false;
  int sms = 0;
  int fused_clusters = 0;  // 2-CTA clusters of the fused kernels resident at once
  int logits_clusters = 0; // clusters of the logits kernel resident at once
  int pipe_clusters = 0;   // 2-CTA clusters of the pipelined backward resident at once
  int head_clusters = 0;   // 2-CTA clusters of the head log-probability kernel resident at once
  int muon_clusters = 0;   // 2-CTA clusters of the orthogonalised updates' products resident at once, set by the first of them
  TokenOccupancy token;    // of the token log-probability kernels
  unsigned pace_epoch = 0;  // epoch of the last paced fused launch on this device
  int* status = nullptr;
  std::string why;
};

void clear_error();
hylo_status fail(hylo_status s, const char* fmt, ...);
hylo_status cuda_fail(cudaError_t e, const char* what);

// Time limit of one device-side wait.
unsigned long long wait_limit_ns();

// The current device's state, set up on first use; HYLO_ERR_ARCH if it is not sm_103.
hylo_status current_device(DeviceState** out);

// 2-D tensor map, 128-byte swizzle, zero fill outside the tensor.
hylo_status make_map(CUtensorMap* m, const void* base, CUtensorMapDataType dt, uint64_t inner, uint64_t outer,
                     uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer);
// 3-D tensor map [outer2][outer1][inner] (contiguous), zero fill outside.
hylo_status make_map_3d(CUtensorMap* m, const void* base, CUtensorMapDataType dt, uint64_t inner, uint64_t outer1,
                        uint64_t outer2, uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer1,
                        CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B);

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// An array of an optimizer step, [begin, end).
struct Span {
  uintptr_t begin, end;
  bool written;
  int tensor;
};
// Thread blocks update their elements in any order, so no array that the step writes may overlap another one. Sorts the spans.
hylo_status check_spans(Span* spans, size_t n);

inline size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Vocabulary segments per 256-token tile (at most `most`) for `workers` persistent clusters.
int choose_segments(int64_t token_tiles, int64_t vtiles, int workers, int most);

// Bytes of the pipelined backward's G ring for one bf16 term; its counters follow the ring(s).
size_t bwd_bytes(int64_t N, int64_t V, int64_t token_chunk);
// Rows of its token blocks.
int64_t pipe_rows(int64_t N, int64_t token_chunk);
// Words of its vocabulary blocks (pipe_setup takes another number of them in `width`, a multiple of 256, or 0).
int64_t pipe_width(int64_t R, int64_t V);
constexpr size_t kPipeCtrlBytes = 256;
hylo_status pipe_setup(const uint16_t* h, const uint16_t* W, int64_t N, int64_t d, int64_t V, float tau,
                       int64_t token_chunk, int64_t width, float* dh, float* dW, void* workspace, size_t g_total, bool split,
                       DeviceState** dev, CUtensorMap* maps, BwdPipeParams* p, int* clusters);

}  // namespace hylo
