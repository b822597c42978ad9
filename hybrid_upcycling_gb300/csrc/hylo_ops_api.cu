// Host side of the C ABI declared in include/hylo_ops.h: argument checks and launches.
#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>
#include <memory>
#include <new>

#include "hylo_host.h"

using namespace hylo;

namespace {

bool dtype_ok(int d) { return d == HYLO_F32 || d == HYLO_BF16 || d == HYLO_F16; }
constexpr float kLog2eHost = 1.4426950408889634f;
uintptr_t dtype_bytes(int d) { return d == HYLO_F32 ? 4 : 2; }

// The kernels work with 1 / tau and, the larger of the two, log2(e) / tau.
bool tau_ok(float tau) { return std::isfinite(tau) && tau > 0.f && std::isfinite(kLog2eHost / tau); }

hylo_status check_rows(const void* z, int dtype, int64_t N, int64_t V, int64_t ld, float tau, const int64_t* tokens) {
  if (!z || !tokens) return fail(HYLO_ERR_NULL, "a required pointer is NULL");
  if (!dtype_ok(dtype)) return fail(HYLO_ERR_DIM, "unknown dtype %d", dtype);
  if (N < 1 || V < 1 || N > 0x7fffffffLL || V > 0x7fffffffLL || ld < V || ld > (int64_t(1) << 40))
    return fail(HYLO_ERR_DIM, "invalid sizes N=%lld V=%lld ld=%lld (need 1 <= N, V < 2^31, ld >= V)",
                static_cast<long long>(N), static_cast<long long>(V), static_cast<long long>(ld));
  if (!aligned(z, dtype_bytes(dtype))) return fail(HYLO_ERR_ALIGN, "logits must be element-aligned");
  if (!aligned(tokens, 8)) return fail(HYLO_ERR_ALIGN, "tokens must be 8-byte aligned");
  if (!tau_ok(tau)) return fail(HYLO_ERR_TAU, "tau must be finite and > 0, and so must log2(e) / tau");
  return HYLO_OK;
}

TokenRows rows_of(const void* z, int64_t N, int64_t V, int64_t ld, float tau, const int64_t* tokens) {
  return TokenRows{z, ld, static_cast<int>(N), static_cast<int>(V), 1.0f / tau, kLog2eHost / tau, tokens};
}

bool head_sizes_ok(int64_t N, int64_t d, int64_t V) {
  return N >= 1 && V >= 1 && N <= 0x7fffffffLL && V <= 0x7fffffffLL && d >= 8 && d <= 65536 && d % 8 == 0;
}

// The forward's vocabulary segments per 256-token tile at most: enough for every cluster of a large device
// to have a unit when there are few tiles.
int head_segments(int64_t N) {
  const int64_t s = cdiv(kMaxClusters, cdiv(N, 2 * kBM));
  return s > kMaxSegments ? static_cast<int>(s) : kMaxSegments;
}

// Copies of h in the workspace. All clusters read h all the time, and less than 128 KiB lies in a few of L2's slices,
// which then hold everything up: 8 tokens of d = 4096, V = 128256 took 190 to 280 us by where h lay, and 172 us (179
// with logits in parts, kLogitDepth) with copies of 512 KiB in all. A small LM head is read in a few microseconds, in
// which the copies cost more.
constexpr int64_t kHotBytes = 128 << 10, kCopyBytes = 512 << 10, kCopyHeadBytes = 64 << 20;
constexpr int64_t kMaxCopies = 64;  // about one for each cluster
int head_copies(int64_t N, int64_t d, int64_t V) {
  const int64_t bytes = N * d * 2;
  if (bytes >= kHotBytes || V * d * 2 < kCopyHeadBytes) return 1;
  const int64_t copies = cdiv(kCopyBytes, bytes);
  return static_cast<int>(copies < kMaxCopies ? copies : kMaxCopies);
}

// The forward's workspace: the tokens' logits, two partial sums per token and segment, and copies of h.
struct HeadFwd {
  size_t part, copies, total;
};
HeadFwd head_fwd_layout(int64_t N, int64_t d, int64_t V) {
  HeadFwd l{};
  l.part = round256(N * sizeof(float));
  l.copies = l.total = l.part + static_cast<size_t>(N) * 2 * head_segments(N) * sizeof(float4);
  const int copies = head_copies(N, d, V);
  if (copies > 1) {
    l.copies = round256(l.copies);
    l.total = l.copies + static_cast<size_t>(copies) * N * d * 2;
  }
  return l;
}

// The backward's workspace: the G ring(s), the counters, and the fp32 sums (of the gradients that are wanted) that are joined or
// rounded at the end.
struct HeadBwd {
  size_t ctrl, dh, dW, total;
  int64_t width;     // words of a vocabulary block, or 0 (pipe_width)
  int64_t parts;     // dh is stored in this many parts, or 0
  int64_t dh_words;  // words of a part
  bool dW_direct;    // dW is written in bf16 by the pipelined backward itself
};
// Few tokens: dh in parts, one per vocabulary block (at most 16 of those) or several. Long blocks wait less for ring
// slots, short ones spread dh over more clusters, which counts with more tokens. Measured at d = 2048, V = 128256 with
// blocks of 8192, 12288, 16384 and 24576 words: 256 tokens 642, 550, 587, 534 us; 512 tokens 777, 714, 649, 643; 1024
// tokens 1062, 1054, 1075 us (24576 words do not fit the ring; all before the logits came in parts, which adds 1 to 4%
// in every case). Fewer words where that leaves fewer than three blocks. N d is bounded so that a part is at most 8 MiB;
// with more tokens the chain of additions is short beside the rest.
constexpr int64_t kPartTokens = 1024, kPartElems = int64_t(1) << 21, kMaxParts = 16;
constexpr int64_t part_words(int64_t N) { return N <= 512 ? 24576 : 12288; }
// With few 256 x 256 tiles of dh (N d small) a block's words are cut up too, into parts of their own, so that the long
// products run on more clusters. Measured (1, 2, 3, 4 parts a block; V = 128256 if not said): 256 tokens, d = 2048 538,
// 462, 475, 486 us, d = 4096 854, 878, 897, 908; 512 tokens, d = 2048 644, 625, 636, 653; 1000 tokens, d = 2048 1077,
// 1129, 1184, 1197 (again before the parts of logits); 800 tokens, d = 1024, V = 32000 242, 183, 183, 174; 1000 tokens,
// d = 512, V = 151936 795, 527, 463, 435. So up to 16 items a block with one tile of tokens and up to 32 with more, of
// at least 1024 words.
constexpr int64_t kPartBytes = int64_t(128) << 20;  // of all parts together
constexpr int64_t kMinPartWords = 1024;
int64_t block_parts(int64_t N, int64_t d, int64_t blocks) {
  const int64_t tiles = cdiv(N, 256) * cdiv(d, 256), fit = kPartBytes / (blocks * N * d * 4);
  const int64_t want = cdiv(N <= 256 ? 16 : 32, tiles);
  return want < fit ? want : fit < 1 ? 1 : fit;
}

HeadBwd head_bwd_layout(int64_t N, int64_t d, int64_t V, int64_t token_chunk, bool split, int grad_dtype, bool want_dh,
                        bool want_dW) {
  HeadBwd l{};
  const int64_t R = pipe_rows(N, token_chunk);
  size_t ring = bwd_bytes(N, V, token_chunk);
  if (N <= R && N <= kPartTokens && N * d <= kPartElems) {
    int64_t w = cdiv(V, kGRing) < part_words(N) ? cdiv(V, kGRing) : part_words(N);
    if (w < cdiv(V, kMaxParts)) w = cdiv(V, kMaxParts);
    w = cdiv(w, 256) * 256;
    if (kGRing * R * w * 2 <= kGBlockBytes) {
      l.width = w;
      l.dh_words = cdiv(cdiv(w, block_parts(N, d, cdiv(V, w))), 64) * 64;
      if (l.dh_words < kMinPartWords) l.dh_words = kMinPartWords;
      l.parts = (cdiv(V, w) - 1) * cdiv(w, l.dh_words) + cdiv(V - (cdiv(V, w) - 1) * w, l.dh_words);
      ring = static_cast<size_t>(kGRing) * R * w * 2;
    }
  }
  l.ctrl = round256(ring) * (split ? 2 : 1);
  l.dh = l.dW = l.total = l.ctrl + kPipeCtrlBytes;
  if (want_dh && (grad_dtype == HYLO_BF16 || l.parts > 0))
    l.dW = l.total = l.dh + round256(static_cast<size_t>(l.parts > 0 ? l.parts : 1) * N * d * sizeof(float));
  if (grad_dtype == HYLO_BF16) {
    l.dW_direct = N <= R;
    if (want_dW && !l.dW_direct) l.total = l.dW + round256(static_cast<size_t>(V) * d * sizeof(float));
  }
  return l;
}

hylo_status check_head(const uint16_t* h, const uint16_t* W, int64_t N, int64_t d, int64_t V, float tau,
                       const int64_t* tokens, void* workspace, size_t workspace_bytes, size_t need) {
  if (!h || !W || !tokens || !workspace) return fail(HYLO_ERR_NULL, "a required pointer is NULL");
  if (!head_sizes_ok(N, d, V))
    return fail(HYLO_ERR_DIM, "invalid sizes N=%lld d=%lld V=%lld (d must be a multiple of 8, 8..65536)",
                static_cast<long long>(N), static_cast<long long>(d), static_cast<long long>(V));
  if (!aligned(h, 16) || !aligned(W, 16)) return fail(HYLO_ERR_ALIGN, "h and W must be 16-byte aligned");
  if (!aligned(tokens, 8)) return fail(HYLO_ERR_ALIGN, "tokens must be 8-byte aligned");
  if (!aligned(workspace, 256)) return fail(HYLO_ERR_ALIGN, "workspace must be 256-byte aligned");
  if (!tau_ok(tau)) return fail(HYLO_ERR_TAU, "tau must be finite and > 0, and so must log2(e) / tau");
  if (workspace_bytes < need)
    return fail(HYLO_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu required", workspace_bytes, need);
  return HYLO_OK;
}

// An array of an optimizer step, [begin, end).
struct Span {
  uintptr_t begin, end;
  bool written;
  int tensor;
};

// Thread blocks update their elements in any order, so no array that the step writes may overlap another one.
hylo_status check_apart(const hylo_adamw_tensor* tensors, int count, size_t param_bytes, size_t grad_bytes, size_t state_bytes) {
  const std::unique_ptr<Span[]> spans(new (std::nothrow) Span[7 * static_cast<size_t>(count)]);
  if (!spans) return fail(HYLO_ERR_CUDA, "no host memory for %d tensors", count);
  size_t n = 0;
  for (int i = 0; i < count; ++i) {
    const hylo_adamw_tensor& t = tensors[i];
    if (t.n == 0) continue;
    auto add = [&](const void* p, size_t bytes, bool written) {
      const uintptr_t a = reinterpret_cast<uintptr_t>(p);
      if (p) spans[n++] = Span{a, a + bytes, written, i};
    };
    const size_t k = static_cast<size_t>(t.n);
    add(t.param, k * param_bytes, true);
    add(t.grad, k * grad_bytes, false);
    add(t.master, k * 4, true);
    add(t.m, k * state_bytes, true);
    add(t.v, k * state_bytes, true);
    if (state_bytes == 1) {
      add(t.m_exp, (k + 255) / 256, true);
      add(t.v_exp, (k + 255) / 256, true);
    }
  }
  std::sort(spans.get(), spans.get() + n, [](const Span& a, const Span& b) { return a.begin < b.begin; });
  Span any{}, written{};  // of those so far, the ones that reach furthest
  for (size_t i = 0; i < n; ++i) {
    const Span& s = spans[i];
    const Span& before = s.written ? any : written;
    if (s.begin < before.end)
      return fail(HYLO_ERR_DIM, "arrays of tensors %d and %d overlap, and the step writes to them", before.tensor, s.tensor);
    if (s.end > any.end) any = s;
    if (s.written && s.end > written.end) written = s;
  }
  return HYLO_OK;
}

}  // namespace

extern "C" {

hylo_status hylo_token_logprobs(const void* z, int dtype, int64_t N, int64_t V, int64_t ld, float tau,
                                const int64_t* tokens, int k, float* logp, float* entropy, float* lse, float* stats,
                                float* top_logp, int64_t* top_ids, cudaStream_t stream) {
  clear_error();
  hylo_status st = check_rows(z, dtype, N, V, ld, tau, tokens);
  if (st != HYLO_OK) return st;
  if (!logp || (k > 0 && (!top_logp || !top_ids))) return fail(HYLO_ERR_NULL, "an output pointer is NULL");
  if (k < 0 || k > HYLO_TOP_MAX || k > V)
    return fail(HYLO_ERR_DIM, "k=%d alternatives (0 <= k <= min(V, %d))", k, HYLO_TOP_MAX);
  if (!aligned(logp, 4) || !aligned(entropy, 4) || !aligned(lse, 4) || !aligned(stats, 8) || !aligned(top_logp, 4) ||
      !aligned(top_ids, 8))
    return fail(HYLO_ERR_ALIGN, "output pointers must be aligned to their elements (stats: 8 bytes)");
  DeviceState* dev = nullptr;
  if ((st = current_device(&dev)) != HYLO_OK) return st;
  const TokenOut out{k, logp, entropy, lse, reinterpret_cast<float2*>(stats), top_logp, top_ids};
  const cudaError_t e = launch_token_logprobs(rows_of(z, N, V, ld, tau, tokens), out, dtype, dev->token, stream);
  return e == cudaSuccess ? HYLO_OK : cuda_fail(e, "launch token log-probabilities");
}

hylo_status hylo_token_logprobs_backward(const void* z, int dtype, int64_t N, int64_t V, int64_t ld, float tau,
                                         const int64_t* tokens, const float* stats, const float* entropy,
                                         const float* g_logp, const float* g_entropy, void* dz, int64_t ldd,
                                         cudaStream_t stream) {
  clear_error();
  hylo_status st = check_rows(z, dtype, N, V, ld, tau, tokens);
  if (st != HYLO_OK) return st;
  if (!stats || !dz || (g_entropy && !entropy)) return fail(HYLO_ERR_NULL, "a required pointer is NULL");
  if (ldd < V || ldd > (int64_t(1) << 40))
    return fail(HYLO_ERR_DIM, "invalid gradient row stride %lld", static_cast<long long>(ldd));
  if (!aligned(dz, dtype_bytes(dtype)) || !aligned(stats, 8) || !aligned(entropy, 4) || !aligned(g_logp, 4) ||
      !aligned(g_entropy, 4))
    return fail(HYLO_ERR_ALIGN, "pointers must be aligned to their elements (stats: 8 bytes)");
  DeviceState* dev = nullptr;
  if ((st = current_device(&dev)) != HYLO_OK) return st;
  const TokenGrad g{reinterpret_cast<const float2*>(stats), entropy, g_logp, g_entropy, dz, ldd};
  const cudaError_t e = launch_token_logprobs_bwd(rows_of(z, N, V, ld, tau, tokens), g, dtype, dev->sms, stream);
  return e == cudaSuccess ? HYLO_OK : cuda_fail(e, "launch token log-probabilities backward");
}

size_t hylo_head_logprobs_workspace_bytes(int64_t N, int64_t d, int64_t V, int64_t token_chunk, int split_g,
                                          int grad_dtype) {
  clear_error();
  if (!head_sizes_ok(N, d, V) || (grad_dtype != HYLO_F32 && grad_dtype != HYLO_BF16)) return 0;
  const size_t f = head_fwd_layout(N, d, V).total;
  const size_t b = head_bwd_layout(N, d, V, token_chunk, split_g != 0, grad_dtype, true, true).total;
  return f > b ? f : b;
}

size_t hylo_head_logprobs_forward_workspace_bytes(int64_t N, int64_t d, int64_t V) {
  clear_error();
  return head_sizes_ok(N, d, V) ? head_fwd_layout(N, d, V).total : 0;
}

size_t hylo_head_logprobs_backward_workspace_bytes(int64_t N, int64_t d, int64_t V, int64_t token_chunk, int split_g,
                                                   int grad_dtype, int want_dh, int want_dW) {
  clear_error();
  if (!head_sizes_ok(N, d, V) || (grad_dtype != HYLO_F32 && grad_dtype != HYLO_BF16) || (!want_dh && !want_dW)) return 0;
  return head_bwd_layout(N, d, V, token_chunk, split_g != 0, grad_dtype, want_dh != 0, want_dW != 0).total;
}

hylo_status hylo_head_logprobs(const uint16_t* h, const uint16_t* W, int64_t N, int64_t d, int64_t V, float tau,
                               const int64_t* tokens, float* logp, float* entropy, float* lse, void* workspace,
                               size_t workspace_bytes, cudaStream_t stream) {
  clear_error();
  if (!logp) return fail(HYLO_ERR_NULL, "logp is NULL");
  if (!aligned(logp, 4) || !aligned(entropy, 4) || !aligned(lse, 4))
    return fail(HYLO_ERR_ALIGN, "output pointers must be 4-byte aligned");
  const HeadFwd l = head_sizes_ok(N, d, V) ? head_fwd_layout(N, d, V) : HeadFwd{};
  hylo_status st = check_head(h, W, N, d, V, tau, tokens, workspace, workspace_bytes, l.total);
  if (st != HYLO_OK) return st;
  DeviceState* dev = nullptr;
  if ((st = current_device(&dev)) != HYLO_OK) return st;
  HeadParams p{};
  p.N = static_cast<int>(N);
  p.V = static_cast<int>(V);
  p.c = kLog2eHost / tau;
  p.inv_tau = 1.0f / tau;
  p.tokens = tokens;
  p.z_token = static_cast<float*>(workspace);
  p.part = reinterpret_cast<float4*>(static_cast<char*>(workspace) + l.part);
  p.ctl = WaitCtl{dev->status, wait_limit_ns()};
  // With lse a backward may follow. It takes exp(z - lse) of logits that it computes again for probabilities, and 1 - p of a
  // confident token loses as many digits as those differ from the forward's: both then accumulate alike. (With dot products
  // here the gradients of one token with 1 - p = 1e-3 and d = 4096 were 8% off.)
  if (!lse && head_few_fits(N, d)) {
    p.slots = dev->sms < 2 * head_segments(N) ? dev->sms : 2 * head_segments(N);
    const cudaError_t e = launch_head_few(h, W, static_cast<int>(d), p, logp, entropy, lse, stream);
    return e == cudaSuccess ? HYLO_OK : cuda_fail(e, "launch head log-probabilities of few tokens");
  }
  CUtensorMap m_h, m_W;
  const CUtensorMapDataType bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  p.copies = head_copies(N, d, V);
  if (p.copies > 1) {
    void* const copies = static_cast<char*>(workspace) + l.copies;
    const cudaError_t e = launch_head_copy(h, copies, N * d, p.copies, stream);
    if (e != cudaSuccess) return cuda_fail(e, "copy the hidden states");
    h = static_cast<const uint16_t*>(copies);
  }
  if ((st = make_map_3d(&m_h, h, bf, d, N, p.copies, d * 2, kBK, kBM)) != HYLO_OK) return st;
  if ((st = make_map(&m_W, W, bf, d, V, d * 2, kBK, kFusedBN / 2)) != HYLO_OK) return st;
  p.kb = static_cast<int>(cdiv(d, kBK));
  p.depths = static_cast<int>(cdiv(p.kb, kLogitDepth));
  p.token_tiles = static_cast<int>(cdiv(N, 2 * kBM));
  p.vtiles = static_cast<int>(cdiv(V, kFusedBN));
  p.nseg = choose_segments(p.token_tiles, p.vtiles, dev->head_clusters, head_segments(N));
  p.units = p.token_tiles * p.nseg;
  p.slots = 2 * p.nseg;
  const int clusters = p.units < dev->head_clusters ? p.units : dev->head_clusters;
  const cudaError_t e = launch_head_logprobs(m_h, m_W, p, logp, entropy, lse, clusters, stream);
  return e == cudaSuccess ? HYLO_OK : cuda_fail(e, "launch head log-probabilities");
}

hylo_status hylo_head_logprobs_backward(const uint16_t* h, const uint16_t* W, int64_t N, int64_t d, int64_t V,
                                        float tau, int64_t token_chunk, const int64_t* tokens, const float* lse,
                                        const float* entropy, const float* g_logp, const float* g_entropy, int split_g,
                                        int grad_dtype, void* dh, void* dW, void* workspace, size_t workspace_bytes,
                                        cudaStream_t stream) {
  clear_error();
  if (!lse || (!dh && !dW) || (g_entropy && !entropy)) return fail(HYLO_ERR_NULL, "a required pointer is NULL");
  if (grad_dtype != HYLO_F32 && grad_dtype != HYLO_BF16) return fail(HYLO_ERR_DIM, "gradients are fp32 or bf16 (dtype %d)", grad_dtype);
  const bool split = split_g != 0;
  const HeadBwd l = head_sizes_ok(N, d, V) ? head_bwd_layout(N, d, V, token_chunk, split, grad_dtype, dh != nullptr, dW != nullptr)
                                            : HeadBwd{};
  hylo_status st = check_head(h, W, N, d, V, tau, tokens, workspace, workspace_bytes, l.total);
  if (st != HYLO_OK) return st;
  if (!aligned(dh, 16) || !aligned(dW, 16)) return fail(HYLO_ERR_ALIGN, "gradient pointers must be 16-byte aligned");
  if (!aligned(lse, 4) || !aligned(entropy, 4) || !aligned(g_logp, 4) || !aligned(g_entropy, 4))
    return fail(HYLO_ERR_ALIGN, "per-token pointers must be 4-byte aligned");
  // The sums are fp32: for bf16 gradients they are formed in the workspace and rounded once, or, where dW has one token
  // block, as they leave the tensor cores.
  char* ws = static_cast<char*>(workspace);
  const bool bf16 = grad_dtype == HYLO_BF16;
  float* dh32 = bf16 || l.parts > 0 ? reinterpret_cast<float*>(ws + l.dh) : static_cast<float*>(dh);
  float* dW32 = l.dW_direct ? static_cast<float*>(dW) : bf16 ? reinterpret_cast<float*>(ws + l.dW) : static_cast<float*>(dW);
  // A tensor map has to have some address; of a gradient that is not wanted nothing is stored.
  if (!dh) dh32 = reinterpret_cast<float*>(ws);
  if (!dW) dW32 = reinterpret_cast<float*>(ws);
  DeviceState* dev = nullptr;
  CUtensorMap maps[kPipeMaps];
  BwdPipeParams p{};
  int clusters = 0;
  if ((st = pipe_setup(h, W, N, d, V, tau, token_chunk, l.width, dh32, dW32, workspace, l.ctrl, split, &dev, maps, &p, &clusters)) !=
      HYLO_OK)
    return st;
  maps[1] = maps[0];  // no teacher: never loaded from
  maps[3] = maps[2];
  if (dW && l.dW_direct && (st = make_map_3d(&maps[7], dW, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, d, V, 1, d * 2, 32, 32,
                                       CU_TENSOR_MAP_SWIZZLE_64B)) != HYLO_OK)
    return st;
  if (dh && l.parts > 0 && (st = make_map_3d(&maps[6], dh32, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, d, N, l.parts, d * 4, 32, 32)) != HYLO_OK)
    return st;
  cudaError_t e = cudaMemsetAsync(p.ctrl, 0, (kPipeCtrlWords + kGRing) * sizeof(unsigned), stream);
  if (e != cudaSuccess) return cuda_fail(e, "clear the backward's work counters");
  const int order = l.parts > 0 ? kOrderParts : p.TB == 1 || (dh && p.VB >= kGRing) ? kOrderDh : kOrderChain;
  const HeadGrad g{tokens, lse, entropy, g_logp, g_entropy, 1.0f / tau, l.dW_direct ? 1 : 0, order, dh ? 1 : 0, dW ? 1 : 0,
                   l.parts > 0 ? static_cast<int>(l.dh_words) : INT_MAX};
  e = launch_bwd_pipe_head(maps, p, g, clusters, stream);
  if (e == cudaSuccess && dh && (bf16 || l.parts > 0))
    e = launch_join_parts(dh32, l.parts > 0 ? static_cast<int>(l.parts) : 1, dh, bf16, N * d, dev->sms, stream);
  if (e == cudaSuccess && dW && bf16 && !l.dW_direct) e = launch_join_parts(dW32, 1, dW, true, V * d, dev->sms, stream);
  return e == cudaSuccess ? HYLO_OK : cuda_fail(e, "launch head log-probabilities backward");
}

size_t hylo_grad_norm_workspace_bytes(void) {
  clear_error();
  return kNormPartials * sizeof(float);
}

hylo_status hylo_grad_norm(const void* const* grads, const int64_t* sizes, int count, int dtype, float* norm,
                           void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  clear_error();
  if (!norm || !workspace || (count > 0 && (!grads || !sizes))) return fail(HYLO_ERR_NULL, "a required pointer is NULL");
  if (count < 0) return fail(HYLO_ERR_DIM, "count=%d", count);
  if (dtype != HYLO_F32 && dtype != HYLO_BF16) return fail(HYLO_ERR_DIM, "gradients are fp32 or bf16 (dtype %d)", dtype);
  for (int i = 0; i < count; ++i) {
    if (sizes[i] < 0 || sizes[i] > (int64_t(1) << 40))
      return fail(HYLO_ERR_DIM, "gradient %d has %lld elements", i, static_cast<long long>(sizes[i]));
    if (sizes[i] > 0 && !grads[i]) return fail(HYLO_ERR_NULL, "gradient %d is NULL", i);
    if (!aligned(grads[i], dtype_bytes(dtype))) return fail(HYLO_ERR_ALIGN, "gradient %d is not element-aligned", i);
  }
  if (!aligned(norm, 4) || !aligned(workspace, 16)) return fail(HYLO_ERR_ALIGN, "workspace must be 16-byte aligned");
  if (workspace_bytes < kNormPartials * sizeof(float))
    return fail(HYLO_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu required", workspace_bytes,
                kNormPartials * sizeof(float));
  DeviceState* dev = nullptr;
  const hylo_status st = current_device(&dev);
  if (st != HYLO_OK) return st;
  const cudaError_t e =
      launch_grad_norm(grads, sizes, count, dtype, norm, static_cast<float*>(workspace), dev->sms, stream);
  return e == cudaSuccess ? HYLO_OK : cuda_fail(e, "launch gradient norm");
}

hylo_status hylo_adamw_step(const hylo_adamw_tensor* tensors, int count, int param_dtype, int grad_dtype,
                            int state_bits, double beta1, double beta2, double eps, int64_t step, float grad_scale,
                            const float* norm, float max_norm, uint32_t seed, cudaStream_t stream) {
  clear_error();
  if (count < 0) return fail(HYLO_ERR_DIM, "count=%d", count);
  if (count > 0 && !tensors) return fail(HYLO_ERR_NULL, "tensors is NULL");
  if ((param_dtype != HYLO_F32 && param_dtype != HYLO_BF16) || (grad_dtype != HYLO_F32 && grad_dtype != HYLO_BF16) ||
      (state_bits != 32 && state_bits != 8))
    return fail(HYLO_ERR_DIM, "param_dtype=%d grad_dtype=%d state_bits=%d (fp32 or bf16; 32 or 8)", param_dtype,
                grad_dtype, state_bits);
  if (!(beta1 >= 0 && beta1 < 1) || !(beta2 >= 0 && beta2 < 1) || !(eps >= 0) || !std::isfinite(eps) || step < 1)
    return fail(HYLO_ERR_DIM, "beta1=%g beta2=%g eps=%g step=%lld (0 <= beta < 1, eps >= 0, step >= 1)", beta1, beta2,
                eps, static_cast<long long>(step));
  // The kernel's reciprocal takes a smaller eps for 0: an element without moments would become 0 / 0.
  if (state_bits == 8 && !(eps >= FLT_MIN)) return fail(HYLO_ERR_DIM, "8-bit states need eps >= 2^-126");
  if (!std::isfinite(grad_scale) || (norm && !(max_norm > 0)))
    return fail(HYLO_ERR_TAU, "grad_scale must be finite and max_norm > 0");
  int some = -1;  // the first tensor that has elements
  for (int i = 0; i < count; ++i) {
    const hylo_adamw_tensor& t = tensors[i];
    if (t.n < 0 || t.n > (int64_t(1) << 40))
      return fail(HYLO_ERR_DIM, "tensor %d has %lld elements", i, static_cast<long long>(t.n));
    if (!std::isfinite(t.lr) || !std::isfinite(t.weight_decay))
      return fail(HYLO_ERR_TAU, "lr and weight_decay of tensor %d must be finite", i);
    if (t.n == 0) continue;
    if (some < 0) some = i;
    if ((t.master != nullptr) != (tensors[some].master != nullptr) || (t.master && param_dtype == HYLO_F32))
      return fail(HYLO_ERR_DIM, "tensor %d: masters go with bf16 parameters, for all tensors or none", i);
    if (!t.param || !t.grad || !t.m || !t.v || (state_bits == 8 && (!t.m_exp || !t.v_exp)))
      return fail(HYLO_ERR_NULL, "a required pointer of tensor %d is NULL", i);
    const uintptr_t s = state_bits == 8 ? 1 : 4;
    if (!aligned(t.param, dtype_bytes(param_dtype)) || !aligned(t.grad, dtype_bytes(grad_dtype)) ||
        !aligned(t.master, 4) || !aligned(t.m, s) || !aligned(t.v, s))
      return fail(HYLO_ERR_ALIGN, "tensor %d is not element-aligned", i);
  }
  hylo_status st = check_apart(tensors, count, dtype_bytes(param_dtype), dtype_bytes(grad_dtype), state_bits == 8 ? 1 : 4);
  if (st != HYLO_OK) return st;
  DeviceState* dev = nullptr;
  if ((st = current_device(&dev)) != HYLO_OK) return st;
  if (some < 0) return HYLO_OK;
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  const cudaError_t asked = cudaStreamIsCapturing(stream, &capture);
  if (asked != cudaSuccess) return cuda_fail(asked, "ask whether the stream is being captured");
  if (capture != cudaStreamCaptureStatusNone)
    return fail(HYLO_ERR_CAPTURE, "an AdamW step may not be captured: its step number, learning rates and seed are host values that "
                                  "every replay would repeat");
  AdamWHyper h;
  h.beta1 = static_cast<float>(beta1);
  h.beta2 = static_cast<float>(beta2);
  h.one_minus_beta1 = static_cast<float>(1.0 - beta1);
  h.one_minus_beta2 = static_cast<float>(1.0 - beta2);
  h.eps = static_cast<float>(eps);
  h.rbc2 = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(beta2, static_cast<double>(step))));
  h.grad_scale = grad_scale;
  h.norm = norm;
  h.max_norm = max_norm;
  h.seed = seed;
  const double bias1 = 1.0 - std::pow(beta1, static_cast<double>(step));
  const cudaError_t e = launch_adamw(tensors, count, param_dtype, grad_dtype, state_bits, tensors[some].master != nullptr, bias1, h, dev->sms, stream);
  return e == cudaSuccess ? HYLO_OK : cuda_fail(e, "launch AdamW");
}

}  // extern "C"
