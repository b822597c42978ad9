// Host side of the orthogonalised updates declared in include/hylo_ops.h: argument checks, the groups of matrices that share
// the workspace, the scales of every step, and the launches.
#include <cmath>
#include <memory>
#include <mutex>
#include <new>

#include "hylo_host.h"
#include "muon.h"

using namespace hylo;

namespace {

constexpr int64_t kMaxSide = int64_t(1) << 20, kMaxShort = 16384;
constexpr int kMaxSteps = kMuonStepsMax;
// Matrices that go through the products together: enough tiles for every SM (groups of half as much take 3 % longer), and no
// more memory than that takes.
constexpr int64_t kGroupRows = (int64_t(1024) << 20) / 128;

uintptr_t bytes_of(int dtype) { return dtype == HYLO_F32 ? 4 : 2; }

bool sides_ok(int64_t rows, int64_t cols) {
  return rows >= 0 && cols >= 0 && rows <= kMaxSide && cols <= kMaxSide && (rows < cols ? rows : cols) <= kMaxShort;
}

// One matrix of the list, from either entry point.
struct Item {
  const void* src;
  void* dst;
  float* master;
  float* mom;
  int64_t rows, cols, ld;
  double decay, step;
};
Item item_of(const hylo_orth_matrix& x) {
  return Item{x.x, x.out, nullptr, nullptr, x.rows, x.cols, x.rows == 1 ? x.cols : x.ld, 1.0, 0.0};
}
Item item_of(const hylo_muon_tensor& x) {
  return Item{x.grad, x.param, x.master, x.momentum, x.rows, x.cols, x.cols, 1.0 - x.lr * x.weight_decay, x.lr * x.scale};
}

struct Shape {
  int64_t m, n, mp, np, x_rows, a_rows, parts;
};
Shape shape_of(int64_t rows, int64_t cols) {
  Shape s;
  s.m = rows < cols ? rows : cols;
  s.n = rows < cols ? cols : rows;
  s.mp = cdiv(s.m, 256) * 256;
  s.np = cdiv(s.n, 256) * 256;
  s.x_rows = s.np / 64 * s.mp;
  s.a_rows = s.mp / 64 * s.mp;
  const int64_t parts = cdiv(rows * cols, 8) / 1024;
  s.parts = parts < 1 ? 1 : parts > kMuonParts ? kMuonParts : parts;
  return s;
}
// 128-byte rows: X twice, its second term, A and B.
int64_t rows_of(const Shape& s) { return 3 * s.x_rows + 2 * s.a_rows; }

// The sum of an item of Gram (K = n) is split where the group has so few that clusters would be idle beside a long one. A 64-deep
// k-block takes 550 cycles and a part 3500 to be written, read and added, so sqrt(n / 64 / 6.4) parts. bf16, without and with:
// 256 x 16384 512 and 292 us, 2048 x 8192 619 and 588, 1 x 100000 2.38 ms and 0.48; sums half as long are even (1024 x 4096 292
// and 299). The clusters are those of a whole GPU: the workspace's size may not depend on the device.
constexpr int64_t kSplitClusters = 76, kSplitFrom = 128, kMaxSplits = 64;
int64_t splits_of(const Shape& s, int64_t group_tiles) {
  const int64_t kn = cdiv(s.n, 64), room = kSplitClusters / group_tiles;
  if (kn < kSplitFrom || room < 2) return 1;
  const int64_t n = static_cast<int64_t>(std::sqrt(static_cast<double>(kn) / 6.4));
  return n < room ? n : room < kMaxSplits ? room : kMaxSplits;
}
int64_t sym_tiles(const Shape& s) { return (s.mp / 256) * (s.mp / 256 + 1) / 2; }

// Items [first, last) that go through the products together; empty ones among them take no place.
struct Group {
  int first, last, mats;
  int64_t rows, parts;
  bool deep;      // some sum is longer than the tensor cores take at a time
  int64_t tiles;  // of Gram
  int64_t split_tiles, split_items;
  size_t sums_at() const { return static_cast<size_t>(rows) * 128; }
  size_t ctrl_at() const { return sums_at() + round256(static_cast<size_t>(parts) * kMuonSums * sizeof(float)); }
  int ctrl_words() const { return kMuonCtrlWords + static_cast<int>(split_tiles) * 16; }
  size_t scratch_at() const { return ctrl_at() + round256(ctrl_words() * sizeof(unsigned)); }
  size_t splits_at() const { return scratch_at() + (deep ? 2 * kMaxClusters * kMuonScratch : 0); }
  size_t bytes() const { return splits_at() + static_cast<size_t>(split_items) * 2 * kMuonScratch; }
};
template <typename T>
Group next_group(const T* list, int count, int first) {
  Group g{};
  g.first = g.last = first;
  for (; g.last < count; ++g.last) {
    const Item x = item_of(list[g.last]);
    if (x.rows == 0 || x.cols == 0) continue;
    const Shape s = shape_of(x.rows, x.cols);
    if (g.mats > 0 && (g.mats == kMuonMats || g.rows + rows_of(s) > kGroupRows)) break;
    ++g.mats;
    g.rows += rows_of(s);
    g.parts += s.parts;
    g.tiles += sym_tiles(s);
  }
  for (int i = first; i < g.last; ++i) {
    const Item x = item_of(list[i]);
    if (x.rows == 0 || x.cols == 0) continue;
    const Shape s = shape_of(x.rows, x.cols);
    const int64_t splits = splits_of(s, g.tiles);
    if (splits > 1) g.split_tiles += sym_tiles(s), g.split_items += sym_tiles(s) * splits;
    g.deep |= cdiv(cdiv(s.n, 64), splits) > kMuonDepth || s.m > kMuonDepth * 64;
  }
  return g;
}

// Whether the upper triangles' products are done sooner by halves of tiles, 296 cycles for a 64-deep block, than by whole ones, 512
// (the tensor cores' rate; 517 over the 128 blocks of a 2048 x 8192 matrix's items): by the longest item and by all of them shared
// out. (5003 x 520, 1000 x 1001 and 8192 x 2048 together 612 us with whole tiles, 560 so. Apply, whose epilogue is as long as its
// products, gains only where every cluster has one half: one 2048 x 2048 221 us, 227 with its 64 tiles halved.)
bool halves_are_sooner(const MuonTable& tab, int64_t clusters, int MuonMat::*depth) {
  int64_t longest = 0, work = 0;
  for (int i = 0; i < tab.count; ++i) {
    const MuonMat& t = tab.t[i];
    longest = t.*depth > longest ? t.*depth : longest;
    work += static_cast<int64_t>(t.mt) * (t.mt + 1) / 2 * (t.*depth);
  }
  longest *= clusters;
  return 296 * (longest > 2 * work ? longest : 2 * work) < 512 * (longest > work ? longest : work);
}

template <typename T>
size_t workspace(const T* list, int count) {
  size_t most = 256;
  for (int i = 0; i < count;) {
    const Group g = next_group(list, count, i);
    if (g.bytes() > most) most = g.bytes();
    i = g.last;
  }
  return most;
}

// The largest a x + b x^3 + c x^5 and b y + c y^2 (y = x^2) in magnitude for singular values 0 <= x <= u.
void bounds(const double* k, double u, double* x_out, double* b_out) {
  const double a = k[0], b = k[1], c = k[2], y = u * u;
  auto f = [&](double t) { return std::fabs(std::sqrt(t) * (a + t * (b + t * c))); };  // t = x^2
  auto g = [&](double t) { return std::fabs(t * (b + t * c)); };
  double most = f(y), poly = g(y);
  auto try_at = [&](double t) {
    if (t > 0 && t < y) {
      most = std::fmax(most, f(t));
      poly = std::fmax(poly, g(t));
    }
  };
  if (c != 0) {  // a + 3 b t + 5 c t^2 = 0
    const double d = 9 * b * b - 20 * a * c;
    if (d >= 0) {
      try_at((-3 * b + std::sqrt(d)) / (10 * c));
      try_at((-3 * b - std::sqrt(d)) / (10 * c));
    }
    try_at(-b / (2 * c));
  } else if (b != 0) {
    try_at(-a / (3 * b));
  }
  *x_out = most;
  *b_out = poly;
}

// A power of two that brings magnitudes up to `most` below 2^15: fp16 holds twice that.
double scale_for(double most) { return std::exp2(14 - std::ilogb(std::fmax(most, 0x1p-40))); }

struct Steps {
  int count;
  double x[kMaxSteps + 1], a[kMaxSteps], b[kMaxSteps];  // scales of X before each step (and behind the last), A, B
  const double* k;
};

hylo_status plan_steps(int steps, const double* coefficients, double eps, Steps* out) {
  if (steps < 1 || steps > kMaxSteps) return fail(HYLO_ERR_DIM, "steps=%d (1 to %d)", steps, kMaxSteps);
  if (!coefficients) return fail(HYLO_ERR_NULL, "coefficients is NULL");
  if (!(eps >= 0) || !std::isfinite(static_cast<float>(eps))) return fail(HYLO_ERR_TAU, "eps must be finite and >= 0");
  out->count = steps;
  out->k = coefficients;
  double u = 1.0;  // singular values of the scaled matrix are at most its norm
  for (int i = 0; i < steps; ++i) {
    const double* k = coefficients + 3 * i;
    if (!std::isfinite(k[0]) || !std::isfinite(k[1]) || !std::isfinite(k[2])) return fail(HYLO_ERR_TAU, "the coefficients must be finite");
    double next, poly;
    bounds(k, u, &next, &poly);
    out->x[i] = scale_for(u);
    out->a[i] = scale_for(u * u);
    out->b[i] = scale_for(poly);
    u = next * 1.01;  // rounding
    if (!(u <= 0x1p20) || !(poly <= 0x1p20))
      return fail(HYLO_ERR_TAU, "with these coefficients singular values can grow beyond 2^20 (step %d)", i + 1);
  }
  out->x[steps] = scale_for(u);
  return HYLO_OK;
}

bool aligned_rows(const void* p, int64_t ld, uintptr_t bytes) { return aligned(p, 16) && ld * bytes % 16 == 0; }

// The current device with the products' kernels set up: by the first call that needs them, so that a device on which their clusters do
// not fit runs everything else.
hylo_status muon_device(DeviceState** out) {
  static std::mutex mu;
  const hylo_status st = current_device(out);
  if (st != HYLO_OK) return st;
  std::lock_guard<std::mutex> lock(mu);
  int& clusters = (*out)->muon_clusters;
  if (clusters > 0) return HYLO_OK;
  int n = 0;
  const cudaError_t e = muon_pipe_prepare(&n);
  if (e != cudaSuccess) return cuda_fail(e, "set-up of the orthogonalised updates' kernels");
  if (n < 1) return fail(HYLO_ERR_CUDA, "no thread-block cluster of the orthogonalised updates' kernels fits on the device");
  clusters = n;
  return HYLO_OK;
}

// All launches of one list. dtype: of the matrices or gradients; out_dtype: of the results or parameters.
template <typename T>
hylo_status run(const T* list, int count, int dtype, int out_dtype, bool masters, const Steps& s, MuonHyper h, void* ws,
                cudaStream_t stream) {
  DeviceState* dev = nullptr;
  hylo_status st = muon_device(&dev);
  if (st != HYLO_OK) return st;
  uint64_t pos = 0;
  h.scale_in = static_cast<float>(s.x[0]);
  h.unscale = static_cast<float>(1.0 / s.x[s.count]);
  h.ws = static_cast<uint8_t*>(ws);
  for (int i = 0; i < count;) {
    const Group group = next_group(list, count, i);
    MuonTable tab;
    tab.count = 0;
    MuonPipe p{};
    int64_t row = 0;
    uint32_t sums = 0, fill = 0;
    int split = 0, parts = 0;
    for (; i < group.last; ++i) {
      const Item x = item_of(list[i]);
      const uint64_t start = pos;
      pos += static_cast<uint64_t>(cdiv(x.rows * x.cols, 256)) * 256;
      if (x.rows == 0 || x.cols == 0) continue;
      const Shape d = shape_of(x.rows, x.cols);
      MuonMat& t = tab.t[tab.count++];
      t = MuonMat{};
      t.src = x.src, t.ld = x.ld, t.mom = x.mom, t.dst = x.dst, t.master = x.master, t.pos = start;
      t.decay = static_cast<float>(x.decay), t.step = static_cast<float>(x.step);
      t.rows = static_cast<int>(x.rows), t.cols = static_cast<int>(x.cols);
      t.mt = static_cast<int>(d.mp / 256), t.nt = static_cast<int>(d.np / 256);
      t.kn = static_cast<int>(cdiv(d.n, 64)), t.km = static_cast<int>(cdiv(d.m, 64));
      t.tall = x.rows > x.cols;
      t.src_vec = aligned_rows(x.src, x.ld, bytes_of(dtype)) && (!x.mom || aligned_rows(x.mom, x.cols, 4));
      t.dst_vec = aligned_rows(x.dst, x.cols, bytes_of(out_dtype)) && (!x.master || aligned_rows(x.master, x.cols, 4));
      t.x[0] = static_cast<uint32_t>(row);
      t.x[1] = static_cast<uint32_t>(row + d.x_rows);
      t.lo = static_cast<uint32_t>(row + 2 * d.x_rows);
      t.a = static_cast<uint32_t>(row + 3 * d.x_rows);
      t.b = static_cast<uint32_t>(row + 3 * d.x_rows + d.a_rows);
      t.sum0 = sums, t.parts = static_cast<uint32_t>(d.parts);
      t.splits = static_cast<int>(splits_of(d, group.tiles)), t.split0 = split, t.part0 = parts;
      for (int k = 0; k < 3; ++k) t.item0[k] = p.items[k];
      const int sym = t.mt * (t.mt + 1) / 2;
      if (t.splits > 1) split += sym, parts += sym * t.splits;
      p.items[kMuonGram] += sym * t.splits, p.items[kMuonPoly] += sym, p.items[kMuonApply] += t.mt * t.nt;
      row += rows_of(d);
      sums += t.parts;
    }
    if (tab.count == 0) continue;
    // One 64 x 64 block a thread block where there are few (each waits for the norm first), up to eight where there are many.
    int64_t blocks = 0;
    for (int k = 0; k < tab.count; ++k) blocks += static_cast<int64_t>(tab.t[k].kn) * tab.t[k].km;
    h.fill_blocks = static_cast<int>(blocks / (8 * dev->sms) < 1 ? 1 : blocks / (8 * dev->sms) > 8 ? 8 : blocks / (8 * dev->sms));
    for (int k = 0; k < tab.count; ++k) {
      tab.t[k].fill0 = fill;
      fill += muon_fill_ctas(tab.t[k], h.fill_blocks);
    }
    CUtensorMap load;
    if ((st = make_map(&load, ws, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 64, row, 128, 64, 64)) != HYLO_OK) return st;
    h.sums = reinterpret_cast<float*>(h.ws + group.sums_at());
    h.ctrl = p.ctrl = reinterpret_cast<unsigned*>(h.ws + group.ctrl_at());
    h.ctrl_words = group.ctrl_words();
    p.scratch = h.ws + group.scratch_at();
    p.parts = h.ws + group.splits_at();
    p.ctl = WaitCtl{dev->status, wait_limit_ns()};
    p.steps = s.count;
    p.half[kMuonApply] = 2 * p.items[kMuonApply] <= dev->muon_clusters;
    p.half[kMuonGram] = split == 0 && halves_are_sooner(tab, dev->muon_clusters, &MuonMat::kn);
    p.half[kMuonPoly] = halves_are_sooner(tab, dev->muon_clusters, &MuonMat::km);
    for (int k = 0; k < s.count; ++k) {
      const double *c = s.k + 3 * k, x = s.x[k], a = s.a[k], b = s.b[k], next = s.x[k + 1];
      p.acc[k][kMuonGram] = static_cast<float>(a / (x * x));
      p.acc[k][kMuonPoly] = static_cast<float>(c[2] * b / (a * a)), p.add[k][kMuonPoly] = static_cast<float>(c[1] * b / a);
      p.acc[k][kMuonApply] = static_cast<float>(next / (b * x)), p.add[k][kMuonApply] = static_cast<float>(c[0] * next / x);
    }
    const int out = !h.muon ? out_dtype == HYLO_BF16 ? kMuonOutBf16 : kMuonOutF16
                            : out_dtype == HYLO_F32 ? kMuonParamF32 : masters ? kMuonParamMaster : kMuonParamBf16;
    cudaError_t e = launch_muon_sums(tab, h, dtype, sums, stream);
    if (e == cudaSuccess) e = launch_muon_fill(tab, h, dtype, fill, stream);
    if (e == cudaSuccess) e = launch_muon_pipe(load, tab, p, h, out, split > 0, dev->muon_clusters, stream);
    if (e != cudaSuccess) return cuda_fail(e, "launch orthogonalised updates");
  }
  return HYLO_OK;
}

template <typename T>
hylo_status check_sides(const T* list, int count) {
  if (count < 0) return fail(HYLO_ERR_DIM, "count=%d", count);
  if (count > 0 && !list) return fail(HYLO_ERR_NULL, "the list of matrices is NULL");
  for (int i = 0; i < count; ++i)
    if (!sides_ok(list[i].rows, list[i].cols))
      return fail(HYLO_ERR_DIM, "matrix %d is %lld x %lld (at most 2^20, the shorter side at most %lld)", i,
                  static_cast<long long>(list[i].rows), static_cast<long long>(list[i].cols), static_cast<long long>(kMaxShort));
  return HYLO_OK;
}

template <typename T>
hylo_status check_workspace(const T* list, int count, void* ws, size_t bytes) {
  if (!ws) return fail(HYLO_ERR_NULL, "workspace is NULL");
  if (!aligned(ws, 256)) return fail(HYLO_ERR_ALIGN, "workspace must be 256-byte aligned");
  const size_t need = workspace(list, count);
  if (bytes < need) return fail(HYLO_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu required", bytes, need);
  return HYLO_OK;
}

void add_span(Span* spans, size_t* n, const void* p, uintptr_t bytes, bool written, int tensor) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  if (p && bytes) spans[(*n)++] = Span{a, a + bytes, written, tensor};
}

}  // namespace

extern "C" {

size_t hylo_orthogonalize_workspace_bytes(const hylo_orth_matrix* matrices, int count) {
  clear_error();
  return check_sides(matrices, count) == HYLO_OK ? workspace(matrices, count) : 0;
}

hylo_status hylo_orthogonalize(const hylo_orth_matrix* matrices, int count, int dtype, int out_dtype, int steps,
                               const double* coefficients, double eps, void* ws, size_t workspace_bytes, cudaStream_t stream) {
  clear_error();
  hylo_status st = check_sides(matrices, count);
  if (st != HYLO_OK) return st;
  if ((dtype != HYLO_F32 && dtype != HYLO_BF16 && dtype != HYLO_F16) || (out_dtype != HYLO_BF16 && out_dtype != HYLO_F16))
    return fail(HYLO_ERR_DIM, "dtype=%d out_dtype=%d (fp32, bf16 or fp16 matrices; bf16 or fp16 results)", dtype, out_dtype);
  Steps s;
  if ((st = plan_steps(steps, coefficients, eps, &s)) != HYLO_OK) return st;
  if ((st = check_workspace(matrices, count, ws, workspace_bytes)) != HYLO_OK) return st;
  const std::unique_ptr<Span[]> spans(new (std::nothrow) Span[2 * static_cast<size_t>(count) + 1]);
  if (!spans) return fail(HYLO_ERR_CUDA, "no host memory for %d matrices", count);
  size_t n = 0;
  for (int i = 0; i < count; ++i) {
    const hylo_orth_matrix& x = matrices[i];
    if (x.rows == 0 || x.cols == 0) continue;
    if (!x.x || !x.out) return fail(HYLO_ERR_NULL, "a required pointer of matrix %d is NULL", i);
    if (x.rows > 1 && (x.ld < x.cols || x.ld > (int64_t(1) << 40)))
      return fail(HYLO_ERR_DIM, "matrix %d: invalid row stride %lld", i, static_cast<long long>(x.ld));
    if (!aligned(x.x, bytes_of(dtype)) || !aligned(x.out, 2)) return fail(HYLO_ERR_ALIGN, "matrix %d is not element-aligned", i);
    const uintptr_t reach = (static_cast<uintptr_t>(x.rows - 1) * (x.rows > 1 ? x.ld : 0) + x.cols) * bytes_of(dtype);
    add_span(spans.get(), &n, x.x, reach, false, i);
    add_span(spans.get(), &n, x.out, static_cast<uintptr_t>(x.rows) * x.cols * 2, true, i);
  }
  add_span(spans.get(), &n, ws, workspace(matrices, count), true, count);
  if ((st = check_spans(spans.get(), n)) != HYLO_OK) return st;
  MuonHyper h{};
  h.eps = static_cast<float>(eps);
  return run(matrices, count, dtype, out_dtype, false, s, h, ws, stream);
}

size_t hylo_muon_workspace_bytes(const hylo_muon_tensor* tensors, int count) {
  clear_error();
  return check_sides(tensors, count) == HYLO_OK ? workspace(tensors, count) : 0;
}

hylo_status hylo_muon_step(const hylo_muon_tensor* tensors, int count, int param_dtype, int grad_dtype, double momentum,
                           int nesterov, int steps, const double* coefficients, double eps, float grad_scale, const float* norm,
                           float max_norm, uint32_t seed, void* ws, size_t workspace_bytes, cudaStream_t stream) {
  clear_error();
  hylo_status st = check_sides(tensors, count);
  if (st != HYLO_OK) return st;
  if ((param_dtype != HYLO_F32 && param_dtype != HYLO_BF16) || (grad_dtype != HYLO_F32 && grad_dtype != HYLO_BF16))
    return fail(HYLO_ERR_DIM, "param_dtype=%d grad_dtype=%d (fp32 or bf16)", param_dtype, grad_dtype);
  if (!(momentum >= 0 && momentum < 1)) return fail(HYLO_ERR_DIM, "momentum=%g (0 <= momentum < 1)", momentum);
  if (!std::isfinite(grad_scale) || (norm && !(max_norm > 0))) return fail(HYLO_ERR_TAU, "grad_scale must be finite and max_norm > 0");
  if (!aligned(norm, 4)) return fail(HYLO_ERR_ALIGN, "norm is not element-aligned");
  Steps s;
  if ((st = plan_steps(steps, coefficients, eps, &s)) != HYLO_OK) return st;
  if ((st = check_workspace(tensors, count, ws, workspace_bytes)) != HYLO_OK) return st;
  const std::unique_ptr<Span[]> spans(new (std::nothrow) Span[4 * static_cast<size_t>(count) + 2]);
  if (!spans) return fail(HYLO_ERR_CUDA, "no host memory for %d tensors", count);
  size_t n = 0;
  int some = -1;  // the first tensor that has elements
  for (int i = 0; i < count; ++i) {
    const hylo_muon_tensor& t = tensors[i];
    if (!std::isfinite(t.lr) || !std::isfinite(t.weight_decay) || !std::isfinite(t.scale))
      return fail(HYLO_ERR_TAU, "lr, weight_decay and scale of tensor %d must be finite", i);
    if (t.rows == 0 || t.cols == 0) continue;
    if (some < 0) some = i;
    if ((t.master != nullptr) != (tensors[some].master != nullptr) || (t.master && param_dtype == HYLO_F32))
      return fail(HYLO_ERR_DIM, "tensor %d: masters go with bf16 parameters, for all tensors or none", i);
    if (!t.param || !t.grad || !t.momentum) return fail(HYLO_ERR_NULL, "a required pointer of tensor %d is NULL", i);
    if (!aligned(t.param, bytes_of(param_dtype)) || !aligned(t.grad, bytes_of(grad_dtype)) || !aligned(t.master, 4) ||
        !aligned(t.momentum, 4))
      return fail(HYLO_ERR_ALIGN, "tensor %d is not element-aligned", i);
    const uintptr_t k = static_cast<uintptr_t>(t.rows) * t.cols;
    add_span(spans.get(), &n, t.param, k * bytes_of(param_dtype), true, i);
    add_span(spans.get(), &n, t.grad, k * bytes_of(grad_dtype), false, i);
    add_span(spans.get(), &n, t.master, k * 4, true, i);
    add_span(spans.get(), &n, t.momentum, k * 4, true, i);
  }
  add_span(spans.get(), &n, norm, 4, false, count);
  add_span(spans.get(), &n, ws, workspace(tensors, count), true, count);
  if ((st = check_spans(spans.get(), n)) != HYLO_OK) return st;
  DeviceState* dev = nullptr;
  if ((st = current_device(&dev)) != HYLO_OK) return st;
  if (some < 0) return HYLO_OK;
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  const cudaError_t asked = cudaStreamIsCapturing(stream, &capture);
  if (asked != cudaSuccess) return cuda_fail(asked, "ask whether the stream is being captured");
  if (capture != cudaStreamCaptureStatusNone)
    return fail(HYLO_ERR_CAPTURE,
                "a Muon step may not be captured: its learning rates and seed are host values that every replay would repeat");
  MuonHyper h{};
  h.muon = 1;
  h.nesterov = nesterov != 0;
  h.mu = static_cast<float>(momentum);
  h.one_minus_mu = static_cast<float>(1.0 - momentum);
  h.grad_scale = grad_scale;
  h.norm = norm;
  h.max_norm = max_norm;
  h.eps = static_cast<float>(eps);
  h.seed = seed;
  return run(tensors, count, grad_dtype, param_dtype, tensors[some].master != nullptr, s, h, ws, stream);
}

}  // extern "C"
