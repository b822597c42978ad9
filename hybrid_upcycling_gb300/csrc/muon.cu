// The elementwise kernels around the Newton-Schulz products of orthogonalised updates: momentum and sums of squares, and
// the scaled update as fp16 panels. HBM bounds both: 67M bf16 gradients with their momenta 101 us (0.98 of a copy's
// rate) and 131 us (0.76: every piece waits for its loads; the products take 1.6 ms); without momenta the three sums of squares
// are instructions, 41 us; the layout of the workspace is in muon.h, the parameters' step in muon_pipe.cu.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "hylo_ops_internal.h"
#include "muon.h"

namespace hylo {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_float(float x, float* y) { *y = x; }

template <typename T>
struct alignas(16) Pack16 {
  T v[16 / sizeof(T)];
};

// Eight elements at p, `left` of which exist; missing ones are 0.
template <typename T>
__device__ __forceinline__ void load8(const T* p, int left, bool vec, float* z) {
  if (vec && left >= 8) {
    constexpr int E = 16 / sizeof(T);
#pragma unroll
    for (int k = 0; k < 8 / E; ++k) {
      const Pack16<T> a = reinterpret_cast<const Pack16<T>*>(p)[k];
#pragma unroll
      for (int j = 0; j < E; ++j) z[k * E + j] = to_float(a.v[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) z[j] = j < left ? to_float(p[j]) : 0.f;
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, int left, bool vec, const float* z) {
  if (vec && left >= 8) {
    constexpr int E = 16 / sizeof(T);
#pragma unroll
    for (int k = 0; k < 8 / E; ++k) {
      Pack16<T> a;
#pragma unroll
      for (int j = 0; j < E; ++j) from_float(z[k * E + j], &a.v[j]);
      reinterpret_cast<Pack16<T>*>(p)[k] = a;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < left) from_float(z[j], p + j);
  }
}

// The factor on the gradients; false if the step is skipped.
__device__ __forceinline__ bool gradient_factor(const MuonHyper& h, float& gs) {
  gs = h.grad_scale;
  if (h.norm != nullptr) {
    const float norm = h.norm[0];
    if (!isfinite(norm)) return false;
    gs *= fminf(1.f, h.max_norm / (norm * fabsf(h.grad_scale) + 1e-6f));
  }
  return true;
}

template <uint32_t MuonMat::* START>
__device__ __forceinline__ int find_mat(const MuonTable& tab, uint32_t b) {
  int lo = 0, hi = tab.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tab.t[mid].*START <= b)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// The update before it is orthogonalised, from the gradient (scaled) and the momentum after this step's.
__device__ __forceinline__ float update_of(const MuonHyper& h, float g, float m) {
  return h.nesterov ? fmaf(h.mu, m, h.one_minus_mu * g) : m;
}

__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) s += red[i];
  return s;
}

// Momentum, and the sums of squares of the update. Squares of very small and very large values leave fp32's range, so there are
// three sums, of x 2^80, x and x 2^-80, of which square_sum() takes one that did not. A thread block's pieces of
// eight elements of a row lie `parts` blocks apart, whatever the row stride, so that results do not depend on it.
constexpr float kUp = 0x1p80f, kDown = 0x1p-80f;
template <typename T>
__global__ void __launch_bounds__(kThreads) muon_sums_kernel(const __grid_constant__ MuonTable tab, const MuonHyper h) {
  __shared__ float red[kThreads / 32];
  if (blockIdx.x == 0) {
    for (int i = threadIdx.x; i < h.ctrl_words; i += kThreads) h.ctrl[i] = 0u;
  }
  float gs = 1.f;
  if (h.muon && !gradient_factor(h, gs)) return;
  const MuonMat& t = tab.t[find_mat<&MuonMat::sum0>(tab, blockIdx.x)];
  const uint32_t per_row = static_cast<uint32_t>(t.cols + 7) / 8;
  const int64_t pieces = static_cast<int64_t>(per_row) * t.rows;
  const bool vec = t.src_vec != 0;
  const T* src = static_cast<const T*>(t.src);
  float sum[kMuonSums] = {0.f, 0.f, 0.f};
  for (int64_t piece = static_cast<int64_t>(blockIdx.x - t.sum0) * kThreads + threadIdx.x; piece < pieces;
       piece += static_cast<int64_t>(t.parts) * kThreads) {
    const int64_t r = pieces < (int64_t(1) << 32) ? static_cast<uint32_t>(piece) / per_row : piece / per_row;
    const int c = static_cast<int>(piece - r * per_row) * 8, left = min(8, t.cols - c);
    float x[8];
    load8(src + r * t.ld + c, left, vec, x);
    if (h.muon) {  // gradients and momentum have no gaps
      float m[8];
      load8(t.mom + r * t.ld + c, left, vec, m);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float g = x[j] * gs;
        m[j] = fmaf(h.mu, m[j], h.one_minus_mu * g);
        x[j] = update_of(h, g, m[j]);
      }
      store8(t.mom + r * t.ld + c, left, vec, m);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float up = x[j] * kUp, down = x[j] * kDown;
      sum[0] = fmaf(up, up, sum[0]);
      sum[1] = fmaf(x[j], x[j], sum[1]);
      sum[2] = fmaf(down, down, sum[2]);
    }
  }
#pragma unroll
  for (int k = 0; k < kMuonSums; ++k) {
    const float s = block_sum(sum[k], red);
    if (threadIdx.x == 0) h.sums[static_cast<int64_t>(blockIdx.x) * kMuonSums + k] = s;
  }
}

// Two factors whose product is scale / (norm + eps): one alone could leave fp32's range. NaN if the norm is not finite. One thread
// works in 64 bits, which are slow here.
__device__ __forceinline__ float2 scale_factors(const MuonMat& t, const MuonHyper& h, float* red) {
  float s[kMuonSums] = {0.f, 0.f, 0.f};
  for (uint32_t i = threadIdx.x; i < t.parts; i += kThreads) {
    const float* a = h.sums + static_cast<int64_t>(t.sum0 + i) * kMuonSums;
#pragma unroll
    for (int k = 0; k < kMuonSums; ++k) s[k] += a[k];
  }
#pragma unroll
  for (int k = 0; k < kMuonSums; ++k) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s[k] += __shfl_xor_sync(0xffffffffu, s[k], o);
    if ((threadIdx.x & 31) == 0) red[k * (kThreads / 32) + (threadIdx.x >> 5)] = s[k];
  }
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int k = 0; k < kMuonSums; ++k) {
      s[k] = 0.f;
      for (int i = 0; i < kThreads / 32; ++i) s[k] += red[k * (kThreads / 32) + i];
    }
    // all sums of magnitudes below 2^-20: x 2^80 stays below 2^60 and loses nothing; inf: x 2^-80 does not overflow
    const double root = sqrt(static_cast<double>(s[1] < 0x1p-40f ? s[0] : isfinite(s[1]) ? s[1] : s[2]));
    const double norm = s[1] < 0x1p-40f ? root * 0x1p-80 : isfinite(s[1]) ? root : root * 0x1p80;
    const double f = norm > 0.0 || h.eps > 0.f ? static_cast<double>(h.scale_in) / (norm + h.eps) : 0.0;
    const double first = f > 0x1p100 ? 0x1p100 : f < 0x1p-100 ? 0x1p-100 : 1.0;
    const bool fine = isfinite(norm);
    red[0] = fine ? static_cast<float>(f / first) : __int_as_float(0x7fffffff);
    red[1] = fine ? static_cast<float>(first) : 1.f;
  }
  __syncthreads();
  return make_float2(red[0], red[1]);
}

// Eight columns from c on of X's row r.
__device__ __forceinline__ void put_x(const MuonHyper& h, const MuonMat& t, int r, int c, const float* u, float2 f) {
  uint32_t hi[4], lo[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float a = u[2 * j] * f.y * f.x, b = u[2 * j + 1] * f.y * f.x;
    const __half2 p = __floats2half2_rn(a, b);
    const float2 r2 = __half22float2(p);
    const __half2 q = __floats2half2_rn(a - r2.x, b - r2.y);
    hi[j] = *reinterpret_cast<const uint32_t*>(&p);
    lo[j] = *reinterpret_cast<const uint32_t*>(&q);
  }
  const size_t at = (static_cast<size_t>(c >> 6) * t.mt * 256 + r) * 128 + (c & 63) * 2;
  *reinterpret_cast<uint4*>(h.ws + static_cast<size_t>(t.x[0]) * 128 + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  const int warp = (r >> 5 & 3) + (c >> 7 & 1) * 4;
  const int64_t sector = muon_lo_sector((c >> 8) * t.mt + (r >> 8), r >> 7 & 1, warp) + (c >> 4 & 7) * 32 + (r & 31);
  *reinterpret_cast<uint4*>(h.ws + static_cast<size_t>(t.lo) * 128 + sector * 32 + (c & 8) * 2) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
}

// X's panels from the scaled update, padded with zeros to whole k-blocks: 64 x 64 blocks of the matrix, h.fill_blocks a thread block
// along its rows; a tall matrix is transposed through shared memory.
template <typename T>
__global__ void __launch_bounds__(kThreads) muon_fill_kernel(const __grid_constant__ MuonTable tab, const MuonHyper h) {
  __shared__ float red[kMuonSums * (kThreads / 32)];
  __shared__ float tile[64][65];
  const MuonMat& t = tab.t[find_mat<&MuonMat::fill0>(tab, blockIdx.x)];
  float gs = 1.f;
  const bool skipped = h.muon && !gradient_factor(h, gs);
  float2 f = make_float2(0.f, 0.f);
  if (!skipped) f = scale_factors(t, h, red);
  const int wide = t.tall ? t.km : t.kn, local = static_cast<int>(blockIdx.x - t.fill0);
  const int per = (wide + h.fill_blocks - 1) / h.fill_blocks;
  const int br = local / per, bc0 = (local - br * per) * h.fill_blocks;
  for (int bc = bc0; bc < min(wide, bc0 + h.fill_blocks); ++bc) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int rr = half * 32 + static_cast<int>(threadIdx.x >> 3), cc = static_cast<int>(threadIdx.x & 7) * 8;
      const int r = br * 64 + rr, c = bc * 64 + cc;
      float u[8];
      const int left = r < t.rows && !skipped ? max(0, min(8, t.cols - c)) : 0;
      load8(static_cast<const T*>(t.src) + static_cast<int64_t>(r) * t.ld + c, left, t.src_vec != 0, u);
      if (h.muon) {
        float m[8];
        load8(t.mom + static_cast<int64_t>(r) * t.ld + c, left, t.src_vec != 0, m);
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j] = update_of(h, u[j] * gs, m[j]);
      }
      if (t.tall) {
#pragma unroll
        for (int j = 0; j < 8; ++j) tile[rr][cc + j] = u[j];
      } else {
        put_x(h, t, r, c, u, f);
      }
    }
    if (t.tall) {
      __syncthreads();
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int xr = half * 32 + static_cast<int>(threadIdx.x >> 3), xc = static_cast<int>(threadIdx.x & 7) * 8;
        float u[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j] = tile[xc + j][xr];
        put_x(h, t, bc * 64 + xr, br * 64 + xc, u, f);
      }
      __syncthreads();
    }
  }
}

}  // namespace

uint32_t muon_fill_ctas(const MuonMat& t, int blocks) {
  const int down = t.tall ? t.kn : t.km, across = t.tall ? t.km : t.kn;  // 64 x 64 blocks
  return static_cast<uint32_t>(down) * static_cast<uint32_t>((across + blocks - 1) / blocks);
}

cudaError_t launch_muon_sums(const MuonTable& t, const MuonHyper& h, int dtype, uint32_t ctas, cudaStream_t stream) {
  if (dtype == HYLO_F32)
    muon_sums_kernel<float><<<ctas, kThreads, 0, stream>>>(t, h);
  else if (dtype == HYLO_BF16)
    muon_sums_kernel<__nv_bfloat16><<<ctas, kThreads, 0, stream>>>(t, h);
  else
    muon_sums_kernel<__half><<<ctas, kThreads, 0, stream>>>(t, h);
  return cudaGetLastError();
}

cudaError_t launch_muon_fill(const MuonTable& t, const MuonHyper& h, int dtype, uint32_t ctas, cudaStream_t stream) {
  if (dtype == HYLO_F32)
    muon_fill_kernel<float><<<ctas, kThreads, 0, stream>>>(t, h);
  else if (dtype == HYLO_BF16)
    muon_fill_kernel<__nv_bfloat16><<<ctas, kThreads, 0, stream>>>(t, h);
  else
    muon_fill_kernel<__half><<<ctas, kThreads, 0, stream>>>(t, h);
  return cudaGetLastError();
}

}  // namespace hylo
