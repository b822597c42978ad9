// Layer norm and RMS norm of rows, with an optional sum of two streams in front, and their backward.
//
//   s = x + residual (rounded to the type of x; s = x without one),  mu = mean(s) (RMS: 0),
//   r = 1 / sqrt(mean((s - mu)^2) + eps),  xh = (s - mu) r,  y = xh w + b
//   g = dy w,  dx = r (g - mean(g) - xh mean(g xh)) + dsum   (RMS: without mean(g))
//   dw = sum over rows of dy xh,  db = sum over rows of dy
//
// HBM bounds both passes. A row is held in registers by the threads that share it, C columns each, so each input crosses HBM
// once and the variance is taken around the mean. The backward keeps the columns' sums of dw and db in registers over all
// rows of a CTA and writes them once; a second small kernel adds the CTAs' sums up in a fixed order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "hylo_ops_internal.h"

namespace hylo {
namespace {

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_float<__half>(float x) { return __float2half_rn(x); }

// VB elements at p, as fp32 (VB elements of T are one access of up to 16 bytes).
template <typename T, int VB>
struct alignas(VB * sizeof(T)) Pack {
  T v[VB];
};

template <typename T, int VB>
__device__ __forceinline__ void load(const T* p, float* out) {
  if constexpr (VB * sizeof(T) > 16) {
    load<T, VB / 2>(p, out);
    load<T, VB / 2>(p + VB / 2, out + VB / 2);
  } else {
    const Pack<T, VB> a = *reinterpret_cast<const Pack<T, VB>*>(p);
#pragma unroll
    for (int j = 0; j < VB; ++j) out[j] = to_float(a.v[j]);
  }
}

template <typename T, int VB>
__device__ __forceinline__ void store(T* p, const float* x) {
  Pack<T, VB> a;
#pragma unroll
  for (int j = 0; j < VB; ++j) a.v[j] = from_float<T>(x[j]);
  *reinterpret_cast<Pack<T, VB>*>(p) = a;
}

// Gain or bias of VB columns, in T or fp32.
template <typename T, int VB>
__device__ __forceinline__ void load_gain(const void* w, bool f32, int64_t c, float* out) {
  if (f32)
    load<float, VB>(static_cast<const float*>(w) + c, out);
  else
    load<T, VB>(static_cast<const T*>(w) + c, out);
}

// Sums of M values over the threads that share a row: a part of a warp, a power of two (`threads` <= 32), or all warps of the
// CTA through `red` (M x 32 floats, another one for each of two consecutive calls).
template <int M>
__device__ __forceinline__ void row_sums(float (&v)[M], int threads, float* red) {
  const int width = threads < 32 ? threads : 32;
  for (int o = width >> 1; o > 0; o >>= 1) {
#pragma unroll
    for (int i = 0; i < M; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  }
  if (threads <= 32) return;
  const int warps = threads >> 5, lane = threadIdx.x & 31;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < M; ++i) red[i * 32 + (threadIdx.x >> 5)] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < M; ++i) v[i] = lane < warps ? red[i * 32 + lane] : 0.f;
  for (int o = 16; o > 0; o >>= 1) {
#pragma unroll
    for (int i = 0; i < M; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  }
}

// One row at a time for each group of p.threads threads, K vectors of VB columns a thread.
template <typename T, int VB, int K>
__global__ void __launch_bounds__(1024) norm_fwd_kernel(const NormParams p) {
  __shared__ float red[2][32];
  const int group = threadIdx.x / p.threads, t = threadIdx.x - group * p.threads;
  const int groups = blockDim.x / p.threads;
  const float inv_d = 1.f / static_cast<float>(p.d);
  for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * groups; row0 < p.N; row0 += static_cast<int64_t>(gridDim.x) * groups) {
    const int64_t row = row0 + group;
    const bool live = row < p.N;
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    float s[K * VB];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * p.threads + t) * VB;
      if (live && c < p.d) {
        load<T, VB>(x + c, s + k * VB);
      } else {
#pragma unroll
        for (int j = 0; j < VB; ++j) s[k * VB + j] = 0.f;
      }
    }
    if (p.residual != nullptr) {
      const T* r = static_cast<const T*>(p.residual) + row * p.ldr;
      T* sum = static_cast<T*>(p.sum) + row * p.d;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int c = (k * p.threads + t) * VB;
        if (live && c < p.d) {
          float a[VB];
          load<T, VB>(r + c, a);
#pragma unroll
          for (int j = 0; j < VB; ++j) s[k * VB + j] = to_float(from_float<T>(s[k * VB + j] + a[j]));  // as the next layer reads it
          store<T, VB>(sum + c, s + k * VB);
        }
      }
    }
    float mu = 0.f;
    if (!p.rms) {
      float v[1] = {0.f};
#pragma unroll
      for (int j = 0; j < K * VB; ++j) v[0] += s[j];
      row_sums(v, p.threads, red[0]);
      mu = v[0] * inv_d;
    }
    float v[1] = {0.f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * p.threads + t) * VB;
      if (c < p.d) {
#pragma unroll
        for (int j = 0; j < VB; ++j) {
          s[k * VB + j] -= mu;
          v[0] = fmaf(s[k * VB + j], s[k * VB + j], v[0]);
        }
      }
    }
    row_sums(v, p.threads, red[1]);
    const float rstd = rsqrtf(fmaf(v[0], inv_d, p.eps));
    if (live && t == 0 && p.stats != nullptr) p.stats[row] = make_float2(mu, rstd);
    T* y = static_cast<T*>(p.y) + row * p.d;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * p.threads + t) * VB;
      if (live && c < p.d) {
        float a[VB];
        if (p.weight != nullptr) {
          load_gain<T, VB>(p.weight, p.gain_f32, c, a);
#pragma unroll
          for (int j = 0; j < VB; ++j) s[k * VB + j] = s[k * VB + j] * rstd * a[j];
        } else {
#pragma unroll
          for (int j = 0; j < VB; ++j) s[k * VB + j] *= rstd;
        }
        if (p.bias != nullptr) {
          load_gain<T, VB>(p.bias, p.gain_f32, c, a);
#pragma unroll
          for (int j = 0; j < VB; ++j) s[k * VB + j] += a[j];
        }
        store<T, VB>(y + c, s + k * VB);
      }
    }
    if (p.rms && p.threads > 32) __syncthreads();  // red[1] is written again by the next row
  }
}

// Rows too wide for the registers: a CTA reads its row again for each of the three steps.
template <typename T, int VB>
__global__ void __launch_bounds__(1024) norm_fwd_wide_kernel(const NormParams p) {
  __shared__ float red[2][32];
  const float inv_d = 1.f / static_cast<float>(p.d);
  for (int64_t row = blockIdx.x; row < p.N; row += gridDim.x) {
    const T* s = static_cast<const T*>(p.x) + row * p.ldx;
    float a[VB], b[VB];
    if (p.residual != nullptr) {
      const T* r = static_cast<const T*>(p.residual) + row * p.ldr;
      T* sum = static_cast<T*>(p.sum) + row * p.d;
      for (int c = threadIdx.x * VB; c < p.d; c += blockDim.x * VB) {
        load<T, VB>(s + c, a);
        load<T, VB>(r + c, b);
#pragma unroll
        for (int j = 0; j < VB; ++j) a[j] += b[j];
        store<T, VB>(sum + c, a);
      }
      s = sum;  // below every thread reads what it wrote itself
    }
    float mu = 0.f;
    if (!p.rms) {
      float v[1] = {0.f};
      for (int c = threadIdx.x * VB; c < p.d; c += blockDim.x * VB) {
        load<T, VB>(s + c, a);
#pragma unroll
        for (int j = 0; j < VB; ++j) v[0] += a[j];
      }
      row_sums(v, blockDim.x, red[0]);
      mu = v[0] * inv_d;
    }
    float v[1] = {0.f};
    for (int c = threadIdx.x * VB; c < p.d; c += blockDim.x * VB) {
      load<T, VB>(s + c, a);
#pragma unroll
      for (int j = 0; j < VB; ++j) v[0] = fmaf(a[j] - mu, a[j] - mu, v[0]);
    }
    row_sums(v, blockDim.x, red[1]);
    const float rstd = rsqrtf(fmaf(v[0], inv_d, p.eps));
    if (threadIdx.x == 0 && p.stats != nullptr) p.stats[row] = make_float2(mu, rstd);
    T* y = static_cast<T*>(p.y) + row * p.d;
    for (int c = threadIdx.x * VB; c < p.d; c += blockDim.x * VB) {
      load<T, VB>(s + c, a);
#pragma unroll
      for (int j = 0; j < VB; ++j) a[j] = (a[j] - mu) * rstd;
      if (p.weight != nullptr) {
        load_gain<T, VB>(p.weight, p.gain_f32, c, b);
#pragma unroll
        for (int j = 0; j < VB; ++j) a[j] *= b[j];
      }
      if (p.bias != nullptr) {
        load_gain<T, VB>(p.bias, p.gain_f32, c, b);
#pragma unroll
        for (int j = 0; j < VB; ++j) a[j] += b[j];
      }
      store<T, VB>(y + c, a);
    }
    __syncthreads();  // both halves of red are written again by the next row
  }
}

// The gradients, with the columns' sums of this CTA's rows: part [2][CTAs][d] (dw, then db).
template <typename T, int VB, int K>
__global__ void __launch_bounds__(1024) norm_bwd_kernel(const NormParams p, const NormGrad q) {
  constexpr int C = K * VB;
  extern __shared__ float shared[];  // [2][2][32] sums of rows, then [groups][d] columns' sums where a CTA has several groups
  const int group = threadIdx.x / p.threads, t = threadIdx.x - group * p.threads;
  const int groups = blockDim.x / p.threads;
  const float inv_d = 1.f / static_cast<float>(p.d);
  float dw[C], db[C];
#pragma unroll
  for (int j = 0; j < C; ++j) dw[j] = db[j] = 0.f;
  int flip = 0;
  for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * groups; row0 < p.N; row0 += static_cast<int64_t>(gridDim.x) * groups) {
    const int64_t row = row0 + group;
    const bool live = row < p.N;
    const T* s = static_cast<const T*>(p.x) + row * p.ldx;
    const T* dy = static_cast<const T*>(q.dy) + row * q.lddy;
    float xh[C], g[C];
    const float2 st = live ? p.stats[row] : make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * p.threads + t) * VB;
      if (live && c < p.d) {
        load<T, VB>(s + c, xh + k * VB);
        load<T, VB>(dy + c, g + k * VB);
      } else {
#pragma unroll
        for (int j = 0; j < VB; ++j) {
          xh[k * VB + j] = st.x;
          g[k * VB + j] = 0.f;
        }
      }
    }
    float v[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * p.threads + t) * VB;
      float a[VB];
      if (p.weight != nullptr && c < p.d) load_gain<T, VB>(p.weight, p.gain_f32, c, a);
#pragma unroll
      for (int j = k * VB; j < (k + 1) * VB; ++j) {
        xh[j] = (xh[j] - st.x) * st.y;
        dw[j] = fmaf(g[j], xh[j], dw[j]);
        db[j] += g[j];
        if (p.weight != nullptr && c < p.d) g[j] *= a[j - k * VB];
        v[0] = fmaf(g[j], xh[j], v[0]);
        v[1] += g[j];
      }
    }
    if (q.dx == nullptr) continue;
    row_sums(v, p.threads, shared + flip * 64);
    flip ^= 1;
    const float c1 = v[0] * inv_d, c2 = p.rms ? 0.f : v[1] * inv_d;
    T* dx = static_cast<T*>(q.dx) + row * p.d;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * p.threads + t) * VB;
      if (live && c < p.d) {
#pragma unroll
        for (int j = k * VB; j < (k + 1) * VB; ++j) g[j] = st.y * (g[j] - c2 - xh[j] * c1);
        if (q.dsum != nullptr) {
          float a[VB];
          load<T, VB>(static_cast<const T*>(q.dsum) + row * q.ldds + c, a);
#pragma unroll
          for (int j = 0; j < VB; ++j) g[k * VB + j] += a[j];
        }
        store<T, VB>(dx + c, g + k * VB);
      }
    }
  }
  grid_dep_launch();
  if (q.part == nullptr) return;
  float* part = q.part + static_cast<int64_t>(blockIdx.x) * p.d;
  const int64_t second = static_cast<int64_t>(gridDim.x) * p.d;
  if (groups == 1) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * p.threads + t) * VB;
      if (c < p.d) {
        if (q.want_dw) store<float, (VB > 4 ? 4 : VB)>(part + c, dw + k * VB);
        if (q.want_db) store<float, (VB > 4 ? 4 : VB)>(part + second + c, db + k * VB);
        if constexpr (VB > 4) {
          if (q.want_dw) store<float, 4>(part + c + 4, dw + k * VB + 4);
          if (q.want_db) store<float, 4>(part + second + c + 4, db + k * VB + 4);
        }
      }
    }
    return;
  }
  float* cols = shared + 128;
  for (int pass = 0; pass < 2; ++pass) {
    if (pass == 0 ? !q.want_dw : !q.want_db) continue;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * p.threads + t) * VB;
      if (c < p.d) {
#pragma unroll
        for (int j = 0; j < VB; ++j) cols[group * p.d + c + j] = pass == 0 ? dw[k * VB + j] : db[k * VB + j];
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < p.d; c += blockDim.x) {
      float a = 0.f;
      for (int i = 0; i < groups; ++i) a += cols[i * p.d + c];
      part[pass * second + c] = a;
    }
  }
}

// dx of rows too wide for the registers.
template <typename T, int VB>
__global__ void __launch_bounds__(1024) norm_bwd_wide_kernel(const NormParams p, const NormGrad q) {
  __shared__ float red[2][32];
  const float inv_d = 1.f / static_cast<float>(p.d);
  for (int64_t row = blockIdx.x; row < p.N; row += gridDim.x) {
    const T* s = static_cast<const T*>(p.x) + row * p.ldx;
    const T* dy = static_cast<const T*>(q.dy) + row * q.lddy;
    const float2 st = p.stats[row];
    float xh[VB], g[VB], a[VB], v[2] = {0.f, 0.f};
    auto read = [&](int c) {
      load<T, VB>(s + c, xh);
      load<T, VB>(dy + c, g);
      if (p.weight != nullptr) load_gain<T, VB>(p.weight, p.gain_f32, c, a);
#pragma unroll
      for (int j = 0; j < VB; ++j) {
        xh[j] = (xh[j] - st.x) * st.y;
        if (p.weight != nullptr) g[j] *= a[j];
      }
    };
    for (int c = threadIdx.x * VB; c < p.d; c += blockDim.x * VB) {
      read(c);
#pragma unroll
      for (int j = 0; j < VB; ++j) {
        v[0] = fmaf(g[j], xh[j], v[0]);
        v[1] += g[j];
      }
    }
    row_sums(v, blockDim.x, red[0]);
    const float c1 = v[0] * inv_d, c2 = p.rms ? 0.f : v[1] * inv_d;
    T* dx = static_cast<T*>(q.dx) + row * p.d;
    for (int c = threadIdx.x * VB; c < p.d; c += blockDim.x * VB) {
      read(c);
#pragma unroll
      for (int j = 0; j < VB; ++j) g[j] = st.y * (g[j] - c2 - xh[j] * c1);
      if (q.dsum != nullptr) {
        load<T, VB>(static_cast<const T*>(q.dsum) + row * q.ldds + c, a);
#pragma unroll
        for (int j = 0; j < VB; ++j) g[j] += a[j];
      }
      store<T, VB>(dx + c, g);
    }
    __syncthreads();  // red is written again by the next row
  }
}

// The columns' sums of rows blockIdx.y, blockIdx.y + gridDim.y, ... for 1024 / sizeof(T) columns a CTA, read once more.
template <typename T>
__global__ void __launch_bounds__(256) norm_columns_kernel(const NormParams p, const NormGrad q) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c < p.d) {
    float dw = 0.f, db = 0.f;
    for (int64_t row = blockIdx.y; row < p.N; row += gridDim.y) {
      const float2 st = p.stats[row];
      const float g = to_float(static_cast<const T*>(q.dy)[row * q.lddy + c]);
      dw = fmaf(g, (to_float(static_cast<const T*>(p.x)[row * p.ldx + c]) - st.x) * st.y, dw);
      db += g;
    }
    if (q.want_dw) q.part[static_cast<int64_t>(blockIdx.y) * p.d + c] = dw;
    if (q.want_db) q.part[(static_cast<int64_t>(gridDim.y) + blockIdx.y) * p.d + c] = db;
  }
  grid_dep_launch();
}

// dw (blockIdx.y 0) and db (1): the sums of `parts` rows of part in a fixed order. 32 columns a CTA, kSlices threads a column.
constexpr int kSlices = 16;
template <typename G>
__global__ void __launch_bounds__(32 * kSlices) norm_join_kernel(const float* part, int parts, int d, void* dw, void* db) {
  __shared__ float red[kSlices][33];
  grid_dep_wait();
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int which = dw == nullptr ? 1 : blockIdx.y, c = blockIdx.x * 32 + lane;
  const float* a = part + static_cast<int64_t>(which) * parts * d;
  float sum = 0.f;
  if (c < d) {
#pragma unroll 4
    for (int i = slice; i < parts; i += kSlices) sum += a[static_cast<int64_t>(i) * d + c];
  }
  red[slice][lane] = sum;
  __syncthreads();
  if (slice == 0 && c < d) {
    for (int i = 1; i < kSlices; ++i) sum += red[i][lane];
    static_cast<G*>(which == 0 ? dw : db)[c] = from_float<G>(sum);
  }
}

template <typename... A, typename... B>
cudaError_t launch(void (*kernel)(A...), dim3 grid, int threads, size_t smem, cudaStream_t stream, bool dependent, B... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = dependent ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<A>(args)...);
}

int round_threads(int64_t n) {  // a power of two up to a warp, whole warps above
  if (n > 32) return static_cast<int>((n + 31) / 32 * 32);
  int t = 1;
  while (t < n) t *= 2;
  return t;
}

bool vectors(const void* p, int64_t ld, int64_t N, int64_t bytes, int64_t unit) {
  return reinterpret_cast<uintptr_t>(p) % unit == 0 && (N == 1 || ld * bytes % unit == 0);
}

int64_t cdiv64(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int kBwdCols = 8;    // columns of a thread in the backward: 16 sums, and a row's 1024 threads have 64 registers each
constexpr int kGridSms = 152;  // the workspace's size may not depend on the device

template <typename T, int VB, int K>
cudaError_t fwd(NormParams p, int sms, cudaStream_t stream) {
  p.threads = round_threads(cdiv64(p.d, VB * K));
  const int cta = p.threads > 32 ? p.threads : 128;
  const int64_t blocks = cdiv64(p.N, cta / p.threads), most = static_cast<int64_t>(sms) * (2048 / cta);
  return launch(norm_fwd_kernel<T, VB, K>, dim3(static_cast<unsigned>(blocks < most ? blocks : most)), cta, 0, stream, false, p);
}

template <typename T, int VB>
cudaError_t fwd_cols(const NormParams& p, int sms, cudaStream_t stream) {
  if (p.d <= 512 || (p.d <= 8192 && p.N <= 2 * sms)) return fwd<T, VB, 8 / VB>(p, sms, stream);
  if (p.d <= 16384) return fwd<T, VB, 16 / VB>(p, sms, stream);
  if (p.d <= 32768) return fwd<T, VB, 32 / VB>(p, sms, stream);
  const int64_t most = 2 * static_cast<int64_t>(sms);
  return launch(norm_fwd_wide_kernel<T, VB>, dim3(static_cast<unsigned>(p.N < most ? p.N : most)), 1024, 0, stream, false, p);
}

template <typename T>
cudaError_t fwd_type(const NormParams& p, int sms, cudaStream_t stream) {
  constexpr int VB = 16 / sizeof(T);
  const int64_t e = sizeof(T), ge = p.gain_f32 ? 4 : e;
  const bool vec = p.d % VB == 0 && vectors(p.x, p.ldx, p.N, e, 16) && vectors(p.residual, p.ldr, p.N, e, 16) &&
                   vectors(p.sum, p.d, p.N, e, 16) && vectors(p.y, p.d, p.N, e, 16) && vectors(p.weight, 0, 1, ge, 16) &&
                   vectors(p.bias, 0, 1, ge, 16);
  return vec ? fwd_cols<T, VB>(p, sms, stream) : fwd_cols<T, 1>(p, sms, stream);
}

template <typename T, int VB, int K>
cudaError_t bwd(NormParams p, const NormGrad& q, int ctas, cudaStream_t stream) {
  static_assert(VB * K == kBwdCols);
  p.threads = round_threads(cdiv64(p.d, kBwdCols));
  const int cta = p.threads > 32 ? p.threads : 128;
  const int groups = cta / p.threads;
  const size_t smem = 128 * sizeof(float) + (groups > 1 ? static_cast<size_t>(groups) * p.d * sizeof(float) : 0);
  return launch(norm_bwd_kernel<T, VB, K>, dim3(ctas), cta, smem, stream, false, p, q);
}

template <typename T, int VB>
cudaError_t bwd_cols(const NormParams& p, const NormGrad& q, int ctas, int sms, cudaStream_t stream) {
  if (p.d <= kNormFusedCols) return bwd<T, VB, kBwdCols / VB>(p, q, ctas, stream);
  cudaError_t e = cudaSuccess;
  if (q.dx != nullptr) {
    const int64_t most = 2 * static_cast<int64_t>(sms);
    e = launch(norm_bwd_wide_kernel<T, VB>, dim3(static_cast<unsigned>(p.N < most ? p.N : most)), 1024, 0, stream, false, p, q);
  }
  if (e == cudaSuccess && q.part != nullptr)
    e = launch(norm_columns_kernel<T>, dim3(static_cast<unsigned>(cdiv64(p.d, 256)), ctas), 256, 0, stream, false, p, q);
  return e;
}

template <typename T>
cudaError_t bwd_type(const NormParams& p, const NormGrad& q, int ctas, int sms, cudaStream_t stream) {
  constexpr int VB = 16 / sizeof(T);
  const int64_t e = sizeof(T), ge = p.gain_f32 ? 4 : e;
  const bool vec = p.d % VB == 0 && vectors(p.x, p.ldx, p.N, e, 16) && vectors(q.dy, q.lddy, p.N, e, 16) &&
                   vectors(q.dsum, q.ldds, p.N, e, 16) && vectors(q.dx, p.d, p.N, e, 16) && vectors(p.weight, 0, 1, ge, 16);
  cudaError_t err = vec ? bwd_cols<T, VB>(p, q, ctas, sms, stream) : bwd_cols<T, 1>(p, q, ctas, sms, stream);
  if (err != cudaSuccess || q.part == nullptr) return err;
  const dim3 grid(static_cast<unsigned>(cdiv64(p.d, 32)), q.want_dw && q.want_db ? 2 : 1);
  void* dw = q.want_dw ? q.dw : nullptr;
  if (p.gain_f32) return launch(norm_join_kernel<float>, grid, 32 * kSlices, 0, stream, true, q.part, ctas, p.d, dw, q.db);
  return launch(norm_join_kernel<T>, grid, 32 * kSlices, 0, stream, true, q.part, ctas, p.d, dw, q.db);
}

}  // namespace

int norm_parts(int64_t N, int d) {
  if (d > kNormFusedCols) {
    const int64_t want = cdiv64(8 * kGridSms, cdiv64(d, 256));
    return static_cast<int>(N < want ? N : want);
  }
  const int threads = round_threads(cdiv64(d, kBwdCols)), cta = threads > 32 ? threads : 128;
  const int64_t blocks = cdiv64(N, cta / threads), most = kGridSms * (1024 / cta);
  return static_cast<int>(blocks < most ? blocks : most);
}

cudaError_t launch_norm(const NormParams& p, int dtype, int sms, cudaStream_t stream) {
  if (dtype == HYLO_F32) return fwd_type<float>(p, sms, stream);
  if (dtype == HYLO_BF16) return fwd_type<__nv_bfloat16>(p, sms, stream);
  return fwd_type<__half>(p, sms, stream);
}

cudaError_t launch_norm_bwd(const NormParams& p, const NormGrad& q, int dtype, int ctas, int sms, cudaStream_t stream) {
  if (dtype == HYLO_F32) return bwd_type<float>(p, q, ctas, sms, stream);
  if (dtype == HYLO_BF16) return bwd_type<__nv_bfloat16>(p, q, ctas, sms, stream);
  return bwd_type<__half>(p, q, ctas, sms, stream);
}

}  // namespace hylo
