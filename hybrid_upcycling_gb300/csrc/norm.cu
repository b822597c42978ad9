// Layer norm and RMS norm of rows, with an optional sum of two streams in front, and their backward.
//
//   s = x + residual (rounded to the type of x; s = x without one),  mu = mean(s) (RMS: 0),
//   r = 1 / sqrt(mean((s - mu)^2) + eps),  xh = (s - mu) r,  y = xh w + b
//   g = dy w,  dx = r (g - mean(g) - xh mean(g xh)) + dsum   (RMS: without mean(g))
//   dw = sum over rows of dy xh,  db = sum over rows of dy
//
// HBM bounds both passes, so each input is read once and what is still needed of it stays in registers, in its own type.
//
// Rows of 16-byte vectors: every thread copies the vectors that it will use itself into its own places of a ring in shared memory
// (cp.async), several rows ahead, so that an SM has 100 KB and more on their way without a register or a barrier for them. (One row
// ahead in registers: 0.5 of HBM's rate in the backward, and rows that wait for one another in the forward.) Other rows go by
// single elements through registers.
//
// Backward: a thread takes the same columns of all rows of its CTA, so that the sums of dw and db stay in registers; each CTA
// writes them once and a second small kernel adds them up in a fixed order. Rows of more than 4096 columns are shared by a cluster
// of CTAs of up to 8192 columns, which exchange their sums through distributed shared memory and form a row's dx only after
// the next row's sums, so that nobody waits for the exchange.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <type_traits>

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

// VB elements as they lie in memory (one access of up to 16 bytes). Two at a time are converted by one instruction.
template <typename T, int VB>
struct alignas(VB * sizeof(T)) Pack {
  T v[VB];
  __device__ __forceinline__ void get(float* x) const {
    if constexpr (sizeof(T) == 2 && VB % 2 == 0) {
#pragma unroll
      for (int j = 0; j < VB; j += 2) {
        const uint32_t w = reinterpret_cast<const uint32_t*>(v)[j / 2];
        if constexpr (std::is_same<T, __half>::value) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
          x[j] = f.x, x[j + 1] = f.y;
        } else {
          x[j] = __uint_as_float(w << 16), x[j + 1] = __uint_as_float(w & 0xffff0000u);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < VB; ++j) x[j] = to_float(v[j]);
    }
  }
  __device__ __forceinline__ void set(const float* x) {
    if constexpr (sizeof(T) == 2 && VB % 2 == 0) {
#pragma unroll
      for (int j = 0; j < VB; j += 2) {
        uint32_t w;
        if constexpr (std::is_same<T, __half>::value) {
          const __half2 h = __floats2half2_rn(x[j], x[j + 1]);
          w = *reinterpret_cast<const uint32_t*>(&h);
        } else {
          w = pack_bf16x2(x[j], x[j + 1]);
        }
        reinterpret_cast<uint32_t*>(v)[j / 2] = w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < VB; ++j) v[j] = from_float<T>(x[j]);
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < VB; ++j) v[j] = from_float<T>(0.f);
  }
};

template <typename T, int VB>
__device__ __forceinline__ void load(const T* p, float* out) {
  if constexpr (VB * sizeof(T) > 16) {
    load<T, VB / 2>(p, out);
    load<T, VB / 2>(p + VB / 2, out + VB / 2);
  } else {
    reinterpret_cast<const Pack<T, VB>*>(p)->get(out);
  }
}

template <typename T, int VB>
__device__ __forceinline__ void store(T* p, const float* x) {
  Pack<T, VB> a;
  a.set(x);
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
  int top = 16;
  while (top >= warps) top >>= 1;
  for (int o = top; o > 0; o >>= 1) {
#pragma unroll
    for (int i = 0; i < M; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  }
  if (top < 16) {
#pragma unroll
    for (int i = 0; i < M; ++i) v[i] = __shfl_sync(0xffffffffu, v[i], 0);
  }
}

// Two fp32 operations by one instruction.
__device__ __forceinline__ float2 two(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 pair(const float* x) { return make_float2(x[0], x[1]); }
// x <- (x - mu) r, in this order: r may be large beside 1 / mu. CENTRE false: mu is 0.
template <bool CENTRE, int N>
__device__ __forceinline__ void normalise(float (&x)[N], float mu, float r) {
#pragma unroll
  for (int j = 0; j + 1 < N; j += 2) {
    float2 y = pair(x + j);
    if (CENTRE) y = __fadd2_rn(y, two(-mu));
    y = __fmul2_rn(y, two(r));
    x[j] = y.x, x[j + 1] = y.y;
  }
  if constexpr (N % 2 == 1) x[N - 1] = (CENTRE ? x[N - 1] - mu : x[N - 1]) * r;
}
template <int N>
__device__ __forceinline__ void times(float (&x)[N], const float (&a)[N]) {
#pragma unroll
  for (int j = 0; j + 1 < N; j += 2) {
    const float2 y = __fmul2_rn(pair(x + j), pair(a + j));
    x[j] = y.x, x[j + 1] = y.y;
  }
  if constexpr (N % 2 == 1) x[N - 1] *= a[N - 1];
}
template <int N>
__device__ __forceinline__ void plus(float (&x)[N], const float (&a)[N]) {
#pragma unroll
  for (int j = 0; j + 1 < N; j += 2) {
    const float2 y = __fadd2_rn(pair(x + j), pair(a + j));
    x[j] = y.x, x[j + 1] = y.y;
  }
  if constexpr (N % 2 == 1) x[N - 1] += a[N - 1];
}

// Few rows, each by a group of p.threads threads that have one vector of VB columns: what counts is the time of one row.
template <typename T, int VB>
__global__ void __launch_bounds__(1024) norm_fwd_kernel(const NormParams p) {
  using V = Pack<T, VB>;
  __shared__ float red[2][32];
  const int group = threadIdx.x / p.threads, t = threadIdx.x - group * p.threads, c = t * VB;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / p.threads) + group;
  const bool mine = row < p.N && c < p.d;
  const float inv_d = 1.f / static_cast<float>(p.d);
  V raw;
  raw.clear();
  if (mine) raw = *reinterpret_cast<const V*>(static_cast<const T*>(p.x) + row * p.ldx + c);
  float x[VB];
  if (p.residual != nullptr && mine) {
    const V more = *reinterpret_cast<const V*>(static_cast<const T*>(p.residual) + row * p.ldr + c);
    float a[VB];
    raw.get(x);
    more.get(a);
    plus(x, a);
    raw.set(x);  // as the next layer reads it
    *reinterpret_cast<V*>(static_cast<T*>(p.sum) + row * p.d + c) = raw;
  }
  raw.get(x);
  float mu[1] = {0.f}, v[1] = {0.f};
  if (!p.rms) {
#pragma unroll
    for (int j = 0; j < VB; ++j) mu[0] += x[j];
    row_sums(mu, p.threads, red[0]);
    mu[0] *= inv_d;
  }
  if (mine) {
#pragma unroll
    for (int j = 0; j < VB; ++j) v[0] = fmaf(x[j] - mu[0], x[j] - mu[0], v[0]);
  }
  row_sums(v, p.threads, red[1]);
  if (row >= p.N) return;
  const float rstd = rsqrtf(fmaf(v[0], inv_d, p.eps));
  if (t == 0 && p.stats != nullptr) p.stats[row] = make_float2(mu[0], rstd);
  if (!mine) return;
  float w[VB], b[VB];  // (asked for before the sums, their conversion holds up the row: 2.37 us for 64 x 4096, 2.24 so)
  if (p.weight != nullptr) load_gain<T, VB>(p.weight, p.gain_f32, c, w);
  if (p.bias != nullptr) load_gain<T, VB>(p.bias, p.gain_f32, c, b);
  normalise<true>(x, mu[0], rstd);
  if (p.weight != nullptr) times(x, w);
  if (p.bias != nullptr) plus(x, b);
  store<T, VB>(static_cast<T*>(p.y) + row * p.d + c, x);
}

// 16 bytes from global to shared memory, or 16 zero bytes.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }
template <typename V>
__device__ __forceinline__ V shared_vector(uint32_t a) {
  V v;
  uint32_t* w = reinterpret_cast<uint32_t*>(&v);
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(a) : "memory");
  return v;
}

// Totals over the CTA of M values a thread, for all threads. A warp halves the values that a lane carries with every exchange, so
// that 32 / M lanes end with one each; `red` holds [warps][M]: another one for each of two consecutive calls.
template <int M>
__device__ __forceinline__ void column_totals(float (&v)[M], float* red) {
  static_assert((M & (M - 1)) == 0 && M <= 16);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int owned = 0;  // which value v[0] is in the end
#pragma unroll
  for (int half = M / 2, bit = 16; half > 0; half >>= 1, bit >>= 1) {
    const bool up = (lane & bit) != 0;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float send = up ? v[i] : v[i + half];
      const float keep = up ? v[i + half] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, bit);
    }
    owned += up ? half : 0;
  }
#pragma unroll
  for (int bit = 16 / M; bit > 0; bit >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], bit);
  if ((lane & (32 / M - 1)) == 0) red[warp * M + owned] = v[0];
  __syncthreads();
  // lane l: value l % M of the warps l / M, l / M + 32 / M, ...
  float sum = 0.f;
  for (int w = lane / M; w < warps; w += 32 / M) sum += red[w * M + (lane & (M - 1))];
#pragma unroll
  for (int bit = 16; bit >= M; bit >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, bit);
#pragma unroll
  for (int i = 0; i < M; ++i) v[i] = __shfl_sync(0xffffffffu, sum, i);
}

// Means and sums of squared distances from them, of R rows: exactly as by two readings within a warp, then joined over the warps by
// sum of M2 + count (mean - total mean)^2. counts: columns of this warp and, by warp, in shared memory; red [warps][R][2].
template <int R, int KC, int VB, typename V>
__device__ __forceinline__ void row_moments(const V (&raw)[R][KC], const NormParams& p, int t, float count, const float* counts, float* red,
                                            float inv_d, float (&mu)[R], float (&m2)[R]) {
  const int width = p.threads < 32 ? p.threads : 32;
  float m[R], s[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float sum[VB];
#pragma unroll
    for (int j = 0; j < VB; ++j) sum[j] = 0.f;
#pragma unroll
    for (int k = 0; k < KC; ++k) {  // zeros behind the last column
      float a[VB];
      raw[r][k].get(a);
      plus(sum, a);
    }
    m[r] = 0.f;
#pragma unroll
    for (int j = 0; j < VB; ++j) m[r] += sum[j];
  }
  for (int o = width >> 1; o > 0; o >>= 1) {
#pragma unroll
    for (int r = 0; r < R; ++r) m[r] += __shfl_xor_sync(0xffffffffu, m[r], o);
  }
  const float inv = count > 0.f ? 1.f / count : 0.f;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    m[r] *= inv;
    float2 sum = two(0.f);
#pragma unroll
    for (int k = 0; k < KC; ++k) {
      if ((k * p.threads + t) * VB < p.d) {
        float a[VB];
        raw[r][k].get(a);
#pragma unroll
        for (int j = 0; j < VB; j += 2) {
          const float2 x = __fadd2_rn(pair(a + j), two(-m[r]));
          sum = __ffma2_rn(x, x, sum);
        }
      }
    }
    s[r] = sum.x + sum.y;
  }
  for (int o = width >> 1; o > 0; o >>= 1) {
#pragma unroll
    for (int r = 0; r < R; ++r) s[r] += __shfl_xor_sync(0xffffffffu, s[r], o);
  }
  if (p.threads <= 32) {
#pragma unroll
    for (int r = 0; r < R; ++r) mu[r] = m[r], m2[r] = s[r];
    return;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  if (lane == 0) {
#pragma unroll
    for (int r = 0; r < R; ++r) red[(warp * R + r) * 2] = m[r], red[(warp * R + r) * 2 + 1] = s[r];
  }
  __syncthreads();
  static_assert(R <= 2);
  const int row = R == 2 ? lane >> 4 : 0, w = R == 2 ? lane & 15 : lane;  // 16 warps at most
  float mw = 0.f, sw = 0.f, cw = 0.f;
  if (w < warps) mw = red[(w * R + row) * 2], sw = red[(w * R + row) * 2 + 1], cw = counts[w];
  float total = cw * mw;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  total *= inv_d;
  float all = fmaf(cw * (mw - total), mw - total, sw);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    mu[r] = __shfl_sync(0xffffffffu, total, r * 16);
    m2[r] = __shfl_sync(0xffffffffu, all, r * 16);
  }
}

// R rows at a time for each group of p.threads threads, KC vectors a thread and row, S - 1 times as many rows on their way. RMS:
// no means; BIAS: room for one. bf16 with two streams 65536 x 2048 180 us (0.88 of a copy's rate), 8192 x 4096 49; 4096 x 16384 52;
// fp32 8192 x 8192 93. What is left there is the start and the end, 6 us, and the barrier of a turn.
template <typename T, int KC, int R, int S, bool RMS, bool BIAS, bool RES>
__global__ void __launch_bounds__(512, 1) norm_fwd_ring_kernel(const NormParams p) {
  constexpr int VB = 16 / sizeof(T), C = KC * VB, STREAMS = RES ? 2 : 1;
  using V = Pack<T, VB>;
  extern __shared__ __align__(16) uint8_t ring[];  // [S][streams][R][KC][threads]
  __shared__ float red[2][16 * R * 2], counts[16];
  const int group = threadIdx.x / p.threads, t = threadIdx.x - group * p.threads;
  const int groups = blockDim.x / p.threads;
  const float inv_d = 1.f / static_cast<float>(p.d);
  const uint32_t vec = blockDim.x * 16, mine = smem_u32(ring) + threadIdx.x * 16;
  auto place = [&](int slot, int stream, int r, int k) {
    return mine + static_cast<uint32_t>(((slot * STREAMS + stream) * R + r) * KC + k) * vec;
  };
  auto fetch = [&](int slot, int64_t row0) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool live = row0 + r < p.N;
      const int64_t row = live ? row0 + r : 0;
#pragma unroll
      for (int k = 0; k < KC; ++k) {
        const int c = (k * p.threads + t) * VB;
        const bool there = live && c < p.d;
        const int at = there ? c : 0;
        copy16(place(slot, 0, r, k), static_cast<const T*>(p.x) + row * p.ldx + at, there);
        if (RES) copy16(place(slot, 1, r, k), static_cast<const T*>(p.residual) + row * p.ldr + at, there);
      }
    }
    copy_commit();
  };
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups * R;
  int64_t row0 = (static_cast<int64_t>(blockIdx.x) * groups + group) * R;
  int64_t base = static_cast<int64_t>(blockIdx.x) * groups * R;  // of the CTA: all its threads take part in every sum
#pragma unroll
  for (int i = 0; i < S - 1; ++i) fetch(i, row0 + i * step);
  float w[C], b[BIAS ? C : 1], count = 0.f;
  b[0] = 0.f;
#pragma unroll
  for (int k = 0; k < KC; ++k) {
    const int c = (k * p.threads + t) * VB;
#pragma unroll
    for (int j = k * VB; j < (k + 1) * VB; ++j) {
      w[j] = 1.f;
      if (BIAS) b[j] = 0.f;
    }
    if (c < p.d) {
      count += VB;
      if (p.weight != nullptr) load_gain<T, VB>(p.weight, p.gain_f32, c, w + k * VB);
      if (BIAS && p.bias != nullptr) load_gain<T, VB>(p.bias, p.gain_f32, c, b + k * VB);
    }
  }
  if (!RMS) {
    for (int o = (p.threads < 32 ? p.threads : 32) >> 1; o > 0; o >>= 1) count += __shfl_xor_sync(0xffffffffu, count, o);
    if ((threadIdx.x & 31) == 0) counts[threadIdx.x >> 5] = count;  // read after the first row's barrier
  }
  int slot = 0, ahead = S - 1, flip = 0;
  for (; base < p.N; base += step, row0 += step) {
    fetch(ahead, row0 + (S - 1) * step);
    ahead = ahead + 1 == S ? 0 : ahead + 1;
    copy_wait<S - 1>();
    V raw[R][KC];
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int k = 0; k < KC; ++k) {
        raw[r][k] = shared_vector<V>(place(slot, 0, r, k));
        if (RES) {
          const int c = (k * p.threads + t) * VB;
          float x[VB], y[VB];
          raw[r][k].get(x);
          shared_vector<V>(place(slot, 1, r, k)).get(y);
          plus(x, y);
          raw[r][k].set(x);  // as the next layer reads it
          if (row0 + r < p.N && c < p.d) *reinterpret_cast<V*>(static_cast<T*>(p.sum) + (row0 + r) * p.d + c) = raw[r][k];
        }
      }
    }
    slot = slot + 1 == S ? 0 : slot + 1;
    float mu[R], m2[R];
    if constexpr (RMS) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float2 sum = two(0.f);
#pragma unroll
        for (int k = 0; k < KC; ++k) {
          float x[VB];
          raw[r][k].get(x);
#pragma unroll
          for (int j = 0; j < VB; j += 2) sum = __ffma2_rn(pair(x + j), pair(x + j), sum);
        }
        mu[r] = 0.f;
        m2[r] = sum.x + sum.y;
      }
      if (p.threads <= 32) {
        for (int o = p.threads >> 1; o > 0; o >>= 1) {
#pragma unroll
          for (int r = 0; r < R; ++r) m2[r] += __shfl_xor_sync(0xffffffffu, m2[r], o);
        }
      } else {
        column_totals<R>(m2, red[flip]);
      }
    } else {
      row_moments<R, KC, VB>(raw, p, t, count, counts, red[flip], inv_d, mu, m2);
    }
    flip ^= 1;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float rstd = rsqrtf(fmaf(m2[r], inv_d, p.eps));
      const bool live = row0 + r < p.N;
      if (live && t == 0 && p.stats != nullptr) p.stats[row0 + r] = make_float2(mu[r], rstd);
      T* y = static_cast<T*>(p.y) + (row0 + r) * p.d;
#pragma unroll
      for (int k = 0; k < KC; ++k) {
        const int c = (k * p.threads + t) * VB;
        float x[VB];
        raw[r][k].get(x);
        normalise<!RMS>(x, mu[r], rstd);
#pragma unroll
        for (int j = 0; j < VB; j += 2) {
          float2 v = __fmul2_rn(pair(x + j), pair(w + k * VB + j));
          if (BIAS) v = __fadd2_rn(v, pair(b + k * VB + j));
          x[j] = v.x, x[j + 1] = v.y;
        }
        if (live && c < p.d) store<T, VB>(y + c, x);
      }
    }
  }
  copy_wait<0>();
}

// ---- Rows that are not made of 16-byte vectors (an odd width, stride or start). Their bytes still come as whole 16-byte vectors
// of memory into the ring, shifted by the row's start modulo 16, and are taken apart there: a warp has 32 C consecutive columns, a
// lane every 32nd of them (fewer lanes where a row takes part of a warp), so that a warp reads and writes consecutive elements.
// What these kernels cost is instructions: warps whose columns all exist go without a test for each (51 instructions an element
// with them). 65536 x 1001 bf16 110 us forward and 138 backward (0.35 and 0.42 of a copy's rate), fp32 128 and 156 (0.60 and
// 0.74). A vector's bytes in front of or behind the row belong to the same tensor, except in front of its first element and behind
// its last one, which are not read.
struct OddRows {
  uintptr_t base, end;  // of the tensor
  int64_t stride;       // bytes
};
template <typename T>
__device__ __forceinline__ OddRows odd_rows(const void* p, int64_t ld, const NormParams& n) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  constexpr int64_t E = sizeof(T);
  return OddRows{a, a + static_cast<uintptr_t>(((n.N - 1) * ld + n.d) * E), ld * E};
}
// The group's threads copy row `row` to dst (16-byte aligned); its first element arrives at dst + odd_shift().
__device__ __forceinline__ int odd_shift(const OddRows& x, int64_t row) { return static_cast<int>((x.base + row * x.stride) & 15); }
template <typename T>
__device__ __forceinline__ void odd_fetch(const OddRows& x, int64_t row, int d, uint32_t dst, int t, int threads) {
  const uintptr_t a = x.base + row * x.stride, last = a + static_cast<uintptr_t>(d) * sizeof(T);
  uintptr_t v = (a & ~static_cast<uintptr_t>(15)) + static_cast<uintptr_t>(t) * 16;
  for (dst += t * 16; v < last; v += static_cast<uintptr_t>(threads) * 16, dst += threads * 16) {
    if (v < x.base) {  // the tensor begins inside this vector
      for (uintptr_t e = x.base; e < v + 16 && e < x.end; e += sizeof(T)) {
        const T y = *reinterpret_cast<const T*>(e);
        const uint32_t at = dst + static_cast<uint32_t>(e - v);
        if constexpr (sizeof(T) == 2)
          asm volatile("st.shared.u16 [%0], %1;" :: "r"(at), "h"(*reinterpret_cast<const uint16_t*>(&y)) : "memory");
        else
          asm volatile("st.shared.u32 [%0], %1;" :: "r"(at), "r"(*reinterpret_cast<const uint32_t*>(&y)) : "memory");
      }
    } else {
      const uintptr_t left = x.end - v;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                   :: "r"(dst), "l"(v), "r"(left < 16 ? static_cast<int>(left) : 16) : "memory");
    }
  }
}
// A thread's C columns c0, c0 + L, ..., of which the first `n` exist, of a row: in the ring (0 behind the last one) and in memory.
// MODE kAll: all exist; kSome: L is 32; kFew: L is less.
enum : int { kAll = 0, kSome = 1, kFew = 2 };
template <int MODE>
using Mode = std::integral_constant<int, MODE>;
template <int MODE, typename T, int C>
__device__ __forceinline__ void odd_read(const uint8_t* row, int c0, int L, int n, float (&x)[C]) {
  const T* a = reinterpret_cast<const T*>(row) + c0;
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int at = MODE == kFew ? j * L : j * 32;
    T y = from_float<T>(0.f);
    if (MODE == kAll || j < n) y = a[at];
    x[j] = to_float(y);
  }
}
template <int MODE, typename T, int C>
__device__ __forceinline__ void odd_write(T* row, int c0, int L, int n, const float (&x)[C]) {
  T* a = row + c0;
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const T y = from_float<T>(x[j]);
    if (MODE == kAll || j < n) a[MODE == kFew ? j * L : j * 32] = y;
  }
}
__device__ __forceinline__ void group_barrier(int threads) {
  if (threads <= 32)
    __syncwarp();
  else
    __syncthreads();
}
// Sums over the threads of a group.
template <int M>
__device__ __forceinline__ void group_totals(float (&v)[M], int threads, float* red) {
  if (threads <= 32) {
    for (int o = threads >> 1; o > 0; o >>= 1) {
#pragma unroll
      for (int i = 0; i < M; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    }
  } else {
    column_totals<M>(v, red);
  }
}
__host__ __device__ constexpr int odd_bytes(int d, int size) { return (d * size + 15) / 16 * 16 + 16; }

template <typename T, int C, int R, int S>
__global__ void __launch_bounds__(512, 1) norm_fwd_odd_kernel(const NormParams p) {
  extern __shared__ __align__(16) uint8_t ring[];  // [groups][S][streams][R][odd_bytes]
  __shared__ float red[2][16 * R];
  const int group = threadIdx.x / p.threads, t = threadIdx.x - group * p.threads, groups = blockDim.x / p.threads;
  const int streams = p.residual != nullptr ? 2 : 1, bytes = odd_bytes(p.d, sizeof(T));
  const int L = p.threads < 32 ? p.threads : 32, c0 = (t >> 5) * 32 * C + (t & 31);
  const int n = c0 < p.d ? min(C, (p.d - c0 + L - 1) / L) : 0, mode = L < 32 ? kFew : ((t >> 5) + 1) * 32 * C <= p.d ? kAll : kSome;
  uint8_t* mine = ring + static_cast<size_t>(group) * S * streams * R * bytes;
  auto place = [&](int slot, int stream, int r) { return mine + ((slot * streams + stream) * R + r) * bytes; };
  const OddRows x0 = odd_rows<T>(p.x, p.ldx, p), x1 = odd_rows<T>(p.residual, p.ldr, p);
  const float inv_d = 1.f / static_cast<float>(p.d);
  auto fetch = [&](int slot, int64_t row0) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (row0 + r < p.N) {
        odd_fetch<T>(x0, row0 + r, p.d, smem_u32(place(slot, 0, r)), t, p.threads);
        if (streams == 2) odd_fetch<T>(x1, row0 + r, p.d, smem_u32(place(slot, 1, r)), t, p.threads);
      }
    }
    copy_commit();
  };
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups * R;
  int64_t row0 = (static_cast<int64_t>(blockIdx.x) * groups + group) * R;
  int64_t base = static_cast<int64_t>(blockIdx.x) * groups * R;  // of the CTA: all its threads take part in every barrier
#pragma unroll
  for (int i = 0; i < S - 1; ++i) fetch(i, row0 + i * step);
  float w[C], b[C];
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int c = c0 + j * L;
    w[j] = 1.f, b[j] = 0.f;
    if (p.weight != nullptr && c < p.d) load_gain<T, 1>(p.weight, p.gain_f32, c, w + j);
    if (p.bias != nullptr && c < p.d) load_gain<T, 1>(p.bias, p.gain_f32, c, b + j);
  }
  int slot = 0, ahead = S - 1, flip = 0;
  float x[R][C], mu[R], m2[R];
  auto read = [&](auto m) {
    constexpr int MODE = decltype(m)::value;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mu[r] = 0.f;
      if (row0 + r < p.N) {
        odd_read<MODE, T, C>(place(slot, 0, r) + odd_shift(x0, row0 + r), c0, L, n, x[r]);
        if (streams == 2) {
          float y[C];
          odd_read<MODE, T, C>(place(slot, 1, r) + odd_shift(x1, row0 + r), c0, L, n, y);
          plus(x[r], y);
#pragma unroll
          for (int j = 0; j < C; ++j) x[r][j] = to_float(from_float<T>(x[r][j]));  // as the next layer reads it
          odd_write<MODE, T, C>(static_cast<T*>(p.sum) + (row0 + r) * p.d, c0, L, n, x[r]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < C; ++j) x[r][j] = 0.f;
      }
    }
  };
  auto square = [&](auto m) {
    constexpr int MODE = decltype(m)::value;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float2 sum = two(0.f);
#pragma unroll
      for (int j = 0; j < C; j += 2) {
        const float2 y = __fadd2_rn(pair(x[r] + j), two(-mu[r]));
        x[r][j] = y.x, x[r][j + 1] = y.y;
        float2 z = y;
        if (MODE != kAll) {
          if (j >= n) z.x = 0.f;
          if (j + 1 >= n) z.y = 0.f;
        }
        sum = __ffma2_rn(z, z, sum);
      }
      m2[r] = sum.x + sum.y;
    }
  };
  auto write = [&](auto m) {
    constexpr int MODE = decltype(m)::value;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (row0 + r < p.N) {
        const float rstd = rsqrtf(fmaf(m2[r], inv_d, p.eps));
        if (t == 0 && p.stats != nullptr) p.stats[row0 + r] = make_float2(mu[r], rstd);
        normalise<false>(x[r], 0.f, rstd);
        times(x[r], w);
        plus(x[r], b);
        odd_write<MODE, T, C>(static_cast<T*>(p.y) + (row0 + r) * p.d, c0, L, n, x[r]);
      }
    }
  };
  auto by_mode = [&](auto f) {
    if (mode == kAll)
      f(Mode<kAll>{});
    else if (mode == kSome)
      f(Mode<kSome>{});
    else
      f(Mode<kFew>{});
  };
  for (; base < p.N; base += step, row0 += step) {
    copy_wait<S - 2>();
    group_barrier(p.threads);  // the rows are there, and those of the turn before have been read
    fetch(ahead, row0 + (S - 1) * step);
    ahead = ahead + 1 == S ? 0 : ahead + 1;
    by_mode(read);
    slot = slot + 1 == S ? 0 : slot + 1;
    if (!p.rms) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float2 sum = two(0.f);
#pragma unroll
        for (int j = 0; j < C; j += 2) sum = __fadd2_rn(pair(x[r] + j), sum);
        mu[r] = sum.x + sum.y;
      }
      group_totals<R>(mu, p.threads, red[flip]);
      flip ^= 1;
#pragma unroll
      for (int r = 0; r < R; ++r) mu[r] *= inv_d;
    }
    by_mode(square);
    group_totals<R>(m2, p.threads, red[flip]);
    flip ^= 1;
    by_mode(write);
  }
  copy_wait<0>();
}

// Rows too wide for the registers: a CTA reads its row again for each of the three steps, from L2 (2048 x 100000 bf16 with a
// residual 546 us, 0.44 of a copy's rate by what has to be read).
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

// One vector's part in dw, db and the two sums of its row. x: normalised values, g: dy.
template <bool RMS, int N>
__device__ __forceinline__ void column_step(const float (&x)[N], const float (&g)[N], const float* w, float* dw, float* db, float2& sx,
                                            float2& sg) {
#pragma unroll
  for (int j = 0; j < N; j += 2) {
    const float2 gj = pair(g + j), xj = pair(x + j), gw = __fmul2_rn(gj, pair(w + j)), d = __ffma2_rn(gj, xj, pair(dw + j));
    dw[j] = d.x, dw[j + 1] = d.y;
    sx = __ffma2_rn(gw, xj, sx);
    if (!RMS) {
      const float2 e = __fadd2_rn(gj, pair(db + j));
      db[j] = e.x, db[j + 1] = e.y;
      sg = __fadd2_rn(gw, sg);
    }
  }
}

// g <- r g w + c2 + c1 x
template <int N>
__device__ __forceinline__ void row_step(const float (&x)[N], float (&g)[N], const float* w, float r, float c1, float c2) {
#pragma unroll
  for (int j = 0; j < N; j += 2) {
    const float2 gw = __fmul2_rn(pair(g + j), pair(w + j));
    const float2 y = __ffma2_rn(pair(x + j), two(c1), __ffma2_rn(gw, two(r), two(c2)));
    g[j] = y.x, g[j + 1] = y.y;
  }
}

// The columns' sums of a CTA whose groups of threads have rows of their own; cols: [groups][d] floats of shared memory.
template <int C, int VB>
__device__ __forceinline__ void add_groups(const NormParams& p, const NormGrad& q, const float (&dw)[C], const float (&db)[C], int group,
                                           int groups, int t, float* cols, float* part, int64_t second) {
  for (int pass = 0; pass < 2; ++pass) {
    if (pass == 0 ? !q.want_dw : !q.want_db) continue;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < C / VB; ++k) {
      const int c = (k * p.threads + t) * VB;
      if (c < p.d) {
#pragma unroll
        for (int j = 0; j < VB; ++j) cols[group * p.d + c + j] = pass == 0 ? dw[k * VB + j] : db[k * VB + j];
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < p.d; c += blockDim.x) {
      float sum = 0.f;
      for (int i = 0; i < groups; ++i) sum += cols[i * p.d + c];
      part[pass * second + c] = sum;
    }
  }
}

// The gradients of such rows, one at a time.
template <typename T, int C, int S>
__global__ void __launch_bounds__(512, 1) norm_bwd_odd_kernel(const NormParams p, const NormGrad q) {
  extern __shared__ __align__(16) float shared[];  // [2][32] sums of rows, then the ring [groups][S][streams][odd_bytes], or columns' sums
  uint8_t* ring = reinterpret_cast<uint8_t*>(shared + 64);
  const int group = threadIdx.x / p.threads, t = threadIdx.x - group * p.threads, groups = blockDim.x / p.threads;
  const int streams = q.dsum != nullptr ? 3 : 2, bytes = odd_bytes(p.d, sizeof(T));
  const int L = p.threads < 32 ? p.threads : 32, c0 = (t >> 5) * 32 * C + (t & 31);
  const int n = c0 < p.d ? min(C, (p.d - c0 + L - 1) / L) : 0, mode = L < 32 ? kFew : ((t >> 5) + 1) * 32 * C <= p.d ? kAll : kSome;
  uint8_t* mine = ring + static_cast<size_t>(group) * S * streams * bytes;
  auto place = [&](int slot, int stream) { return mine + (slot * streams + stream) * bytes; };
  const OddRows x0 = odd_rows<T>(p.x, p.ldx, p), x1 = odd_rows<T>(q.dy, q.lddy, p), x2 = odd_rows<T>(q.dsum, q.ldds, p);
  const float inv_d = 1.f / static_cast<float>(p.d);
  auto fetch = [&](int slot, int64_t row) {
    if (row < p.N) {
      odd_fetch<T>(x0, row, p.d, smem_u32(place(slot, 0)), t, p.threads);
      odd_fetch<T>(x1, row, p.d, smem_u32(place(slot, 1)), t, p.threads);
      if (streams == 3) odd_fetch<T>(x2, row, p.d, smem_u32(place(slot, 2)), t, p.threads);
    }
    copy_commit();
  };
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  int64_t row = static_cast<int64_t>(blockIdx.x) * groups + group;
  int64_t base = static_cast<int64_t>(blockIdx.x) * groups;  // of the CTA: all its threads take part in every barrier
#pragma unroll
  for (int i = 0; i < S - 1; ++i) fetch(i, row + i * step);
  float dw[C], db[C], w[C];
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int c = c0 + j * L;
    dw[j] = db[j] = 0.f, w[j] = 1.f;
    if (p.weight != nullptr && c < p.d) load_gain<T, 1>(p.weight, p.gain_f32, c, w + j);
  }
  int slot = 0, ahead = S - 1, flip = 0;
  float x[C], g[C], more[C];
  auto read = [&](auto m) {
    constexpr int MODE = decltype(m)::value;
    odd_read<MODE, T, C>(place(slot, 0) + odd_shift(x0, row), c0, L, n, x);
    odd_read<MODE, T, C>(place(slot, 1) + odd_shift(x1, row), c0, L, n, g);
    if (streams == 3) odd_read<MODE, T, C>(place(slot, 2) + odd_shift(x2, row), c0, L, n, more);
  };
  auto by_mode = [&](auto f) {
    if (mode == kAll)
      f(Mode<kAll>{});
    else if (mode == kSome)
      f(Mode<kSome>{});
    else
      f(Mode<kFew>{});
  };
  for (; base < p.N; base += step, row += step) {
    const bool live = row < p.N;
    const float2 st = live ? p.stats[row] : make_float2(0.f, 0.f);
    copy_wait<S - 2>();
    group_barrier(p.threads);  // the rows are there, and those of the turn before have been read
    fetch(ahead, row + (S - 1) * step);
    ahead = ahead + 1 == S ? 0 : ahead + 1;
#pragma unroll
    for (int j = 0; j < C; ++j) x[j] = g[j] = more[j] = 0.f;
    if (live) by_mode(read);
    slot = slot + 1 == S ? 0 : slot + 1;
    normalise<true>(x, st.x, st.y);
    float2 sx = two(0.f), sg = two(0.f);
    column_step<false>(x, g, w, dw, db, sx, sg);
    if (q.dx == nullptr) continue;
    float v[2] = {sx.x + sx.y, sg.x + sg.y};
    group_totals<2>(v, p.threads, shared + flip * 32);
    flip ^= 1;
    row_step(x, g, w, st.y, -st.y * v[0] * inv_d, p.rms ? 0.f : -st.y * v[1] * inv_d);
    if (streams == 3) plus(g, more);
    T* dx = static_cast<T*>(q.dx) + row * p.d;
    if (live) by_mode([&](auto m) { odd_write<decltype(m)::value, T, C>(dx, c0, L, n, g); });
  }
  grid_dep_launch();
  copy_wait<0>();
  if (q.part == nullptr) return;
  float* part = q.part + static_cast<int64_t>(blockIdx.x) * p.d;
  const int64_t second = static_cast<int64_t>(gridDim.x) * p.d;
  if (groups > 1) {
    add_groups<C, 1>(p, q, dw, db, group, groups, t, reinterpret_cast<float*>(ring), part, second);  // begins with a barrier; threads <= 32
    return;
  }
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int c = c0 + j * L;
    if (c < p.d) {
      if (q.want_dw) part[c] = dw[j];
      if (q.want_db) part[second + c] = db[j];
    }
  }
}

// The gradients for rows of 16-byte vectors: as above, R rows of a group at a time and S - 1 times as many on their way. bf16 with
// dsum 65536 x 2048 165 us (0.96 of a copy's rate), 8192 x 4096 50; fp32 65536 x 512 79.
template <typename T, int KC, int R, int S, bool RMS, bool DSUM>
__global__ void __launch_bounds__(512, 1) norm_bwd_ring_kernel(const NormParams p, const NormGrad q) {
  constexpr int VB = 16 / sizeof(T), C = KC * VB, STREAMS = DSUM ? 3 : 2;
  using V = Pack<T, VB>;
  // [2][32][2 R] sums of rows, then the ring [S][streams][R][KC][threads], or columns' sums
  extern __shared__ __align__(16) float shared[];
  uint8_t* ring = reinterpret_cast<uint8_t*>(shared + 128 * R);
  const int group = threadIdx.x / p.threads, t = threadIdx.x - group * p.threads;
  const int groups = blockDim.x / p.threads;
  const float inv_d = 1.f / static_cast<float>(p.d);
  const uint32_t vec = blockDim.x * 16, mine = smem_u32(ring) + threadIdx.x * 16;
  auto place = [&](int slot, int stream, int r, int k) {
    return mine + static_cast<uint32_t>(((slot * STREAMS + stream) * R + r) * KC + k) * vec;
  };
  float dw[C], db[C], w[C];
#pragma unroll
  for (int j = 0; j < C; ++j) dw[j] = db[j] = 0.f, w[j] = 1.f;
  if (p.weight != nullptr) {
#pragma unroll
    for (int k = 0; k < KC; ++k) {
      const int c = (k * p.threads + t) * VB;
      if (c < p.d) load_gain<T, VB>(p.weight, p.gain_f32, c, w + k * VB);
    }
  }
  auto fetch = [&](int slot, int64_t row0) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool live = row0 + r < p.N;
      const int64_t row = live ? row0 + r : 0;
#pragma unroll
      for (int k = 0; k < KC; ++k) {
        const int c = (k * p.threads + t) * VB;
        const bool there = live && c < p.d;
        const int at = there ? c : 0;
        copy16(place(slot, 0, r, k), static_cast<const T*>(p.x) + row * p.ldx + at, there);
        copy16(place(slot, 1, r, k), static_cast<const T*>(q.dy) + row * q.lddy + at, there);
        if (DSUM) copy16(place(slot, 2, r, k), static_cast<const T*>(q.dsum) + row * q.ldds + at, there);
      }
    }
    copy_commit();
  };
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups * R;
  int64_t row0 = (static_cast<int64_t>(blockIdx.x) * groups + group) * R;
  int64_t base = static_cast<int64_t>(blockIdx.x) * groups * R;  // of the CTA: all its threads take part in every sum
#pragma unroll
  for (int i = 0; i < S - 1; ++i) fetch(i, row0 + i * step);
  float2 st[R];
#pragma unroll
  for (int r = 0; r < R; ++r) st[r] = row0 + r < p.N ? p.stats[row0 + r] : make_float2(0.f, 0.f);
  int slot = 0, ahead = S - 1, flip = 0;
  for (; base < p.N; base += step, row0 += step) {
    fetch(ahead, row0 + (S - 1) * step);
    ahead = ahead + 1 == S ? 0 : ahead + 1;
    float2 now[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      now[r] = st[r];
      st[r] = row0 + step + r < p.N ? p.stats[row0 + step + r] : make_float2(0.f, 0.f);
    }
    copy_wait<S - 1>();
    float v[2 * R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float2 sg = two(0.f), sx = two(0.f);
#pragma unroll
      for (int k = 0; k < KC; ++k) {
        float x[VB], g[VB];
        shared_vector<V>(place(slot, 0, r, k)).get(x);
        shared_vector<V>(place(slot, 1, r, k)).get(g);  // zeros behind the last column
        normalise<!RMS>(x, now[r].x, now[r].y);
        column_step<RMS>(x, g, w + k * VB, dw + k * VB, db + k * VB, sx, sg);
      }
      v[2 * r] = sx.x + sx.y;
      v[2 * r + 1] = sg.x + sg.y;
    }
    if (q.dx != nullptr) {
      if (p.threads <= 32) {
        for (int o = p.threads >> 1; o > 0; o >>= 1) {
#pragma unroll
          for (int i = 0; i < 2 * R; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
        }
      } else {
        column_totals<2 * R>(v, shared + flip * 64 * R);
        flip ^= 1;
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float c1 = -now[r].y * v[2 * r] * inv_d, c2 = RMS || p.rms ? 0.f : -now[r].y * v[2 * r + 1] * inv_d;
        T* dx = static_cast<T*>(q.dx) + (row0 + r) * p.d;
#pragma unroll
        for (int k = 0; k < KC; ++k) {
          const int c = (k * p.threads + t) * VB;
          float x[VB], g[VB];
          shared_vector<V>(place(slot, 0, r, k)).get(x);
          shared_vector<V>(place(slot, 1, r, k)).get(g);
          normalise<!RMS>(x, now[r].x, now[r].y);
          row_step(x, g, w + k * VB, now[r].y, c1, c2);
          if (DSUM) {
            float more[VB];
            shared_vector<V>(place(slot, 2, r, k)).get(more);
            plus(g, more);
          }
          if (row0 + r < p.N && c < p.d) store<T, VB>(dx + c, g);
        }
      }
    }
    slot = slot + 1 == S ? 0 : slot + 1;
  }
  grid_dep_launch();
  copy_wait<0>();
  if (q.part == nullptr) return;
  float* part = q.part + static_cast<int64_t>(blockIdx.x) * p.d;
  const int64_t second = static_cast<int64_t>(gridDim.x) * p.d;
  if (groups == 1) {
#pragma unroll
    for (int k = 0; k < KC; ++k) {
      const int c = (k * p.threads + t) * VB;
      if (c < p.d) {
#pragma unroll
        for (int j = 0; j < VB; j += 4) {
          if (q.want_dw) store<float, 4>(part + c + j, dw + k * VB + j);
          if (q.want_db) store<float, 4>(part + second + c + j, db + k * VB + j);
        }
      }
    }
  } else {
    add_groups<C, VB>(p, q, dw, db, group, groups, t, reinterpret_cast<float*>(ring), part, second);  // begins with a barrier
  }
}

// The same for rows that a cluster shares, q.cta_cols columns a CTA, one row at a time. Order of a turn: the sums of row i; the wait
// for those of row i - 1, which the CTAs have sent one another meanwhile; the sending of row i's; dx of row i - 1. The sums
// arrive with st.async, counted on a barrier of the CTA that receives them (a cluster barrier a turn took twice as long). Three
// places for them are enough: a CTA sends row i + 3's only after it has this CTA's of row i + 2, sent after all here were done with
// row i's. bf16 16384 x 5120 90 us (0.82 of a copy's rate), 4096 x 16384 87; fp32 8192 x 8192 141, 8192 x 16384 496 (0.48: an exchange
// a row, 38 rows at a time).
__device__ __forceinline__ void send_pair(uint32_t to, float a, float b, uint32_t bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];"
               :: "r"(to), "r"(__float_as_uint(a)), "r"(__float_as_uint(b)), "r"(bar) : "memory");
}
template <typename T, int KC, int S, bool RMS, bool DSUM>
__global__ void __launch_bounds__(512, 1) norm_bwd_cluster_kernel(const NormParams p, const NormGrad q) {
  constexpr int VB = 16 / sizeof(T), C = KC * VB, STREAMS = DSUM ? 3 : 2;
  using V = Pack<T, VB>;
  // [2][16 warps][2] sums, [3][8 CTAs][2] exchanged ones, then the ring [S][streams][KC][threads]
  extern __shared__ __align__(16) float shared[];
  float* across = shared + 64;
  __shared__ uint64_t arrived[3];
  __shared__ int given_up;
  uint8_t* ring = reinterpret_cast<uint8_t*>(shared + 128);
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, warps = blockDim.x >> 5;
  const uint32_t rank = cluster_ctarank(), ctas = gridDim.x;
  const int first = static_cast<int>(rank) * q.cta_cols, end = min(p.d, first + q.cta_cols);
  const float inv_d = 1.f / static_cast<float>(p.d);
  const uint32_t vec = blockDim.x * 16, mine = smem_u32(ring) + t * 16;
  auto place = [&](int slot, int stream, int k) { return mine + static_cast<uint32_t>((slot * STREAMS + stream) * KC + k) * vec; };
  float dw[C], db[C], w[C];
#pragma unroll
  for (int j = 0; j < C; ++j) dw[j] = db[j] = 0.f, w[j] = 1.f;
  if (p.weight != nullptr) {
#pragma unroll
    for (int k = 0; k < KC; ++k) {
      const int c = first + (k * blockDim.x + t) * VB;
      if (c < end) load_gain<T, VB>(p.weight, p.gain_f32, c, w + k * VB);
    }
  }
  auto fetch = [&](int slot, int64_t i) {
    const bool live = i < p.N;
    const int64_t row = live ? i : 0;
#pragma unroll
    for (int k = 0; k < KC; ++k) {
      const int c = first + (k * static_cast<int>(blockDim.x) + t) * VB;
      const bool there = live && c < end;
      const int at = there ? c : 0;
      copy16(place(slot, 0, k), static_cast<const T*>(p.x) + row * p.ldx + at, there);
      copy16(place(slot, 1, k), static_cast<const T*>(q.dy) + row * q.lddy + at, there);
      if (DSUM) copy16(place(slot, 2, k), static_cast<const T*>(q.dsum) + row * q.ldds + at, there);
    }
    copy_commit();
  };
  const int64_t step = gridDim.y;
  int64_t row = blockIdx.y;
#pragma unroll
  for (int i = 0; i < S - 1; ++i) fetch(i, row + i * step);
  if (t == 0) {
    for (int j = 0; j < 3; ++j) mbar_init(arrived + j, 1);
    given_up = 0;
    fence_mbar_init();
  }
  cluster_sync_all();  // every CTA's barriers are there before it is written to
  float2 now = row < p.N ? p.stats[row] : make_float2(0.f, 0.f), before = now;
  int slot = 0, last = 0, i = 0;
  auto finish = [&](int64_t r, float2 st, int from, int turn) {  // dx of row r, whose sums were exchanged in this turn
    float a = 0.f, b = 0.f;
    for (uint32_t c = 0; c < ctas; ++c) {
      a += across[(turn % 3) * 16 + c * 2];
      b += across[(turn % 3) * 16 + c * 2 + 1];
    }
    const float c1 = -st.y * a * inv_d, c2 = RMS || p.rms ? 0.f : -st.y * b * inv_d;
    T* dx = static_cast<T*>(q.dx) + r * p.d;
#pragma unroll
    for (int k = 0; k < KC; ++k) {
      const int c = first + (k * static_cast<int>(blockDim.x) + t) * VB;
      float x[VB], g[VB];
      shared_vector<V>(place(from, 0, k)).get(x);
      shared_vector<V>(place(from, 1, k)).get(g);
      normalise<!RMS>(x, st.x, st.y);
      row_step(x, g, w + k * VB, st.y, c1, c2);
      if (DSUM) {
        float more[VB];
        shared_vector<V>(place(from, 2, k)).get(more);
        plus(g, more);
      }
      if (c < end) store<T, VB>(dx + c, g);
    }
  };
  auto take = [&](int turn) {  // the sums of that turn, which other CTAs release at cluster scope, or a time-out that ends the kernel
    if (!wait_bounded<true>(arrived + turn % 3, static_cast<uint32_t>(turn / 3) & 1u, &given_up, q.ctl, 61)) given_up = 1;
  };
  for (; row < p.N; row += step, ++i) {
    copy_wait<S - 2>();
    const float2 next = row + step < p.N ? p.stats[row + step] : make_float2(0.f, 0.f);
    float2 sg = two(0.f), sx = two(0.f);
#pragma unroll
    for (int k = 0; k < KC; ++k) {
      float x[VB], g[VB];
      shared_vector<V>(place(slot, 0, k)).get(x);
      shared_vector<V>(place(slot, 1, k)).get(g);
      normalise<!RMS>(x, now.x, now.y);
      column_step<RMS>(x, g, w + k * VB, dw + k * VB, db + k * VB, sx, sg);
    }
    if (q.dx != nullptr) {
      float a = sx.x + sx.y, b = sg.x + sg.y;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
      }
      float* red = shared + (i & 1) * 32;
      if (lane == 0) red[warp * 2] = a, red[warp * 2 + 1] = b;
      if (t == 0 && i > 0) take(i - 1);
      __syncthreads();
      if (given_up) break;
      if (warp == 0) {  // lane: sum lane / 16 of warp lane % 16
        float sum = (lane & 15) < warps ? red[(lane & 15) * 2 + (lane >> 4)] : 0.f;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float other = __shfl_xor_sync(0xffffffffu, sum, 16);
        if (lane == 0) mbar_arrive_expect_tx(arrived + i % 3, ctas * 8);
        if (lane < static_cast<int>(ctas))  // every lane tells one CTA
          send_pair(mapa_shared(smem_u32(across + (i % 3) * 16 + rank * 2), lane), sum, other,
                    mapa_shared(smem_u32(arrived + i % 3), lane));
      }
      if (i > 0) finish(row - step, before, last, i - 1);
    }
    before = now;
    now = next;
    last = slot;
    slot = slot + 1 == S ? 0 : slot + 1;
    // the place of the row before, or with the first row the one that is still free
    fetch((i + S - 1) % S, row + (S - 1) * step);
  }
  if (q.dx != nullptr && i > 0) {
    if (t == 0 && !given_up) take(i - 1);
    __syncthreads();
    if (!given_up) finish(row - step, before, last, i - 1);
  }
  grid_dep_launch();
  copy_wait<0>();
  if (q.part != nullptr) {
    float* part = q.part + static_cast<int64_t>(blockIdx.y) * p.d;
    const int64_t second = static_cast<int64_t>(gridDim.y) * p.d;
#pragma unroll
    for (int k = 0; k < KC; ++k) {
      const int c = first + (k * static_cast<int>(blockDim.x) + t) * VB;
      if (c < end) {
#pragma unroll
        for (int j = 0; j < VB; j += 4) {
          if (q.want_dw) store<float, 4>(part + c + j, dw + k * VB + j);
          if (q.want_db) store<float, 4>(part + second + c + j, db + k * VB + j);
        }
      }
    }
  }
  cluster_sync_all();  // no CTA leaves while another one may still send to it
}

// dx of rows too wide for the registers (2048 x 100000 bf16 with dsum 509 us, 0.47 of a copy's rate; dw and db as much as 314 more).
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

// The columns' sums of rows blockIdx.y, blockIdx.y + gridDim.y, ... for 256 columns a CTA, read once more.
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

constexpr int kBwdCols = 8;     // columns of a thread in the backward
constexpr int kCtaCols = 4096;  // columns of a CTA of 512 threads; wider rows go to a cluster, 8192 columns (fp32 4096) a CTA
constexpr int kGridSms = 152;   // the workspace's size may not depend on the device
constexpr int kSmemPerSm = 225 << 10;

// Lets a kernel have more than 48 KiB of dynamic shared memory, once on each device.
template <auto KERNEL>
cudaError_t allow_smem() {
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (done.load(std::memory_order_relaxed) >> dev & 1)) return e;
  e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemPerSm);
  if (e == cudaSuccess) done.fetch_or(1ull << dev, std::memory_order_relaxed);
  return e;
}

unsigned blocks_for(int64_t blocks, int64_t most) { return static_cast<unsigned>(blocks < most ? blocks : most); }

template <typename T, int VB>
cudaError_t fwd(NormParams p, cudaStream_t stream) {
  p.threads = round_threads(cdiv64(p.d, VB));
  const int cta = p.threads > 32 ? p.threads : 128;
  const int64_t blocks = cdiv64(p.N, cta / p.threads);
  return launch(norm_fwd_kernel<T, VB>, dim3(static_cast<unsigned>(blocks)), cta, 0, stream, false, p);
}

template <typename T, int KC, int R, int S, bool RMS, bool BIAS, bool RES>
cudaError_t fwd_ring(NormParams p, int sms, cudaStream_t stream) {
  p.threads = round_threads(cdiv64(p.d, 16 / sizeof(T) * KC));
  const int cta = p.threads > 32 ? p.threads : 128, smem = S * (RES ? 2 : 1) * R * KC * 16 * cta;
  const cudaError_t e = allow_smem<norm_fwd_ring_kernel<T, KC, R, S, RMS, BIAS, RES>>();
  if (e != cudaSuccess) return e;
  const int by_smem = kSmemPerSm / (smem + 1536), by_threads = (KC * 16 / sizeof(T) > 8 ? 512 : 768) / cta;
  const int64_t most = static_cast<int64_t>(sms) * (by_smem < by_threads ? by_smem : by_threads);
  const int64_t blocks = cdiv64(p.N, static_cast<int64_t>(cta / p.threads) * R);
  return launch(norm_fwd_ring_kernel<T, KC, R, S, RMS, BIAS, RES>, dim3(blocks_for(blocks, most)), cta, smem, stream, false, p);
}

template <typename T, int C, int R, int S>
cudaError_t fwd_odd(NormParams p, int sms, cudaStream_t stream) {
  p.threads = round_threads(cdiv64(p.d, C));
  const int cta = p.threads > 32 ? p.threads : 128, groups = cta / p.threads;
  const int smem = groups * S * (p.residual ? 2 : 1) * R * odd_bytes(p.d, sizeof(T));
  const cudaError_t e = allow_smem<norm_fwd_odd_kernel<T, C, R, S>>();
  if (e != cudaSuccess) return e;
  const int by_smem = kSmemPerSm / (smem + 1536), by_threads = 512 / cta;
  const int64_t most = static_cast<int64_t>(sms) * (by_smem < by_threads ? by_smem : by_threads);
  const int64_t blocks = cdiv64(p.N, static_cast<int64_t>(groups) * R);
  return launch(norm_fwd_odd_kernel<T, C, R, S>, dim3(blocks_for(blocks, most)), cta, smem, stream, false, p);
}

// Eight columns a thread, two rows at a time; of rows of more than 4096 columns 16 or 32 columns, one row at a time.
template <typename T, bool RMS, bool BIAS, bool RES>
cudaError_t fwd_rings(const NormParams& p, int sms, cudaStream_t stream) {
  constexpr int K8 = 8 * sizeof(T) / 16;
  if (p.d <= 512 * 8) return fwd_ring<T, K8, sizeof(T) == 2 ? 2 : 1, 4, RMS, BIAS, RES>(p, sms, stream);
  if (p.d <= 512 * 16) return fwd_ring<T, 2 * K8, 1, RES && sizeof(T) == 4 ? 3 : 4, RMS, BIAS, RES>(p, sms, stream);
  return fwd_ring<T, 4 * K8, 1, sizeof(T) == 4 || RES ? 3 : 4, RMS, BIAS, RES>(p, sms, stream);
}

template <typename T, int VB>
cudaError_t fwd_cols(const NormParams& p, int sms, cudaStream_t stream) {
  if constexpr (VB == 1) {
    if (p.d <= 1024 && p.N <= 2 * sms) return fwd<T, 1>(p, stream);
    if (p.d <= 512 * 8) return fwd_odd<T, 8, sizeof(T) == 2 ? 2 : 1, 4>(p, sms, stream);
    if (p.d <= 512 * 16) return fwd_odd<T, 16, 1, 3>(p, sms, stream);
    if (p.d <= 512 * 32 && (sizeof(T) == 2 || p.residual == nullptr)) return fwd_odd<T, 32, 1, 3>(p, sms, stream);
  } else {
    if (p.d <= 1024 * VB && p.N <= 4 * sms) return fwd<T, VB>(p, stream);
    if (p.d <= (sizeof(T) == 4 && p.residual ? 512 * 16 : 512 * 32)) {  // what the ring has room for
      const bool res = p.residual != nullptr;
      if (!p.rms) return res ? fwd_rings<T, false, true, true>(p, sms, stream) : fwd_rings<T, false, true, false>(p, sms, stream);
      if (!p.bias) return res ? fwd_rings<T, true, false, true>(p, sms, stream) : fwd_rings<T, true, false, false>(p, sms, stream);
      return res ? fwd_rings<T, true, true, true>(p, sms, stream) : fwd_rings<T, true, true, false>(p, sms, stream);
    }
  }
  return launch(norm_fwd_wide_kernel<T, VB>, dim3(blocks_for(p.N, 2 * static_cast<int64_t>(sms))), 1024, 0, stream, false, p);
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

template <typename T, bool RMS, bool DSUM>
cudaError_t bwd_ring(NormParams p, const NormGrad& q, int* parts, cudaStream_t stream) {
  constexpr int KC = kBwdCols * sizeof(T) / 16, R = sizeof(T) == 2 ? 2 : 1, S = 4;
  p.threads = round_threads(cdiv64(p.d, kBwdCols));
  const int cta = p.threads > 32 ? p.threads : 128, groups = cta / p.threads;
  const cudaError_t e = allow_smem<norm_bwd_ring_kernel<T, KC, R, S, RMS, DSUM>>();
  if (e != cudaSuccess) return e;
  size_t smem = static_cast<size_t>(S) * (DSUM ? 3 : 2) * R * KC * 16 * cta;
  if (groups > 1 && static_cast<size_t>(groups) * p.d * sizeof(float) > smem) smem = static_cast<size_t>(groups) * p.d * sizeof(float);
  *parts = static_cast<int>(blocks_for(cdiv64(p.N, static_cast<int64_t>(groups) * R), *parts));
  return launch(norm_bwd_ring_kernel<T, KC, R, S, RMS, DSUM>, dim3(*parts), cta, 128 * R * sizeof(float) + smem, stream, false, p, q);
}

template <typename T, bool RMS, bool DSUM>
cudaError_t bwd_cluster(NormParams p, NormGrad q, int* parts, cudaStream_t stream) {
  constexpr int KC = 2, S = 4, cols = KC * 16 / sizeof(T);
  const int threads = 512;
  const int ctas = static_cast<int>(cdiv64(p.d, threads * cols));
  const int cta = static_cast<int>(cdiv64(cdiv64(p.d, ctas), 32 * cols) * 32);
  q.cta_cols = cta * cols;
  const cudaError_t e = allow_smem<norm_bwd_cluster_kernel<T, KC, S, RMS, DSUM>>();
  if (e != cudaSuccess) return e;
  const int smem = 512 + S * (DSUM ? 3 : 2) * KC * 16 * cta, by_smem = kSmemPerSm / (smem + 1280), by_threads = (RMS ? 672 : 576) / cta;
  const int64_t most = static_cast<int64_t>(kGridSms / ctas) * (by_smem < by_threads ? by_smem : by_threads);
  *parts = static_cast<int>(blocks_for(p.N, *parts < most ? *parts : most));
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas, *parts);
  cfg.blockDim = dim3(cta);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = ctas;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm_bwd_cluster_kernel<T, KC, S, RMS, DSUM>, p, q);
}

template <typename T, bool RMS, bool DSUM>
cudaError_t bwd_vectors(const NormParams& p, const NormGrad& q, int* parts, cudaStream_t stream) {
  return p.d <= kCtaCols ? bwd_ring<T, RMS, DSUM>(p, q, parts, stream) : bwd_cluster<T, RMS, DSUM>(p, q, parts, stream);
}

template <typename T, int C, int S>
cudaError_t bwd_odd(NormParams p, const NormGrad& q, int* parts, cudaStream_t stream) {
  p.threads = round_threads(cdiv64(p.d, C));
  const int cta = p.threads > 32 ? p.threads : 128, groups = cta / p.threads;
  const cudaError_t e = allow_smem<norm_bwd_odd_kernel<T, C, S>>();
  if (e != cudaSuccess) return e;
  size_t smem = static_cast<size_t>(groups) * S * (q.dsum ? 3 : 2) * odd_bytes(p.d, sizeof(T));
  if (groups > 1 && static_cast<size_t>(groups) * p.d * sizeof(float) > smem) smem = static_cast<size_t>(groups) * p.d * sizeof(float);
  *parts = static_cast<int>(blocks_for(cdiv64(p.N, groups), *parts));
  return launch(norm_bwd_odd_kernel<T, C, S>, dim3(*parts), cta, 64 * sizeof(float) + smem, stream, false, p, q);
}

// *parts: rows of q.part that there may be, and how many were written.
template <typename T, int VB>
cudaError_t bwd_cols(NormParams p, const NormGrad& q, int* parts, int sms, cudaStream_t stream) {
  if constexpr (VB > 1) {
    if (p.d <= (sizeof(T) == 2 ? kNormFusedCols : kNormFusedCols / 2)) {
      if (p.rms && !q.want_db)
        return q.dsum ? bwd_vectors<T, true, true>(p, q, parts, stream) : bwd_vectors<T, true, false>(p, q, parts, stream);
      return q.dsum ? bwd_vectors<T, false, true>(p, q, parts, stream) : bwd_vectors<T, false, false>(p, q, parts, stream);
    }
  } else {
    if (p.d <= kCtaCols) return bwd_odd<T, 8, 4>(p, q, parts, stream);
    if (p.d <= 2 * kCtaCols) return bwd_odd<T, 16, sizeof(T) == 2 ? 4 : 2>(p, q, parts, stream);
  }
  cudaError_t e = cudaSuccess;
  if (q.dx != nullptr)
    e = launch(norm_bwd_wide_kernel<T, VB>, dim3(blocks_for(p.N, 2 * static_cast<int64_t>(sms))), 1024, 0, stream, false, p, q);
  *parts = static_cast<int>(blocks_for(p.N, *parts));
  if (e == cudaSuccess && q.part != nullptr)
    e = launch(norm_columns_kernel<T>, dim3(static_cast<unsigned>(cdiv64(p.d, 256)), *parts), 256, 0, stream, false, p, q);
  return e;
}

template <typename T>
cudaError_t bwd_type(const NormParams& p, const NormGrad& q, int parts, int sms, cudaStream_t stream) {
  constexpr int VB = 16 / sizeof(T);
  const int64_t e = sizeof(T), ge = p.gain_f32 ? 4 : e;
  const bool vec = p.d % VB == 0 && vectors(p.x, p.ldx, p.N, e, 16) && vectors(q.dy, q.lddy, p.N, e, 16) &&
                   vectors(q.dsum, q.ldds, p.N, e, 16) && vectors(q.dx, p.d, p.N, e, 16) && vectors(p.weight, 0, 1, ge, 16);
  cudaError_t err = vec ? bwd_cols<T, VB>(p, q, &parts, sms, stream) : bwd_cols<T, 1>(p, q, &parts, sms, stream);
  if (err != cudaSuccess || q.part == nullptr) return err;
  const dim3 grid(static_cast<unsigned>(cdiv64(p.d, 32)), q.want_dw && q.want_db ? 2 : 1);
  void* dw = q.want_dw ? q.dw : nullptr;
  if (p.gain_f32) return launch(norm_join_kernel<float>, grid, 32 * kSlices, 0, stream, true, q.part, parts, p.d, dw, q.db);
  return launch(norm_join_kernel<T>, grid, 32 * kSlices, 0, stream, true, q.part, parts, p.d, dw, q.db);
}

}  // namespace

int norm_parts(int64_t N, int d) {
  int64_t most;
  // Clusters (of fp32 rows of one or two CTAs, two an SM), or stretches of rows that fill the SMs with 256 columns each.
  if (d > kCtaCols) {
    const int64_t clusters = d > kNormFusedCols ? 0 : 2 * kGridSms / cdiv64(d, 2 * kCtaCols);
    const int64_t stretches = cdiv64(8 * kGridSms, cdiv64(d, 256));
    most = clusters > stretches ? clusters : stretches;
  } else {
    most = kGridSms * (512 / (d > 256 ? round_threads(cdiv64(d, kBwdCols)) : 128));  // 512 threads an SM
  }
  return static_cast<int>(N < most ? N : most);
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
