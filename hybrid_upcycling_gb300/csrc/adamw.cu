// AdamW over a list of tensors in one launch, and the global gradient norm that clips it.
// Both are bound by HBM: the norm reads each gradient once; the step reads the gradient and reads
// and writes the parameter, its fp32 master and both moments once.
//
// The list of tensors travels in the kernel's parameters (no device-side table to build or keep).
// A warp takes 256 consecutive elements of a tensor, eight per lane: the unit that shares one
// power of two when the moments are kept in 8 bits, so the block's largest magnitude is one
// warp reduction and each state byte is read and written by the lane that updates it.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "hylo_ops_internal.h"
#include "sm103_ptx.cuh"

namespace hylo {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBlock = 256;                // elements per warp step and per 8-bit scale
constexpr int kChunk = kWarps * kBlock;    // elements per thread block

struct AdamTensor {
  void* p;
  const void* g;
  float* master;
  void* m;
  void* v;
  int8_t* me;
  int8_t* ve;
  int64_t n;
  uint64_t pos;     // position of element 0 in the list (random bits)
  uint32_t chunk0;  // first thread block
  uint32_t vec;     // every array is aligned for vector access
  float decay;      // 1 - lr weight_decay
  float step;       // lr / (1 - beta1^step)
};

template <int CAP>
struct AdamTable {
  AdamTensor t[CAP];
  int count;
};
constexpr int kSmallTable = 32;
constexpr int kLargeTable = 320;
static_assert(sizeof(AdamTable<kLargeTable>) + sizeof(AdamWHyper) <= 32764, "kernel parameter space");

__device__ __forceinline__ uint32_t mix32(uint32_t x) {  // the finaliser of MurmurHash3
  x = (x ^ (x >> 16)) * 0x85EBCA6Bu;
  x = (x ^ (x >> 13)) * 0xC2B2AE35u;
  return x ^ (x >> 16);
}

__device__ __forceinline__ float sqrt_approx(float x) {
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ void unpack_bf16x8(uint4 v, float* z) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    z[2 * i] = __uint_as_float(w[i] << 16);
    z[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// Eight elements from `i` on (`left` of them exist), widened to fp32; missing ones are 0.
__device__ __forceinline__ void load8(const float* p, int64_t i, int left, bool vec, float* z) {
  if (vec && left >= 8) {
    const float4 a = *reinterpret_cast<const float4*>(p + i), b = *reinterpret_cast<const float4*>(p + i + 4);
    z[0] = a.x, z[1] = a.y, z[2] = a.z, z[3] = a.w, z[4] = b.x, z[5] = b.y, z[6] = b.z, z[7] = b.w;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) z[j] = j < left ? p[i + j] : 0.f;
  }
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, int64_t i, int left, bool vec, float* z) {
  if (vec && left >= 8) {
    unpack_bf16x8(*reinterpret_cast<const uint4*>(p + i), z);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) z[j] = j < left ? __bfloat162float(p[i + j]) : 0.f;
  }
}
__device__ __forceinline__ void store8(float* p, int64_t i, int left, bool vec, const float* z) {
  if (vec && left >= 8) {
    *reinterpret_cast<float4*>(p + i) = make_float4(z[0], z[1], z[2], z[3]);
    *reinterpret_cast<float4*>(p + i + 4) = make_float4(z[4], z[5], z[6], z[7]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < left) p[i + j] = z[j];
  }
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, int64_t i, int left, bool vec, const float* z) {
  if (vec && left >= 8) {
    *reinterpret_cast<uint4*>(p + i) =
        make_uint4(pack_bf16x2(z[0], z[1]), pack_bf16x2(z[2], z[3]), pack_bf16x2(z[4], z[5]), pack_bf16x2(z[6], z[7]));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < left) p[i + j] = __float2bfloat16_rn(z[j]);
  }
}

// ---- 8-bit states: e4m3 codes with one power of two per block
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127

__device__ __forceinline__ float2 decode2(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ uint32_t encode2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void load_codes(const uint8_t* p, int64_t i, int left, bool vec, float scale, float* z) {
  uint2 w = make_uint2(0u, 0u);
  if (vec && left >= 8) {
    w = *reinterpret_cast<const uint2*>(p + i);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t b = j < left ? p[i + j] : 0u;
      if (j < 4)
        w.x |= b << (8 * j);
      else
        w.y |= b << (8 * (j - 4));
    }
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint32_t two = ((q < 2 ? w.x : w.y) >> (16 * (q & 1))) & 0xffffu;
    const float2 f = decode2(two);
    z[2 * q] = f.x * scale;
    z[2 * q + 1] = f.y * scale;
  }
}

// The block's exponent: its largest magnitude (bit pattern `top`) lies in [128, 256) 2^e.
__device__ __forceinline__ int block_exponent(uint32_t top) {
  return min(120, max(-120, static_cast<int>(top >> 23) - 127 - 7));
}

// |x| 2^-e rounded to an e4m3 value: the bits below the three of the mantissa are cut off after
// adding `random` (20 bits) to them. Magnitudes under 2^-6 (codes of a fixed step 2^-9) take the
// same steps once 2^-6 is added.
__device__ __forceinline__ float round_code(float x, float inv_scale, uint32_t random, bool keep) {
  const float a = fabsf(x) * inv_scale;
  const float low = a < 0.015625f ? 0.015625f : 0.f;
  float q = __uint_as_float((__float_as_uint(a + low) + random) & 0xfff00000u) - low;
  if (keep && a > 0.f) q = fmaxf(q, 0.001953125f);
  return copysignf(q, x);
}

__device__ __forceinline__ void store_codes(uint8_t* p, int64_t i, int left, bool vec, const float* q) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) w[k] = encode2(q[2 * k], q[2 * k + 1]);
  if (vec && left >= 8) {
    *reinterpret_cast<uint2*>(p + i) = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < left) p[i + j] = static_cast<uint8_t>(w[j >> 1] >> (8 * (j & 1)));
  }
}

// The entry whose blocks include block `b` (entries ascend by chunk0).
template <typename Table>
__device__ __forceinline__ int find_entry(const Table& tab, uint32_t b) {
  int lo = 0, hi = tab.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tab.t[mid].chunk0 <= b)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// P, G: types of parameter and gradient; MASTER: the step is taken on fp32 masters; BITS8: 8-bit states.
template <typename P, typename G, bool MASTER, bool BITS8, int CAP>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ AdamTable<CAP> tab, const AdamWHyper h) {
  constexpr bool kRandomParam = sizeof(P) == 2 && !MASTER;
  float gs = h.grad_scale;
  if (h.norm != nullptr) {
    const float norm = h.norm[0];
    if (!isfinite(norm)) return;
    gs *= fminf(1.f, h.max_norm / (norm * fabsf(h.grad_scale) + 1e-6f));
  }
  const AdamTensor& t = tab.t[find_entry(tab, blockIdx.x)];
  const int lane = threadIdx.x & 31;
  const int64_t b0 = (static_cast<int64_t>(blockIdx.x - t.chunk0) * kWarps + (threadIdx.x >> 5)) * kBlock;
  if (b0 >= t.n) return;
  const int64_t i = b0 + lane * 8;
  const int left = static_cast<int>(max(int64_t(0), min(int64_t(8), t.n - i)));
  const bool vec = t.vec != 0;
  float w[8], g[8], m[8], v[8];
  load8(static_cast<const G*>(t.g), i, left, vec, g);
  if (MASTER)
    load8(t.master, i, left, vec, w);
  else
    load8(static_cast<const P*>(t.p), i, left, vec, w);
  if (BITS8) {
    load_codes(static_cast<const uint8_t*>(t.m), i, left, vec, pow2(t.me[b0 / kBlock]), m);
    load_codes(static_cast<const uint8_t*>(t.v), i, left, vec, pow2(t.ve[b0 / kBlock]), v);
  } else {
    load8(static_cast<const float*>(t.m), i, left, vec, m);
    load8(static_cast<const float*>(t.v), i, left, vec, v);
  }
  float mtop = 0.f, rtop = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float gj = g[j] * gs;
    m[j] = fmaf(h.beta1, m[j], h.one_minus_beta1 * gj);
    const float old = BITS8 ? v[j] * v[j] : v[j];
    const float nv = fmaf(h.beta2, old, h.one_minus_beta2 * gj * gj);
    const float r = sqrt_approx(nv);
    w[j] = fmaf(w[j], t.decay, -t.step * __fdividef(m[j], fmaf(r, h.rbc2, h.eps)));
    v[j] = BITS8 ? r : nv;
    if (BITS8) {
      mtop = fmaxf(mtop, fabsf(m[j]));
      rtop = fmaxf(rtop, r);
    }
  }
  uint32_t bits[8];
  if (BITS8 || kRandomParam) {
    const uint64_t c = t.pos + static_cast<uint64_t>(i);  // eight positions with the same high half
    const uint32_t key = mix32(h.seed + 0x9E3779B9u * (static_cast<uint32_t>(c >> 32) + 1u));
#pragma unroll
    for (int j = 0; j < 8; ++j) bits[j] = mix32(static_cast<uint32_t>(c) + j + key);
  }
  if (BITS8) {
    const int em = block_exponent(__reduce_max_sync(~0u, __float_as_uint(mtop)));
    const int er = block_exponent(__reduce_max_sync(~0u, __float_as_uint(rtop)));
    const float im = pow2(-em), ir = pow2(-er);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      m[j] = round_code(m[j], im, (bits[j] << 4) & 0xffff0u, false);
      v[j] = round_code(v[j], ir, (bits[j] >> 12) & 0xffff0u, true);
    }
    store_codes(static_cast<uint8_t*>(t.m), i, left, vec, m);
    store_codes(static_cast<uint8_t*>(t.v), i, left, vec, v);
    if (lane == 0) {
      t.me[b0 / kBlock] = static_cast<int8_t>(em);
      t.ve[b0 / kBlock] = static_cast<int8_t>(er);
    }
  } else {
    store8(static_cast<float*>(t.m), i, left, vec, m);
    store8(static_cast<float*>(t.v), i, left, vec, v);
  }
  if (MASTER) store8(t.master, i, left, vec, w);
  if (kRandomParam) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t up = (bits[j] * 0x9E3779B1u) >> 16;
      if (isfinite(w[j])) w[j] = __uint_as_float((__float_as_uint(w[j]) + up) & 0xffff0000u);
    }
  }
  store8(static_cast<P*>(t.p), i, left, vec, w);
}

// ------------------------------------------------------------------------------------- gradient norm
struct NormTensor {
  const void* g;
  int64_t n;
  int64_t chunk0;
};
template <int CAP>
struct NormTable {
  NormTensor t[CAP];
  int64_t chunks;
  int count;
};
constexpr int kNormTable = 640;
constexpr int kNormVecs = 4;  // 16-byte vectors a thread has in flight

// partials[block] (+)= the sum of squares of the block's chunks.
template <typename G, int CAP>
__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const __grid_constant__ NormTable<CAP> tab, float* partials,
                                                             int first) {
  constexpr int VE = 16 / sizeof(G);
  constexpr int64_t kSpan = static_cast<int64_t>(kThreads) * kNormVecs * VE;
  float s[kNormVecs] = {};
  int e = 0;
  for (int64_t c = blockIdx.x; c < tab.chunks; c += gridDim.x) {
    while (e + 1 < tab.count && tab.t[e + 1].chunk0 <= c) ++e;
    const G* g = static_cast<const G*>(tab.t[e].g);
    const int64_t n = tab.t[e].n;
    const bool vec = (reinterpret_cast<uintptr_t>(g) & 15u) == 0;
    const int64_t i0 = (c - tab.t[e].chunk0) * kSpan + threadIdx.x * VE;
#pragma unroll
    for (int k = 0; k < kNormVecs; ++k) {
      const int64_t i = i0 + static_cast<int64_t>(k) * kThreads * VE;
      float z[8];
      if (vec && i + VE <= n) {
        if (sizeof(G) == 2) {
          unpack_bf16x8(__ldg(reinterpret_cast<const uint4*>(g + i)), z);
        } else {
          const float4 a = __ldg(reinterpret_cast<const float4*>(g + i));
          z[0] = a.x, z[1] = a.y, z[2] = a.z, z[3] = a.w;
        }
      } else {
#pragma unroll
        for (int j = 0; j < VE; ++j) z[j] = i + j < n ? static_cast<float>(g[i + j]) : 0.f;
      }
#pragma unroll
      for (int j = 0; j < VE; ++j) s[k] = fmaf(z[j], z[j], s[k]);
    }
  }
  float sum = (s[0] + s[1]) + (s[2] + s[3]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(~0u, sum, off);
  __shared__ float red[kWarps];
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    sum = 0.f;
    for (int w = 0; w < kWarps; ++w) sum += red[w];
    partials[blockIdx.x] = first ? sum : partials[blockIdx.x] + sum;
  }
}

__global__ void __launch_bounds__(1024) grad_norm_final_kernel(const float* partials, int n, float* norm) {
  __shared__ double red[1024];
  double s = 0;
  for (int i = threadIdx.x; i < n; i += 1024) s += static_cast<double>(partials[i]);
  red[threadIdx.x] = s;
  __syncthreads();
  for (int w = 512; w > 0; w >>= 1) {
    if (threadIdx.x < w) red[threadIdx.x] += red[threadIdx.x + w];
    __syncthreads();
  }
  if (threadIdx.x == 0) norm[0] = static_cast<float>(sqrt(red[0]));
}

bool multiple_of(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

template <int CAP, typename P, typename G, bool MASTER, bool BITS8>
cudaError_t step_list(const hylo_adamw_tensor* tensors, int count, double bias1, const AdamWHyper& h,
                      cudaStream_t stream) {
  AdamTable<CAP> tab;
  uint64_t pos = 0;
  int i = 0;
  while (i < count) {
    tab.count = 0;
    uint32_t chunks = 0;
    for (; i < count && tab.count < CAP; ++i) {
      const hylo_adamw_tensor& x = tensors[i];
      const uint64_t padded = static_cast<uint64_t>((x.n + kBlock - 1) / kBlock) * kBlock;
      const int64_t need = (x.n + kChunk - 1) / kChunk;
      if (need > 0) {
        if (chunks + static_cast<uint64_t>(need) > 0x7fffffffu) break;  // the grid is full: next launch
        AdamTensor& t = tab.t[tab.count++];
        t.p = x.param, t.g = x.grad, t.master = x.master, t.m = x.m, t.v = x.v, t.me = x.m_exp, t.ve = x.v_exp;
        t.n = x.n;
        t.pos = pos;
        t.chunk0 = chunks;
        t.vec = multiple_of(x.param, 16) && multiple_of(x.grad, 16) && multiple_of(x.master, 16) &&
                multiple_of(x.m, BITS8 ? 8 : 16) && multiple_of(x.v, BITS8 ? 8 : 16);
        t.decay = static_cast<float>(1.0 - x.lr * x.weight_decay);
        t.step = static_cast<float>(x.lr / bias1);
        chunks += static_cast<uint32_t>(need);
      }
      pos += padded;
    }
    if (tab.count == 0) continue;
    adamw_kernel<P, G, MASTER, BITS8, CAP><<<chunks, kThreads, 0, stream>>>(tab, h);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <typename P, typename G, bool MASTER, bool BITS8>
cudaError_t step_any(const hylo_adamw_tensor* tensors, int count, double bias1, const AdamWHyper& h,
                     cudaStream_t stream) {
  return count <= kSmallTable ? step_list<kSmallTable, P, G, MASTER, BITS8>(tensors, count, bias1, h, stream)
                              : step_list<kLargeTable, P, G, MASTER, BITS8>(tensors, count, bias1, h, stream);
}

template <typename P, bool MASTER>
cudaError_t step_types(const hylo_adamw_tensor* tensors, int count, int grad_dtype, int state_bits, double bias1,
                       const AdamWHyper& h, cudaStream_t stream) {
  if (grad_dtype == HYLO_F32)
    return state_bits == 8 ? step_any<P, float, MASTER, true>(tensors, count, bias1, h, stream)
                           : step_any<P, float, MASTER, false>(tensors, count, bias1, h, stream);
  return state_bits == 8 ? step_any<P, __nv_bfloat16, MASTER, true>(tensors, count, bias1, h, stream)
                         : step_any<P, __nv_bfloat16, MASTER, false>(tensors, count, bias1, h, stream);
}

template <typename G>
cudaError_t norm_list(const void* const* grads, const int64_t* sizes, int count, float* norm, float* partials, int sms,
                      cudaStream_t stream) {
  constexpr int64_t kSpan = static_cast<int64_t>(kThreads) * kNormVecs * (16 / sizeof(G));
  NormTable<kNormTable> tab;
  const int grid = sms * 8 < kNormPartials ? sms * 8 : kNormPartials;
  int i = 0, first = 1;
  do {
    tab.count = 0;
    tab.chunks = 0;
    for (; i < count && tab.count < kNormTable; ++i) {
      if (sizes[i] == 0) continue;
      tab.t[tab.count++] = NormTensor{grads[i], sizes[i], tab.chunks};
      tab.chunks += (sizes[i] + kSpan - 1) / kSpan;
    }
    grad_norm_kernel<G, kNormTable><<<grid, kThreads, 0, stream>>>(tab, partials, first);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    first = 0;
  } while (i < count);
  grad_norm_final_kernel<<<1, 1024, 0, stream>>>(partials, grid, norm);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_grad_norm(const void* const* grads, const int64_t* sizes, int count, int dtype, float* norm,
                             float* partials, int sms, cudaStream_t stream) {
  return dtype == HYLO_F32 ? norm_list<float>(grads, sizes, count, norm, partials, sms, stream)
                           : norm_list<__nv_bfloat16>(grads, sizes, count, norm, partials, sms, stream);
}

cudaError_t launch_adamw(const hylo_adamw_tensor* tensors, int count, int param_dtype, int grad_dtype, int state_bits,
                         bool masters, double bias1, const AdamWHyper& h, cudaStream_t stream) {
  if (param_dtype == HYLO_F32) return step_types<float, false>(tensors, count, grad_dtype, state_bits, bias1, h, stream);
  return masters
             ? step_types<__nv_bfloat16, true>(tensors, count, grad_dtype, state_bits, bias1, h, stream)
             : step_types<__nv_bfloat16, false>(tensors, count, grad_dtype, state_bits, bias1, h, stream);
}

}  // namespace hylo
