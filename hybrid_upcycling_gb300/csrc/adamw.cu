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
#include <type_traits>

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
  int steps;  // 8-bit states: blocks of 256 elements that a warp takes one after another
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

// The factor on the gradients; false if the step is skipped.
__device__ __forceinline__ bool gradient_factor(const AdamWHyper& h, float& gs) {
  gs = h.grad_scale;
  if (h.norm != nullptr) {
    const float norm = h.norm[0];
    if (!isfinite(norm)) return false;
    gs *= fminf(1.f, h.max_norm / (norm * fabsf(h.grad_scale) + 1e-6f));
  }
  return true;
}

// Random bits of eight consecutive positions from c on (a multiple of 8, so they share the high half).
__device__ __forceinline__ void random8(uint32_t seed, uint64_t c, uint32_t (&bits)[8]) {
  const uint32_t start = static_cast<uint32_t>(c) + mix32(seed + 0x9E3779B9u * (static_cast<uint32_t>(c >> 32) + 1u));
#pragma unroll
  for (int j = 0; j < 8; ++j) bits[j] = mix32(start + j);
}

// The same of one position.
__device__ __forceinline__ uint32_t random1(uint32_t seed, uint64_t c) {
  return mix32(static_cast<uint32_t>(c) + mix32(seed + 0x9E3779B9u * (static_cast<uint32_t>(c >> 32) + 1u)));
}

// w rounded to bf16, up with the probability of the part cut off (w finite).
__device__ __forceinline__ float round_bf16(float w, uint32_t bits) {
  return __uint_as_float((__float_as_uint(w) + ((bits * 0x9E3779B1u) >> 16)) & 0xffff0000u);
}

// The step with fp32 moments. P, G: types of parameter and gradient; MASTER: the step is taken on fp32 masters.
// HBM-bound: 385M bf16 elements with masters and fp32 gradients in 1640 us, 7.0 TB/s.
template <typename P, typename G, bool MASTER, int CAP>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ AdamTable<CAP> tab, const AdamWHyper h) {
  constexpr bool kRandomParam = sizeof(P) == 2 && !MASTER;
  float gs;
  if (!gradient_factor(h, gs)) return;
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
  load8(static_cast<const float*>(t.m), i, left, vec, m);
  load8(static_cast<const float*>(t.v), i, left, vec, v);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float gj = g[j] * gs;
    m[j] = fmaf(h.beta1, m[j], h.one_minus_beta1 * gj);
    v[j] = fmaf(h.beta2, v[j], h.one_minus_beta2 * gj * gj);
    w[j] = fmaf(w[j], t.decay, -t.step * __fdividef(m[j], fmaf(sqrt_approx(v[j]), h.rbc2, h.eps)));
  }
  store8(static_cast<float*>(t.m), i, left, vec, m);
  store8(static_cast<float*>(t.v), i, left, vec, v);
  if (MASTER) store8(t.master, i, left, vec, w);
  if (kRandomParam) {
    uint32_t bits[8];
    random8(h.seed, t.pos + static_cast<uint64_t>(i), bits);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (isfinite(w[j])) w[j] = round_bf16(w[j], bits[j]);
  }
  store8(static_cast<P*>(t.p), i, left, vec, w);
}

// ---- 8-bit states: e4m3 codes with one power of two per block
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127

__device__ __forceinline__ float2 decode2(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// The block's exponent: its largest finite magnitude (bit pattern `top`) lies in [128, 256) 2^e.
__device__ __forceinline__ int block_exponent(uint32_t top) {
  return min(120, max(-120, static_cast<int>(top >> 23) - 127 - 7));
}

constexpr uint32_t kInfBits = 0x7f800000u;
__device__ __forceinline__ float finite_or_0(float x) { return isfinite(x) ? x : 0.f; }

__device__ __forceinline__ float sqrt_ftz(float x) {
  float r;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_ftz(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// a + b, where a and b are products that have been rounded: a packed product and a packed sum would be compiled to one
// operation with one rounding.
__device__ __forceinline__ float2 add_rn(float2 a, float2 b) { return make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y)); }

// Eight elements as they lie in memory.
template <typename T>
struct Raw8 {
  uint4 q[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p, int64_t i, int left, bool vec) {
    if (vec && left >= 8) {
#pragma unroll
      for (int k = 0; k < static_cast<int>(sizeof(T) / 2); ++k) q[k] = *reinterpret_cast<const uint4*>(p + i + k * (16 / sizeof(T)));
    } else {
      float z[8];
      load8(p, i, left, false, z);
      if constexpr (sizeof(T) == 4) {
        q[0] = make_uint4(__float_as_uint(z[0]), __float_as_uint(z[1]), __float_as_uint(z[2]), __float_as_uint(z[3]));
        q[1] = make_uint4(__float_as_uint(z[4]), __float_as_uint(z[5]), __float_as_uint(z[6]), __float_as_uint(z[7]));
      } else {
        q[0] = make_uint4(pack_bf16x2(z[0], z[1]), pack_bf16x2(z[2], z[3]), pack_bf16x2(z[4], z[5]), pack_bf16x2(z[6], z[7]));
      }
    }
  }
  __device__ __forceinline__ float2 pair(int j) const {  // elements 2 j, 2 j + 1
    if constexpr (sizeof(T) == 4) {
      const uint4 v = q[j >> 1];
      return j & 1 ? make_float2(__uint_as_float(v.z), __uint_as_float(v.w)) : make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
    } else {
      const uint32_t w = j == 0 ? q[0].x : j == 1 ? q[0].y : j == 2 ? q[0].z : q[0].w;
      return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
  }
};

__device__ __forceinline__ uint2 load_codes(const uint8_t* p, int i, int left, bool vec) {
  if (vec && left >= 8) return *reinterpret_cast<const uint2*>(p + i);
  uint2 w = make_uint2(0u, 0u);
  for (int j = 0; j < left; ++j) (j < 4 ? w.x : w.y) |= static_cast<uint32_t>(p[i + j]) << (8 * (j & 3));
  return w;
}
__device__ __forceinline__ void store_codes(uint8_t* p, int i, int left, bool vec, uint2 w) {
  if (vec && left >= 8) {
    *reinterpret_cast<uint2*>(p + i) = w;
  } else {
    for (int j = 0; j < left; ++j) p[i + j] = static_cast<uint8_t>((j < 4 ? w.x : w.y) >> (8 * (j & 3)));
  }
}

// The code of |y| (< 256), y = x 2^-e, in the top byte, rounded up with the probability of the part cut off. Times
// 2^-120 the smallest normal code, 2^-6, becomes fp32's smallest normal number: the bits of |y| 2^-120 are
// then the code's exponent and mantissa (bits 26..20) with 20 more below, for subnormal codes too. The random number,
// 16 bits at `random` bits 23..8, goes to the upper 16 of those 20; times 16 the sign leaves the word at its
// top, so that rounding is one multiply-add.
__device__ __forceinline__ uint32_t round_code(float y120, uint32_t random) {
  return __float_as_uint(y120) * 16u + random;
}
__device__ __forceinline__ uint32_t low_random(uint32_t bits) { return __byte_perm(bits, 0u, 0x4104); }   // low half << 8
__device__ __forceinline__ uint32_t high_random(uint32_t bits) { return __byte_perm(bits, 0u, 0x4324); }  // high half << 8
// The top bytes of four words.
__device__ __forceinline__ uint32_t tops4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0073), __byte_perm(c, d, 0x0073), 0x5410);
}

// sqrt.approx.ftz is within a relative 2^-23 of the root, so at most 2.5 units in the last place from the root rounded to nearest.
constexpr uint32_t kRootUlps = 4;
constexpr float kMinNormal = 1.17549435e-38f;  // 2^-126
constexpr float kTiny = 7.52316384526264e-37f;  // 2^-120

// Thread blocks of one warp, 32 per SM: their loads and arithmetic fall at different times (200M bf16 elements without
// masters, before the exponents' stores were left out: 461 us with 128 threads, 397 with 64, 367 with 32).
constexpr int kThreads8 = 32;
constexpr int kWarps8 = kThreads8 / 32;
constexpr int kBlocks8 = 32;  // thread blocks per SM
// Blocks of 256 elements that a warp takes one after another: many where instructions count (bf16 parameters alone), so that its
// set-up (finding its tensor, the clip factor) is paid rarely, but no more than leave every SM its thread blocks; one where
// HBM sets the time. Measured with 16 and with 1 (every exponent stored), 200M elements, gradients in bf16 / fp32: bf16 alone
// 367 / 392 us and 407 / 419; fp32 463 / 516 and 433 / 462; masters 532 / 590 and 472 / 522.
constexpr int kMaxSteps8 = 16;  // (at most 32)

// The step with 8-bit moments. Eight elements of a lane in packed fp32 pairs. m, v and r are rounded in the order that the
// interface states, since their last bit can decide a code; the parameter's update is free to fuse. 200M elements, gradients
// in bf16 / fp32: fp32 430 / 461 us and masters 470 / 508, 6.5 to 7.1 TB/s, HBM's copy rate; bf16 alone 363 / 376, where
// instructions (57 per element, 9 of them its random bits) and waits for loads set the time.
//
// The root is approximate at first. Where that could change a code (the value within kRootUlps of its random threshold, or the
// block's largest that close to a power of two; one block in 500), r's codes of the block are left alone until the warp
// has done its blocks, and then come from roots rounded to nearest. (Those for every element: 5% longer in bf16.)
template <typename P, typename G, bool MASTER, int CAP>
__global__ void __launch_bounds__(kThreads8, kBlocks8) adamw8_kernel(const __grid_constant__ AdamTable<CAP> tab, const AdamWHyper h) {
  using W = typename std::conditional<MASTER, float, P>::type;
  constexpr bool kRandomParam = sizeof(P) == 2 && !MASTER;
  float gs;
  if (!gradient_factor(h, gs)) return;
  const AdamTensor& t = tab.t[find_entry(tab, blockIdx.x)];
  const int lane = threadIdx.x & 31;
  const bool vec = t.vec != 0;
  // Everything of the entry that the loop needs, relative to this thread block's first element and this lane's place.
  const int64_t first = static_cast<int64_t>(blockIdx.x - t.chunk0) * tab.steps * (kWarps8 * kBlock);
  const int count = static_cast<int>(min(t.n - first, static_cast<int64_t>(tab.steps) * (kWarps8 * kBlock)));
  W* const wp = (MASTER ? reinterpret_cast<W*>(t.master) : static_cast<W*>(t.p)) + first;
  P* const pp = static_cast<P*>(t.p) + first;
  const G* const gp = static_cast<const G*>(t.g) + first;
  uint8_t* const mp = static_cast<uint8_t*>(t.m) + first;
  uint8_t* const vp = static_cast<uint8_t*>(t.v) + first;
  int8_t* const me = t.me + first / kBlock;
  int8_t* const ve = t.ve + first / kBlock;
  const uint64_t pos = t.pos + static_cast<uint64_t>(first);
  const float decay = t.decay, step = -t.step;

  struct Block {
    Raw8<W> w;
    Raw8<G> g;
    uint2 m, v;
    float sm, sv;  // the blocks' powers of two
  };
  uint32_t again = 0u;  // bit k: the warp's k-th block (of at most kMaxSteps8)
#pragma unroll 1
  for (int b0 = (threadIdx.x >> 5) * kBlock; b0 < count; b0 += kWarps8 * kBlock) {
    const int i = b0 + lane * 8;
    const int left = max(0, min(8, count - i));
    Block cur;
    // The exponents first: 32 blocks share a sector, which other SMs write to. For the same reason they are written only where
    // they change (masters, 200M elements: loaded last 1003 us, first 472 to 519, so 474 to 507; bf16 alone 367 and 359).
    const int e0 = me[b0 / kBlock], e1 = ve[b0 / kBlock];
    cur.w.load(wp, i, left, vec);
    cur.g.load(gp, i, left, vec);
    cur.m = load_codes(mp, i, left, vec);
    cur.v = load_codes(vp, i, left, vec);
    cur.sm = pow2(e0);
    cur.sv = pow2(e1);
    const float2 b1 = both(h.beta1 * cur.sm);  // the product with a power of two is exact
    float2 w[4], m[4], r[4];
    float mtop = 0.f, rtop = 0.f;
    float2 odd = make_float2(0.f, 0.f);  // NaN if a value is not finite
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t two = 16 * (j & 1);
      const float2 g = __fmul2_rn(cur.g.pair(j), both(gs));
      m[j] = add_rn(__fmul2_rn(decode2((j < 2 ? cur.m.x : cur.m.y) >> two & 0xffffu), b1), __fmul2_rn(g, both(h.one_minus_beta1)));
      const float2 ro = __fmul2_rn(decode2((j < 2 ? cur.v.x : cur.v.y) >> two & 0xffffu), both(cur.sv));
      const float2 v = add_rn(__fmul2_rn(__fmul2_rn(ro, ro), both(h.beta2)), __fmul2_rn(__fmul2_rn(g, g), both(h.one_minus_beta2)));
      r[j] = make_float2(sqrt_ftz(v.x), sqrt_ftz(v.y));
      const float2 den = __ffma2_rn(r[j], both(h.rbc2), both(h.eps));
      const float2 u = __fmul2_rn(m[j], make_float2(rcp_ftz(den.x), rcp_ftz(den.y)));
      w[j] = __ffma2_rn(u, both(step), __fmul2_rn(cur.w.pair(j), both(decay)));
      mtop = fmaxf(mtop, fmaxf(fabsf(m[j].x), fabsf(m[j].y)));
      rtop = fmaxf(rtop, fmaxf(r[j].x, r[j].y));
      odd = __ffma2_rn(w[j], make_float2(0.f, 0.f), odd);
    }
    uint32_t mblock = __reduce_max_sync(~0u, __float_as_uint(mtop)), rblock = __reduce_max_sync(~0u, __float_as_uint(rtop));
    if (max(mblock, rblock) >= kInfBits) {  // rare: an infinite value has no part in its block's scale (nor has a NaN, by fmaxf)
      float a = 0.f, b = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        a = fmaxf(a, fmaxf(finite_or_0(fabsf(m[j].x)), finite_or_0(fabsf(m[j].y))));
        b = fmaxf(b, fmaxf(finite_or_0(r[j].x), finite_or_0(r[j].y)));
      }
      mblock = __reduce_max_sync(~0u, __float_as_uint(a));
      rblock = __reduce_max_sync(~0u, __float_as_uint(b));
    }
    const int em = block_exponent(mblock), er = block_exponent(rblock);
    const float2 im = both(pow2(-em)), ir = both(pow2(-er)), low = both(kTiny);
    uint32_t bits[8];
    random8(h.seed, pos + static_cast<uint64_t>(i), bits);
    uint2 mc, rc;
    uint32_t close = ~0u;  // least distance of r above its threshold - kRootUlps; a unit in the last place is 16 << 8
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uint32_t cm[4], cr[4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int p2 = 2 * k + j;
        const float2 ym = __fmul2_rn(__fmul2_rn(m[p2], im), low), yr = __fmul2_rn(__fmul2_rn(r[p2], ir), low);
        cm[2 * j] = round_code(ym.x, low_random(bits[2 * p2]));
        cm[2 * j + 1] = round_code(ym.y, low_random(bits[2 * p2 + 1]));
        cr[2 * j] = round_code(yr.x, high_random(bits[2 * p2]));
        cr[2 * j + 1] = round_code(yr.y, high_random(bits[2 * p2 + 1]));
        close = min(close, min((cr[2 * j] + 16 * kRootUlps) << 8, (cr[2 * j + 1] + 16 * kRootUlps) << 8));
      }
      const uint32_t signs = tops4(__float_as_uint(m[2 * k].x), __float_as_uint(m[2 * k].y), __float_as_uint(m[2 * k + 1].x),
                                   __float_as_uint(m[2 * k + 1].y)) & 0x80808080u;
      (k == 0 ? mc.x : mc.y) = tops4(cm[0], cm[1], cm[2], cm[3]) | signs;
      (k == 0 ? rc.x : rc.y) = tops4(cr[0], cr[1], cr[2], cr[3]);
    }
    // A byte of 0 among r's codes (rare), or a value that is not finite: element by element.
    const uint32_t zero = ((rc.x - 0x01010101u) & ~rc.x & 0x80808080u) | ((rc.y - 0x01010101u) & ~rc.y & 0x80808080u);
    const bool bad = !(odd.x + odd.y == 0.f) || !(mtop < INFINITY) || !(rtop < INFINITY);
    if (zero != 0u || bad) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float mj = j & 1 ? m[j / 2].y : m[j / 2].x, rj = j & 1 ? r[j / 2].y : r[j / 2].x;
        uint32_t& mw = j < 4 ? mc.x : mc.y;
        uint32_t& rw = j < 4 ? rc.x : rc.y;
        const int at = 8 * (j & 3);
        const uint32_t was = (rw >> at) & 0xffu;
        if (rj > 0.f && was == 0u) rw |= 1u << at;  // a non-zero r is not stored as 0
        if (!isfinite(rj)) rw |= 0x7fu << at;        // NaN
        if (!isfinite(mj)) mw |= 0x7fu << at;
      }
    }
    float wf[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) wf[2 * j] = w[j].x, wf[2 * j + 1] = w[j].y;
    if constexpr (MASTER) store8(wp, i, left, vec, wf);
    if constexpr (kRandomParam) {
      uint32_t wb[8];  // rounded in the upper half
#pragma unroll
      for (int j = 0; j < 8; ++j) wb[j] = __float_as_uint(wf[j]) + ((bits[j] * 0x9E3779B1u) >> 16);
      if (bad) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (!isfinite(wf[j])) wb[j] = isnan(wf[j]) ? 0x7fc00000u : __float_as_uint(wf[j]);
      }
      uint16_t* dst = reinterpret_cast<uint16_t*>(pp) + i;
      if (vec && left >= 8) {
        *reinterpret_cast<uint4*>(dst) = make_uint4(__byte_perm(wb[0], wb[1], 0x7632), __byte_perm(wb[2], wb[3], 0x7632),
                                                    __byte_perm(wb[4], wb[5], 0x7632), __byte_perm(wb[6], wb[7], 0x7632));
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < left) dst[j] = static_cast<uint16_t>(wb[j] >> 16);
      }
    } else {
      store8(pp, i, left, vec, wf);
    }
    store_codes(mp, i, left, vec, mc);
    if (lane == 0 && em != e0) me[b0 / kBlock] = static_cast<int8_t>(em);
    // Where an approximate root may lie on the other side of its threshold, or the block's largest of a power of two, r is
    // left as it was, for the exact roots below.
    const bool beside = rblock != 0u && ((rblock + kRootUlps) & 0x7fffffu) < 2 * kRootUlps;
    if (__any_sync(~0u, beside || close < (32 * kRootUlps) << 8)) {
      again |= 1u << (b0 / (kWarps8 * kBlock));
    } else {
      store_codes(vp, i, left, vec, rc);
      if (lane == 0 && er != e1) ve[b0 / kBlock] = static_cast<int8_t>(er);
    }
  }
#pragma unroll 1
  for (; again != 0u; again &= again - 1u) {  // rare: r of those blocks from roots rounded to nearest
    const int b0 = (threadIdx.x >> 5) * kBlock + (__ffs(static_cast<int>(again)) - 1) * (kWarps8 * kBlock);
    const int i = b0 + lane * 8;
    const int left = max(0, min(8, count - i));
    const float sv = pow2(ve[b0 / kBlock]);
    auto root = [&](int j) {
      const float g = __fmul_rn(static_cast<float>(gp[i + j]), gs), ro = __fmul_rn(decode2(vp[i + j]).x, sv);
      const float v = __fadd_rn(__fmul_rn(__fmul_rn(ro, ro), h.beta2), __fmul_rn(__fmul_rn(g, g), h.one_minus_beta2));
      return v < kMinNormal ? 0.f : __fsqrt_rn(v);
    };
    float top = 0.f;
#pragma unroll 1
    for (int j = 0; j < left; ++j) top = fmaxf(top, finite_or_0(root(j)));
    const int er = block_exponent(__reduce_max_sync(~0u, __float_as_uint(top)));
#pragma unroll 1
    for (int j = 0; j < left; ++j) {
      const float x = root(j);
      const uint32_t random = high_random(random1(h.seed, pos + static_cast<uint64_t>(i + j)));
      uint32_t c = max(round_code(x * pow2(-er) * kTiny, random) >> 24, x > 0.f ? 1u : 0u);
      if (!isfinite(x)) c = 0x7fu;
      vp[i + j] = static_cast<uint8_t>(c);
    }
    __syncwarp();  // every lane has read the old exponent
    if (lane == 0) ve[b0 / kBlock] = static_cast<int8_t>(er);
  }
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
constexpr int kSmallNorm = 32, kLargeNorm = 640;
constexpr int kNormVecs = 4;  // 16-byte vectors a thread has in flight

// partials[block] (+)= the sum of squares of the block's chunks. HBM-bound: 385M elements with the final kernel in 118 us
// (bf16, 6.5 TB/s) and 223 us (fp32, 6.9 TB/s); with each load behind its own bounds check, as in the
// ragged chunks, 125 and 235 us.
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
    if (vec && (c - tab.t[e].chunk0 + 1) * kSpan <= n) {  // the whole chunk: all its loads first
      uint4 q[kNormVecs];
#pragma unroll
      for (int k = 0; k < kNormVecs; ++k) q[k] = __ldg(reinterpret_cast<const uint4*>(g + i0 + static_cast<int64_t>(k) * kThreads * VE));
#pragma unroll
      for (int k = 0; k < kNormVecs; ++k) {
        float z[8];
        if (sizeof(G) == 2) {
          unpack_bf16x8(q[k], z);
        } else {
          z[0] = __uint_as_float(q[k].x), z[1] = __uint_as_float(q[k].y);
          z[2] = __uint_as_float(q[k].z), z[3] = __uint_as_float(q[k].w);
        }
#pragma unroll
        for (int j = 0; j < VE; ++j) s[k] = fmaf(z[j], z[j], s[k]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < kNormVecs; ++k) {
        const int64_t i = i0 + static_cast<int64_t>(k) * kThreads * VE;
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          const float z = i + j < n ? static_cast<float>(g[i + j]) : 0.f;
          s[k] = fmaf(z, z, s[k]);
        }
      }
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
cudaError_t step_list(const hylo_adamw_tensor* tensors, int count, double bias1, const AdamWHyper& h, int sms,
                      cudaStream_t stream) {
  AdamTable<CAP> tab;
  int64_t total = 0;
  for (int k = 0; k < count; ++k) total += tensors[k].n;
  const int64_t unit = BITS8 ? kWarps8 * kBlock : kChunk;  // elements of a thread block and step
  const int64_t fill = total / (static_cast<int64_t>(kBlocks8) * sms * unit);
  tab.steps = BITS8 && sizeof(P) == 2 && !MASTER ? static_cast<int>(fill < 1 ? 1 : fill > kMaxSteps8 ? kMaxSteps8 : fill) : 1;
  for (int k = 0; k < count; ++k)  // a tensor's thread blocks have to fit a grid (2^40 elements: 4 steps)
    while (tensors[k].n / (tab.steps * unit) >= (int64_t(1) << 30)) tab.steps *= 2;
  uint64_t pos = 0;
  int i = 0;
  while (i < count) {
    tab.count = 0;
    uint32_t chunks = 0;
    for (; i < count && tab.count < CAP; ++i) {
      const hylo_adamw_tensor& x = tensors[i];
      const uint64_t padded = static_cast<uint64_t>((x.n + kBlock - 1) / kBlock) * kBlock;
      const int64_t chunk = tab.steps * unit;
      const int64_t need = (x.n + chunk - 1) / chunk;
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
    if (BITS8)
      adamw8_kernel<P, G, MASTER, CAP><<<chunks, kThreads8, 0, stream>>>(tab, h);
    else
      adamw_kernel<P, G, MASTER, CAP><<<chunks, kThreads, 0, stream>>>(tab, h);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <typename P, typename G, bool MASTER, bool BITS8>
cudaError_t step_any(const hylo_adamw_tensor* tensors, int count, double bias1, const AdamWHyper& h, int sms,
                     cudaStream_t stream) {
  return count <= kSmallTable ? step_list<kSmallTable, P, G, MASTER, BITS8>(tensors, count, bias1, h, sms, stream)
                              : step_list<kLargeTable, P, G, MASTER, BITS8>(tensors, count, bias1, h, sms, stream);
}

template <typename P, bool MASTER>
cudaError_t step_types(const hylo_adamw_tensor* tensors, int count, int grad_dtype, int state_bits, double bias1,
                       const AdamWHyper& h, int sms, cudaStream_t stream) {
  if (grad_dtype == HYLO_F32)
    return state_bits == 8 ? step_any<P, float, MASTER, true>(tensors, count, bias1, h, sms, stream)
                           : step_any<P, float, MASTER, false>(tensors, count, bias1, h, sms, stream);
  return state_bits == 8 ? step_any<P, __nv_bfloat16, MASTER, true>(tensors, count, bias1, h, sms, stream)
                         : step_any<P, __nv_bfloat16, MASTER, false>(tensors, count, bias1, h, sms, stream);
}

template <int CAP, typename G>
cudaError_t norm_list(const void* const* grads, const int64_t* sizes, int count, float* norm, float* partials, int sms,
                      cudaStream_t stream) {
  constexpr int64_t kSpan = static_cast<int64_t>(kThreads) * kNormVecs * (16 / sizeof(G));
  NormTable<CAP> tab;
  const int grid = sms * 8 < kNormPartials ? sms * 8 : kNormPartials;
  int i = 0, first = 1;
  do {
    tab.count = 0;
    tab.chunks = 0;
    for (; i < count && tab.count < CAP; ++i) {
      if (sizes[i] == 0) continue;
      tab.t[tab.count++] = NormTensor{grads[i], sizes[i], tab.chunks};
      tab.chunks += (sizes[i] + kSpan - 1) / kSpan;
    }
    grad_norm_kernel<G, CAP><<<grid, kThreads, 0, stream>>>(tab, partials, first);
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
  // A short list goes with short kernel parameters.
  if (count <= kSmallNorm)
    return dtype == HYLO_F32 ? norm_list<kSmallNorm, float>(grads, sizes, count, norm, partials, sms, stream)
                             : norm_list<kSmallNorm, __nv_bfloat16>(grads, sizes, count, norm, partials, sms, stream);
  return dtype == HYLO_F32 ? norm_list<kLargeNorm, float>(grads, sizes, count, norm, partials, sms, stream)
                           : norm_list<kLargeNorm, __nv_bfloat16>(grads, sizes, count, norm, partials, sms, stream);
}

cudaError_t launch_adamw(const hylo_adamw_tensor* tensors, int count, int param_dtype, int grad_dtype, int state_bits,
                         bool masters, double bias1, const AdamWHyper& h, int sms, cudaStream_t stream) {
  if (param_dtype == HYLO_F32) return step_types<float, false>(tensors, count, grad_dtype, state_bits, bias1, h, sms, stream);
  return masters
             ? step_types<__nv_bfloat16, true>(tensors, count, grad_dtype, state_bits, bias1, h, sms, stream)
             : step_types<__nv_bfloat16, false>(tensors, count, grad_dtype, state_bits, bias1, h, sms, stream);
}

}  // namespace hylo
