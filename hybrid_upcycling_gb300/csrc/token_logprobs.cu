// Log-probabilities of given tokens from logits, with entropy and the k largest alternatives, and
// their gradient. Per row, with y = z / tau:
//   m = max y, s = sum e^(y - m), a = sum e^(y - m) (y - m)   (one online pass, fp32)
//   log p_v = y_v - m - log s,  entropy = log s - a / s
//   dz = 1/tau [ g_lp (1[v = t] - p_v) - g_H p_v (log p_v + entropy) ]
// Both directions are bound by HBM: the forward reads each logit once, the backward reads it
// once and writes the gradient once.
//
// Alternatives. While a row streams by, each 256-word block's largest logit is kept ("group
// maximum"). Order the groups by (maximum, lower position first): a word of any group behind the
// first k is beaten by the k words that are the maxima of those k groups, also under the tie
// rule, because groups are contiguous runs of words. So only k groups are read again
// (from L2), and of those only words not below the k-th group maximum are candidates; each
// candidate's rank is the number of candidates that beat it.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "hylo_ops_internal.h"
#include "sm103_ptx.cuh"

namespace hylo {
namespace {

constexpr float kLog2eF = 1.4426950408889634f;
constexpr float kLn2F = 0.6931471805599453f;
// log2-probabilities below this are taken as this: e^y is 0 there in fp32, and products with it stay finite
constexpr float kFloor = -200.f;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBlock = 256;      // words per block: one group unless the vocabulary is very long
constexpr int kBatch = 4;        // blocks a warp has in flight
constexpr int kMaxGroups = 1024; // group maxima kept per row
constexpr int kCand = 1024;      // candidates held at once
constexpr int kCandBatch = (kCand - HYLO_TOP_MAX) / kBlock;  // blocks gathered at once when all do not fit

// Maximum that keeps a NaN (a row with one has NaN results).
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float warp_max_nan(float v) {
  float r;
  asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static constexpr int kVec = 4;
  static constexpr int kKeyBits = 32;  // leading bits of the order key in which values differ
  static __device__ __forceinline__ float get(float x) { return x; }
  static __device__ __forceinline__ void unpack(uint4 v, float* z) {
    z[0] = __uint_as_float(v.x);
    z[1] = __uint_as_float(v.y);
    z[2] = __uint_as_float(v.z);
    z[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 pack(const float* z) {
    return make_uint4(__float_as_uint(z[0]), __float_as_uint(z[1]), __float_as_uint(z[2]), __float_as_uint(z[3]));
  }
  static __device__ __forceinline__ float put(float x) { return x; }
};
template <>
struct Elem<__nv_bfloat16> {
  static constexpr int kVec = 8;
  static constexpr int kKeyBits = 16;
  static __device__ __forceinline__ float get(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ void unpack(uint4 v, float* z) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      z[2 * i] = __uint_as_float(w[i] << 16);
      z[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float* z) {
    return make_uint4(pack_bf16x2(z[0], z[1]), pack_bf16x2(z[2], z[3]), pack_bf16x2(z[4], z[5]), pack_bf16x2(z[6], z[7]));
  }
  static __device__ __forceinline__ __nv_bfloat16 put(float x) { return __float2bfloat16_rn(x); }
};
template <>
struct Elem<__half> {
  static constexpr int kVec = 8;
  static constexpr int kKeyBits = 19;
  static __device__ __forceinline__ float get(__half x) { return __half2float(x); }
  static __device__ __forceinline__ void unpack(uint4 v, float* z) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      z[2 * i] = f.x;
      z[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ uint4 pack(const float* z) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(z[2 * i], z[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  static __device__ __forceinline__ __half put(float x) { return __float2half_rn(x); }
};

// Whole numbers in the order of the values: NaN above all, -0 equal to +0.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (isnan(x)) return 0xffffffffu;
  const uint32_t b = __float_as_uint(x + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t key) {
  if (key == 0xffffffffu) return __uint_as_float(0x7fffffffu);
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7fffffffu) : ~key);
}
// A candidate: larger is better (larger logit, then lower index).
__device__ __forceinline__ uint64_t cand_of(uint32_t key, int idx) {
  return (static_cast<uint64_t>(key) << 32) | (0xffffffffu - static_cast<uint32_t>(idx));
}
__device__ __forceinline__ int cand_index(uint64_t c) { return static_cast<int>(0xffffffffu - static_cast<uint32_t>(c)); }

// Running softmax sums of some of a row's words, relative to the largest of them: mx is a raw
// logit, s = sum 2^((z - mx) c), a = the same weighted with (z - mx) c.
struct Sums {
  float mx, s, a;
};

// The finite stand-in for a maximum of -inf (no word allowed so far): z - 0 = -inf is then floored.
__device__ __forceinline__ float base_of(float mx) { return mx == -INFINITY ? 0.f : mx; }

__device__ __forceinline__ void rebase(Sums& r, float mx, float c) {
  const float d = max_nan((r.mx - base_of(mx)) * c, kFloor);
  const float w = ex2_approx(d);
  r.a = w * fmaf(r.s, d, r.a);
  r.s *= w;
  r.mx = mx;
}

__device__ __forceinline__ void merge(Sums& r, Sums o, float c) {
  const float mx = max_nan(r.mx, o.mx);
  rebase(r, mx, c);
  rebase(o, mx, c);
  r.s += o.s;
  r.a += o.a;
}

// A row in aligned coordinates: word v lies at u = v + lead, and u = 0 is 16-byte aligned.
template <typename T>
struct Row {
  const T* base;  // the address of u = 0 (read only at u >= lead)
  int lead;
  int64_t end;    // lead + V
  __device__ Row(const void* z, int64_t offset, int V) {
    const T* p = static_cast<const T*>(z) + offset;
    lead = static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T));
    base = p - lead;
    end = static_cast<int64_t>(lead) + V;
  }
  // The vector at u0 (a multiple of kVec); words outside the row read as -inf. kInPlace: the kernel
  // may write over the logits, so the read-only path is not used.
  template <bool kInPlace = false>
  __device__ __forceinline__ void load(int64_t u0, float* z) const {
    constexpr int VE = Elem<T>::kVec;
    if (u0 >= lead && u0 + VE <= end) {
      const uint4* p = reinterpret_cast<const uint4*>(base + u0);
      Elem<T>::unpack(kInPlace ? *p : __ldg(p), z);
    } else {
#pragma unroll
      for (int i = 0; i < VE; ++i) z[i] = u0 + i >= lead && u0 + i < end ? Elem<T>::get(base[u0 + i]) : -INFINITY;
    }
  }
};

template <typename T>
__global__ void __launch_bounds__(kThreads) token_logprobs_kernel(const TokenRows in, const TokenOut out, int group_shift) {
  constexpr int VE = Elem<T>::kVec;
  constexpr int VL = kBlock / (32 * VE);  // vectors of a block per lane
  __shared__ Sums warp_sums[kWarps];
  __shared__ uint32_t group_key[kMaxGroups];
  __shared__ uint64_t cand[kCand];
  __shared__ uint64_t top[HYLO_TOP_MAX];
  __shared__ int sel[HYLO_TOP_MAX];
  __shared__ uint32_t bound_key;
  __shared__ int count;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int group_blocks = 1 << group_shift;
  const int run = max(kBatch, group_blocks);  // consecutive blocks of one warp

  for (int64_t n = blockIdx.x; n < in.N; n += gridDim.x) {
    const Row<T> row(in.z, n * in.ld, in.V);
    const int64_t blocks = (row.end + kBlock - 1) / kBlock;
    const int groups = static_cast<int>((blocks + group_blocks - 1) >> group_shift);
    Sums r{-INFINITY, 0.f, 0.f};
    for (int64_t b0 = static_cast<int64_t>(warp) * run; b0 < blocks; b0 += kWarps * run) {
      const int64_t b1 = min(blocks, b0 + run);
      float gm = -INFINITY;
      for (int64_t b = b0; b < b1; b += kBatch) {
        float z[kBatch][VL * VE];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
#pragma unroll
          for (int j = 0; j < VL; ++j) row.load((b + i) * kBlock + (j * 32 + lane) * VE, z[i] + j * VE);
        }
        float mx = r.mx;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          float bm = z[i][0];
#pragma unroll
          for (int j = 1; j < VL * VE; ++j) bm = max_nan(bm, z[i][j]);
          mx = max_nan(mx, bm);
          if (out.k > 0 && b + i < b1) {
            gm = max_nan(gm, bm);
            if (((b + i + 1) & (group_blocks - 1)) == 0 || b + i + 1 == blocks) {
              gm = warp_max_nan(gm);
              if (lane == 0) group_key[(b + i) >> group_shift] = order_key(gm);
              gm = -INFINITY;
            }
          }
        }
        rebase(r, mx, in.c);
        const float m0 = base_of(mx);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
#pragma unroll
          for (int j = 0; j < VL * VE; ++j) {
            const float y = max_nan((z[i][j] - m0) * in.c, kFloor);
            const float e = ex2_approx(y);
            r.s += e;
            r.a = fmaf(e, y, r.a);
          }
        }
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
      merge(r, Sums{__shfl_xor_sync(~0u, r.mx, off), __shfl_xor_sync(~0u, r.s, off), __shfl_xor_sync(~0u, r.a, off)}, in.c);
    if (lane == 0) warp_sums[warp] = r;
    if (tid == 0) count = 0;
    __syncthreads();
    r = warp_sums[0];
    for (int w = 1; w < kWarps; ++w) merge(r, warp_sums[w], in.c);  // every thread the same
    const float log_s = logf(r.s);
    if (tid == 0) {
      const int64_t t = in.tokens[n];
      float lp = 0.f;
      if (t >= in.V)
        lp = __uint_as_float(0x7fffffffu);
      else if (t >= 0)
        lp = r.mx == -INFINITY ? -INFINITY : (Elem<T>::get(row.base[t + row.lead]) - r.mx) * in.inv_tau - log_s;
      out.logp[n] = lp;
      if (out.entropy) out.entropy[n] = r.mx == -INFINITY ? 0.f : log_s - kLn2F * r.a / r.s;
      if (out.lse) out.lse[n] = r.mx == -INFINITY ? -INFINITY : r.mx * in.inv_tau + log_s;
      if (out.stats) out.stats[n] = make_float2(r.mx, log_s);
    }
    if (out.k > 0) {
      // ---- the k-th largest group maximum, bit by bit from the top, and the k first groups
      const int kk = min(out.k, groups);
      if (warp == 0) {
        uint32_t t = 0;
        for (int bit = 31; bit >= 32 - Elem<T>::kKeyBits; --bit) {
          const uint32_t probe = t | (1u << bit);
          int have = 0;
          for (int g = lane; g < groups; g += 32) have += group_key[g] >= probe;
          if (__reduce_add_sync(~0u, have) >= kk) t = probe;
        }
        constexpr uint32_t kHigh = Elem<T>::kKeyBits == 32 ? ~0u : ~0u << (32 - Elem<T>::kKeyBits);
        int over = 0;
        for (int g = lane; g < groups; g += 32) over += (group_key[g] & kHigh) > t;
        over = __reduce_add_sync(~0u, over);
        int placed = 0, equal_left = kk - over;  // equal maxima: the first groups
        for (int g0 = 0; g0 < groups; g0 += 32) {
          const uint32_t key = g0 + lane < groups ? group_key[g0 + lane] & kHigh : 0u;
          const bool eq = g0 + lane < groups && key == t;
          const uint32_t eqs = __ballot_sync(~0u, eq);
          const bool take = (g0 + lane < groups && key > t) || (eq && __popc(eqs & ((1u << lane) - 1u)) < equal_left);
          const uint32_t takes = __ballot_sync(~0u, take);
          if (take) sel[placed + __popc(takes & ((1u << lane) - 1u))] = g0 + lane;
          placed += __popc(takes);
          equal_left -= min(equal_left, __popc(eqs));
        }
        if (lane == 0) bound_key = kk == out.k ? t : 0u;  // fewer groups than k: any word may be among the k
      }
      __syncthreads();
      // ---- candidates: all at once if they fit, else some blocks at a time under a rising bound
      uint64_t bound = static_cast<uint64_t>(bound_key) << 32;  // candidates are not below it
      const int64_t nblk = static_cast<int64_t>(kk) << group_shift;  // blocks of the chosen groups
      auto gather = [&](int64_t i0, int64_t i1) {
        for (int64_t i = i0 + warp; i < i1; i += kWarps) {
          const int64_t b = (static_cast<int64_t>(sel[i >> group_shift]) << group_shift) + (i & (group_blocks - 1));
#pragma unroll
          for (int j = 0; j < VL; ++j) {
            const int64_t u = b * kBlock + (j * 32 + lane) * VE;
            float z[VE];
            row.load(u, z);
#pragma unroll
            for (int q = 0; q < VE; ++q) {
              if (u + q < row.lead || u + q >= row.end) continue;
              const uint64_t cd = cand_of(order_key(z[q]), static_cast<int>(u + q - row.lead));
              if (cd >= bound) {
                const int at = atomicAdd(&count, 1);
                if (at < kCand) cand[at] = cd;
              }
            }
          }
        }
      };
      auto rank_all = [&](int have) {  // the best k of cand[0..have), in order, into top
        for (int i = tid; i < have; i += kThreads) {
          const uint64_t mine = cand[i];
          int rank = 0;
          for (int j = 0; j < have; ++j) rank += cand[j] > mine;
          if (rank < out.k) top[rank] = mine;
        }
      };
      gather(0, nblk);
      __syncthreads();
      int have = count;
      if (have > kCand) {
        have = 0;
        for (int64_t i0 = 0; i0 < nblk; i0 += kCandBatch) {
          __syncthreads();
          if (tid == 0) count = have;
          for (int i = tid; i < have; i += kThreads) cand[i] = top[i];
          __syncthreads();
          gather(i0, min(nblk, i0 + kCandBatch));
          __syncthreads();
          const int all = count;
          rank_all(all);
          have = min(out.k, all);
          __syncthreads();
          if (have == out.k) bound = top[out.k - 1];
        }
      } else {
        rank_all(have);
        __syncthreads();
      }
      for (int i = tid; i < out.k; i += kThreads) {
        const uint64_t cd = top[i];
        const float z = key_value(static_cast<uint32_t>(cd >> 32));
        out.top_logp[n * out.k + i] = r.mx == -INFINITY ? -INFINITY : (z - r.mx) * in.inv_tau - log_s;
        out.top_ids[n * out.k + i] = cand_index(cd);
      }
    }
    __syncthreads();  // shared memory is free for the next row
  }
}

constexpr int kBwdThreads = 256;
constexpr int kBwdVecs = 4;  // vectors of a thread per piece

// A block takes pieces of kBwdThreads * kBwdVecs vectors, rows one after another.
template <typename T>
__global__ void __launch_bounds__(kBwdThreads) token_logprobs_bwd_kernel(const TokenRows in, const TokenGrad g,
                                                                         int pieces) {
  constexpr int VE = Elem<T>::kVec;
  constexpr int64_t kPiece = static_cast<int64_t>(kBwdThreads) * kBwdVecs * VE;
  const int64_t total = static_cast<int64_t>(in.N) * pieces;
  for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
    const int64_t n = w / pieces;
    const int64_t u0 = (w - n * pieces) * kPiece;
    const Row<T> row(in.z, n * in.ld, in.V);
    if (u0 >= row.end) continue;
    T* dst = static_cast<T*>(g.dz) + n * g.ldd;
    const bool vec = (reinterpret_cast<uintptr_t>(dst) & 15u) / sizeof(T) == static_cast<uint32_t>(row.lead);
    dst -= row.lead;
    const float2 st = g.stats[n];
    const int64_t tok = in.tokens[n];
    const bool empty = st.x == -INFINITY;
    float gl = g.g_logp != nullptr && tok >= 0 ? g.g_logp[n] : 0.f;
    if (tok >= in.V) gl = __uint_as_float(0x7fffffffu);
    const float gh = g.g_entropy != nullptr ? g.g_entropy[n] : 0.f;
    const float H = gh != 0.f ? g.entropy[n] : 0.f;
    // dz = p (A + B log2 p) + 1[v = t] gl / tau
    const float A = empty ? 0.f : -in.inv_tau * (gl + gh * H), B = empty ? 0.f : -in.inv_tau * gh * kLn2F;
    const float hit = empty ? 0.f : in.inv_tau * gl;
    const int64_t ut = tok >= 0 && tok < in.V ? tok + row.lead : -1;
    const float m0 = base_of(st.x), l2 = empty ? 0.f : st.y * kLog2eF;
    float z[kBwdVecs][VE];
#pragma unroll
    for (int i = 0; i < kBwdVecs; ++i) row.template load<true>(u0 + (i * kBwdThreads + threadIdx.x) * VE, z[i]);
#pragma unroll
    for (int i = 0; i < kBwdVecs; ++i) {
      const int64_t u = u0 + (i * kBwdThreads + threadIdx.x) * VE;
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        const float y = max_nan(fmaf(z[i][j] - m0, in.c, -l2), kFloor);
        float d = ex2_approx(y) * fmaf(B, y, A);
        if (u + j == ut) d += hit;
        z[i][j] = d;
      }
      if (vec && u >= row.lead && u + VE <= row.end) {
        __stcs(reinterpret_cast<uint4*>(dst + u), Elem<T>::pack(z[i]));
      } else {
#pragma unroll
        for (int j = 0; j < VE; ++j)
          if (u + j >= row.lead && u + j < row.end) dst[u + j] = Elem<T>::put(z[i][j]);
      }
    }
  }
}

template <typename T>
cudaError_t launch_fwd(const TokenRows& in, const TokenOut& out, int sms, cudaStream_t stream) {
  const int64_t blocks = (static_cast<int64_t>(in.V) + Elem<T>::kVec + kBlock - 1) / kBlock;
  int shift = 0;
  while ((blocks >> shift) >= kMaxGroups) ++shift;
  const int grid = in.N < 4 * sms ? in.N : 4 * sms;
  token_logprobs_kernel<T><<<grid, kThreads, 0, stream>>>(in, out, shift);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_bwd(const TokenRows& in, const TokenGrad& g, int sms, cudaStream_t stream) {
  const int64_t piece = static_cast<int64_t>(kBwdThreads) * kBwdVecs * Elem<T>::kVec;
  const int64_t pieces = (static_cast<int64_t>(in.V) + Elem<T>::kVec - 1 + piece - 1) / piece;
  const int64_t total = pieces * in.N, cap = static_cast<int64_t>(sms) * 64;
  token_logprobs_bwd_kernel<T>
      <<<static_cast<int>(total < cap ? total : cap), kBwdThreads, 0, stream>>>(in, g, static_cast<int>(pieces));
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_token_logprobs(const TokenRows& in, const TokenOut& out, int dtype, int sms, cudaStream_t stream) {
  switch (dtype) {
    case HYLO_F32: return launch_fwd<float>(in, out, sms, stream);
    case HYLO_BF16: return launch_fwd<__nv_bfloat16>(in, out, sms, stream);
    default: return launch_fwd<__half>(in, out, sms, stream);
  }
}

cudaError_t launch_token_logprobs_bwd(const TokenRows& in, const TokenGrad& g, int dtype, int sms,
                                      cudaStream_t stream) {
  switch (dtype) {
    case HYLO_F32: return launch_bwd<float>(in, g, sms, stream);
    case HYLO_BF16: return launch_bwd<__nv_bfloat16>(in, g, sms, stream);
    default: return launch_bwd<__half>(in, g, sms, stream);
  }
}

}  // namespace hylo
