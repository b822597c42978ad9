// Log-probabilities of given tokens from logits, with entropy and the k largest alternatives, and
// their gradient. Per row, with y = z / tau:
//   m = max y, s = sum e^(y - m), a = sum e^(y - m) (y - m)   (one online pass, fp32)
//   log p_v = y_v - m - log s,  entropy = log s - a / s
//   dz = 1/tau [ g_lp (1[v = t] - p_v) - g_H p_v (log p_v + entropy) ]
// Both directions are bound by HBM: the forward reads each logit once, the backward reads it
// once and writes the gradient once.
//
// Alternatives. While a row streams by, the largest logit of each of at most kMaxGroups contiguous
// groups of words is kept. Order the groups by (maximum, lower position first): a word of any
// group behind the first k is beaten by the k words that are the maxima of those k groups, also
// under the tie rule, because groups are contiguous. So only k groups are read again (from
// L2): of their words, those above the k-th group maximum T are candidates, and the first
// k equal to T; each candidate's rank is the number of candidates that beat it.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "hylo_ops_internal.h"
#include "row_split.h"
#include "sm103_ptx.cuh"

namespace hylo {
namespace {

constexpr float kLog2eF = 1.4426950408889634f;
constexpr float kLn2F = 0.6931471805599453f;
// log2-probabilities below this are taken as this: e^y is 0 there in fp32, and products with it stay finite
constexpr float kFloor = -200.f;

constexpr int kMaxGroups = 256;  // group maxima kept per row
constexpr int kMaxSplit = 16;    // CTAs of a cluster that share a row

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

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static constexpr int kVec = 4;
  static constexpr int kKeyBits = 32;  // leading bits of the order key in which values of the type differ
  static __device__ __forceinline__ float get(float x) { return x; }
  static constexpr uint32_t kMasked = 0xff800000u;  // a 32-bit word of -inf
  static __device__ __forceinline__ float vec_max(uint4 v) {
    return max_nan(max_nan(__uint_as_float(v.x), __uint_as_float(v.y)), max_nan(__uint_as_float(v.z), __uint_as_float(v.w)));
  }
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
  static constexpr uint32_t kMasked = 0xff80ff80u;
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ float vec_max(uint4 v) {
    const uint32_t m = max2(max2(v.x, v.y), max2(v.z, v.w));
    return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
  }
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
  static constexpr uint32_t kMasked = 0xfc00fc00u;
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ float vec_max(uint4 v) {
    const uint32_t m = max2(max2(v.x, v.y), max2(v.z, v.w));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&m));
    return max_nan(f.x, f.y);
  }
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
constexpr uint32_t kMinusInfKey = 0x007fffffu, kInfKey = 0xff800000u;  // those of -inf and inf
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

// The sums of `width` lanes (a power of two; the other lanes hold copies of theirs) together, the same in every lane:
// a fixed tree of additions.
__device__ __forceinline__ Sums join_lanes(Sums r, int width, float c) {
  rebase(r, warp_max_nan(r.mx), c);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    if (off < width) {
      r.s += __shfl_xor_sync(~0u, r.s, off);
      r.a += __shfl_xor_sync(~0u, r.a, off);
    }
  }
  return r;
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
  __device__ __forceinline__ bool inside(int64_t u0, int64_t u1) const { return u0 >= lead && u1 <= end; }
  // The vector at u0 (a multiple of kVec), which lies inside the row. kInPlace: the kernel may write
  // over the logits, so the read-only path is not used.
  template <bool kInPlace = false>
  __device__ __forceinline__ uint4 whole(int64_t u0) const {
    const uint4* p = reinterpret_cast<const uint4*>(base + u0);
    return kInPlace ? *p : __ldg(p);
  }
  // The vector at u0 where it may reach over the row's ends, word by word; words outside are -inf.
  template <bool kInPlace = false>
  __device__ uint4 edge(int64_t u0) const {
    constexpr int VE = Elem<T>::kVec;
    if (inside(u0, u0 + VE)) return whole<kInPlace>(u0);
    uint4 v = make_uint4(Elem<T>::kMasked, Elem<T>::kMasked, Elem<T>::kMasked, Elem<T>::kMasked);
    T* t = reinterpret_cast<T*>(&v);
#pragma unroll
    for (int i = 0; i < VE; ++i)
      if (u0 + i >= lead && u0 + i < end) t[i] = base[u0 + i];
    return v;
  }
};

// Folds the words of one vector, relative to the maximum m0: y = (z - m0) c. The difference comes first: it is
// exact where it matters, and finite logits of any size cannot give inf - inf. A word of -inf has e^y y = 0
// only with kMasked, which floors y; otherwise it makes `a` NaN.
template <typename T, bool kMasked>
__device__ __forceinline__ void fold(uint4 v, float m0, float c, float2& s, float2& a) {
  float z[Elem<T>::kVec];
  Elem<T>::unpack(v, z);
  const float2 nm = make_float2(-m0, -m0), c2 = make_float2(c, c);
#pragma unroll
  for (int j = 0; j < Elem<T>::kVec / 2; ++j) {
    float2 y = __fmul2_rn(__fadd2_rn(make_float2(z[2 * j], z[2 * j + 1]), nm), c2);
    if (kMasked) {
      y.x = max_nan(y.x, kFloor);
      y.y = max_nan(y.y, kFloor);
    }
    const float2 e = make_float2(ex2_approx(y.x), ex2_approx(y.y));
    s = __fadd2_rn(s, e);
    a = __ffma2_rn(e, y, a);
  }
}

// What the selection of alternatives works with, for the kWarps warps that do it.
template <int kWarps>
struct Choice {
  static constexpr int kCand = kWarps > 1 ? 1024 : 512;  // candidates held at once
  static constexpr int kHits = kWarps > 1 ? 256 : 96;    // vectors with candidates
  uint64_t cand[kCand];
  uint64_t top[HYLO_TOP_MAX];
  uint4 hit_vec[kHits];
  int hit_at[kHits];  // which vector of the row
  int sel[HYLO_TOP_MAX];
  int equal[kWarps];
  uint32_t bound_key;
  int count;
  int hits;
};

template <int kWarps>
__device__ __forceinline__ void sync_warps() {
  if (kWarps > 1)
    __syncthreads();
  else
    __syncwarp();
}

// A row's groups: 2^vec_shift vectors each (`count` of them).
struct Groups {
  int vec_shift;
  int count;
};

// The best k of cand[0..have), in order, into top: an entry's rank is the number of entries that beat it.
template <int kWarps>
__device__ __forceinline__ void rank_all(Choice<kWarps>& sh, int have, int k, int tid) {
  for (int i = tid; i < have; i += kWarps * 32) {
    const uint64_t mine = sh.cand[i];
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < have; ++j) rank += sh.cand[j] > mine;
    if (rank < k) sh.top[rank] = mine;
  }
}

// The bound below which no word is looked at, from the kk-th largest group maximum. Where that is -inf (masked words), it is
// the next key: every word above -inf lies in a chosen group, and if fewer than k do, words of -inf are filled in.
template <typename T>
__device__ __forceinline__ uint32_t bound_of(uint32_t key) {
  constexpr uint32_t kHigh = Elem<T>::kKeyBits == 32 ? ~0u : ~0u << (32 - Elem<T>::kKeyBits);
  return (key & kHigh) == (kMinusInfKey & kHigh) ? (kMinusInfKey & kHigh) + (~kHigh + 1u) : key & kHigh;
}

// The first kk groups by (maximum, position) into sh.sel, by position, and the bound into sh.bound_key; one warp. A search for
// the kk-th largest maximum in the leading bits of its key, bit by bit below the bits that the largest and the smallest
// maximum share, until exactly kk maxima reach t. (A thread per group that counts the groups before its own, 256
// comparisons each, took longer: one row of 128256 fp32 words with 20 alternatives 10.2 us against 8.5, 600 rows of
// 1000 words 14.8 against 7.3.) Loops are kept rolled here and below: this code runs once per row.
template <typename T, int kWarps>
__device__ void choose_groups(Choice<kWarps>& sh, const uint32_t* group_key, int groups, int kk, int k) {
  constexpr uint32_t kHigh = Elem<T>::kKeyBits == 32 ? ~0u : ~0u << (32 - Elem<T>::kKeyBits);
  constexpr int kPer = kMaxGroups / 32;
  const int lane = threadIdx.x & 31;
  uint32_t key[kPer], low = ~0u, high = 0u;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const bool real = j * 32 + lane < groups;
    key[j] = real ? group_key[j * 32 + lane] & kHigh : 0u;  // 0: below every key
    low = real ? min(low, key[j]) : low;
    high = max(high, key[j]);
  }
  low = __reduce_min_sync(~0u, low);
  high = __reduce_max_sync(~0u, high);
  uint32_t t = low;  // at least kk maxima reach t
  if (low != high && groups > kk) {
    const int top = 31 - __clz(static_cast<int>(low ^ high));
    t = high & ~((2u << top) - 1u);
#pragma unroll 1
    for (int bit = top; bit >= 32 - Elem<T>::kKeyBits; --bit) {
      const uint32_t probe = t | (1u << bit);
      int h0 = 0, h1 = 0;
#pragma unroll
      for (int j = 0; j < kPer; j += 2) {
        h0 += key[j] >= probe;
        h1 += key[j + 1] >= probe;
      }
      const int have = __reduce_add_sync(~0u, h0 + h1);
      if (have >= kk) t = probe;
      if (have == kk) break;
    }
  }
  int over = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) over += key[j] > t;
  int equal_left = kk - __reduce_add_sync(~0u, over), placed = 0;  // equal maxima: the first groups
  const uint32_t below = (1u << lane) - 1u;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const uint32_t eqs = __ballot_sync(~0u, key[j] == t);
    const bool take = key[j] > t || (key[j] == t && __popc(eqs & below) < equal_left);
    const uint32_t takes = __ballot_sync(~0u, take);
    if (take) sh.sel[placed + __popc(takes & below)] = j * 32 + lane;
    placed += __popc(takes);
    equal_left -= min(equal_left, __popc(eqs));
  }
  if (lane == 0) sh.bound_key = kk == k ? bound_of<T>(t) : 0u;  // fewer groups than k: any word may be among the k
}

// 16-byte copy into shared memory in the background of this thread.
__device__ __forceinline__ void copy_async(uint4* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(smem_u32(dst)), "l"(__cvta_generic_to_global(src)) : "memory");
}
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// The row's best k words into sh.top, in order, from its group maxima. `tid` counts the threads of the kWarps warps.
// Begins and ends with a barrier of those. stage: shared memory for kStage vectors (16 bytes each) through which the chosen
// groups are read, all of a stage in flight at once; or null: through registers, kFirst per thread.
constexpr int kStage = 1024;

template <typename T, int kWarps, bool kStaged = false>
__device__ void best_words(Choice<kWarps>& sh, const uint32_t* group_key, const Row<T>& row, const Groups gr, int k,
                           int tid, uint4* stage = nullptr) {
  constexpr int VE = Elem<T>::kVec;
  constexpr uint32_t kHigh = Elem<T>::kKeyBits == 32 ? ~0u : ~0u << (32 - Elem<T>::kKeyBits);
  constexpr int kCand = Choice<kWarps>::kCand;
  constexpr int kDeep = 4;  // 32-vector chunks a warp has in flight (in the ordered path: 8 bits of `equal` each)
  constexpr int kFirst = kWarps > 1 ? 6 : 4;  // the same in the usual path
  const int lane = tid & 31, warp = tid >> 5;
  const int kk = min(k, gr.count);
  if (tid == 0) sh.count = sh.hits = 0;
  if (tid < 32) choose_groups<T>(sh, group_key, gr.count, kk, k);
  sync_warps<kWarps>();
  uint32_t bound = sh.bound_key;
  const int nv = kk << gr.vec_shift;  // vectors of the chosen groups, in their order
  auto vector_at = [&](int t) {  // where the t-th of them starts
    const int64_t g = sh.sel[t >> gr.vec_shift];
    return ((g << gr.vec_shift) + (t & ((1 << gr.vec_shift) - 1))) * VE;
  };
  auto push = [&](uint64_t cd) {
    const int at = atomicAdd(&sh.count, 1);
    if (at < kCand) sh.cand[at] = cd;
  };
  // Masks tie very many words at one value. If k of the row's first 4 k words equal the bound, the bound can be raised to the
  // next key: the words above it are all in the chosen groups, and those equal words that are needed are among
  // these first words. (The same holds for the first words of -inf where the bound was raised above that.) A row of 151936
  // fp32 words of which a mask leaves five, 8 alternatives: 10.7 us, in the order below 6.6 us more.
  constexpr uint32_t kNextKey = ~kHigh + 1u;
  auto first_words = [&](uint32_t value, auto&& use) {
#pragma unroll 1
    for (int i = tid; i < 4 * k && row.lead + i < row.end; i += kWarps * 32) {
      const uint32_t key = order_key(Elem<T>::get(row.base[row.lead + i]));
      if ((key & kHigh) == value) use(key, i);
    }
  };
  auto fill_up = [&](int& have) {
    if (have >= k) return;  // else the bound was raised, and the missing words are among the first 4 k: those of the value below it
    sync_warps<kWarps>();
    first_words(bound - kNextKey, [&](uint32_t key, int i) { push(cand_of(key, i)); });
    sync_warps<kWarps>();
    have = sh.count;
  };
#pragma unroll 1
  while (true) {
    // The vectors with a word not below the bound are set down in shared memory, and then every thread looks at
    // one word of them. That is all unless very many words equal the bound.
    const float bound_value = bound == 0u ? -INFINITY : key_value(bound);
    auto look = [&](int t, uint4 v) {
      if (!(Elem<T>::vec_max(v) < bound_value)) {  // (also a NaN)
        const int at = atomicAdd(&sh.hits, 1);
        if (at < Choice<kWarps>::kHits) {
          sh.hit_vec[at] = v;
          sh.hit_at[at] = static_cast<int>(vector_at(t) / VE);
        }
      }
    };
    if constexpr (kStaged) {
#pragma unroll 1
      for (int t0 = 0; t0 < nv; t0 += kStage) {
        const int m = min(nv - t0, kStage);
        if (kWarps == 1 && gr.vec_shift >= 5 && (1 << gr.vec_shift) <= kStage) {  // whole groups of whole warp loads
          const int per = 1 << gr.vec_shift;
#pragma unroll 1
          for (int i = 0; i < m; i += per) {
            const int64_t u = vector_at(t0 + i);
            const T* src = row.base + u + tid * VE;
            uint4* dst = stage + i + tid;
            if (row.inside(u, u + static_cast<int64_t>(per) * VE)) {
#pragma unroll 2
              for (int c = 0; c < per; c += 32) copy_async(dst + c, src + c * VE);
            } else {
#pragma unroll 1
              for (int c = 0; c < per; c += 32) dst[c] = row.edge(u + static_cast<int64_t>(c + tid) * VE);
            }
          }
        } else {
#pragma unroll 4
          for (int i = tid; i < m; i += kWarps * 32) {
            const int64_t u = vector_at(t0 + i);
            if (row.inside(u, u + VE))
              copy_async(stage + i, row.base + u);
            else
              stage[i] = row.edge(u);
          }
        }
        copy_wait();  // every thread reads back what it copied
#pragma unroll 4
        for (int i = tid; i < m; i += kWarps * 32) look(t0 + i, stage[i]);
      }
    } else
#pragma unroll 1
    for (int t0 = tid; t0 < nv; t0 += kWarps * kFirst * 32) {
      uint4 v[kFirst];
#pragma unroll
      for (int i = 0; i < kFirst; ++i)
        if (t0 + i * kWarps * 32 < nv) v[i] = row.edge(vector_at(t0 + i * kWarps * 32));
#pragma unroll
      for (int i = 0; i < kFirst; ++i) {
        const int t = t0 + i * kWarps * 32;
        if (t < nv) look(t, v[i]);
      }
    }
    sync_warps<kWarps>();
    if (sh.hits <= Choice<kWarps>::kHits) {
      const int words = sh.hits * VE;
#pragma unroll 1
      for (int e = tid; e < words; e += kWarps * 32) {
        const int64_t u = static_cast<int64_t>(sh.hit_at[e / VE]) * VE + e % VE;
        const uint32_t key = order_key(Elem<T>::get(reinterpret_cast<const T*>(sh.hit_vec)[e]));
        if ((key & kHigh) >= bound && row.inside(u, u + 1)) push(cand_of(key, static_cast<int>(u - row.lead)));
      }
      sync_warps<kWarps>();
      int have = sh.count;
      fill_up(have);
      if (have >= k && have <= kCand) {
        rank_all(sh, have, k, tid);
        sync_warps<kWarps>();
        return;
      }
    }
    if (bound >= (kInfKey & kHigh)) break;
    int equal = 0;
    first_words(bound, [&](uint32_t, int) { ++equal; });
    if constexpr (kWarps > 1)
      equal = __syncthreads_count(equal);  // (at most 4 k threads have a word each)
    else
      equal = __reduce_add_sync(~0u, equal);
    if (equal < k) break;
    bound += kNextKey;
    sync_warps<kWarps>();
    if (tid == 0) sh.count = sh.hits = 0;
    sync_warps<kWarps>();
  }
  // Otherwise in order: the words above the bound, and of those equal to it only the first k.
  sync_warps<kWarps>();
  if (tid == 0) sh.count = 0;
  sync_warps<kWarps>();
  int equal_before = 0;
#pragma unroll 1
  for (int t0 = 0; t0 < nv; t0 += kWarps * kDeep * 32) {
    const int tw = t0 + warp * kDeep * 32 + lane;
    float top[kDeep];
#pragma unroll
    for (int i = 0; i < kDeep; ++i) top[i] = tw + i * 32 < nv ? Elem<T>::vec_max(row.edge(vector_at(tw + i * 32))) : -INFINITY;
    uint32_t hits = 0u;  // bit i: this lane's vector of chunk i holds a word not below the bound
#pragma unroll
    for (int i = 0; i < kDeep; ++i) hits |= (tw + i * 32 < nv && (order_key(top[i]) & kHigh) >= bound) << i;
    const uint32_t any = __reduce_or_sync(~0u, hits);
    uint32_t equal = 0u;  // bit 8 i + q: word q of that vector equals the bound
#pragma unroll 1
    for (int i = 0; i < kDeep; ++i) {
      if (!((hits >> i) & 1u)) continue;
      const int64_t u = vector_at(tw + i * 32);
#pragma unroll 1
      for (int q = 0; q < VE; ++q) {
        if (!row.inside(u + q, u + q + 1)) continue;
        const uint32_t key = order_key(Elem<T>::get(row.base[u + q]));
        if ((key & kHigh) > bound) push(cand_of(key, static_cast<int>(u + q - row.lead)));
        equal |= static_cast<uint32_t>((key & kHigh) == bound) << (8 * i + q);
      }
    }
    __syncwarp();
    const int equals = __reduce_add_sync(~0u, __popc(equal));
    if (lane == 0) sh.equal[warp] = equals;
    sync_warps<kWarps>();
    int rank = equal_before;  // of this warp's first equal word among all of them
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      rank += w < warp ? sh.equal[w] : 0;
      equal_before += sh.equal[w];
    }
    if (equals > 0 && rank < k) {
      const uint64_t base = static_cast<uint64_t>((bound & 0x80000000u) ? bound : bound | ~kHigh) << 32;  // the full key
#pragma unroll 1
      for (int i = 0; i < kDeep; ++i) {
        if (!((any >> i) & 1u)) continue;
        uint32_t bits = (equal >> (8 * i)) & 0xffu;
        int pre = __popc(bits);  // inclusive prefix over the lanes
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int o = __shfl_up_sync(~0u, pre, off);
          if (lane >= off) pre += o;
        }
        int r = rank + pre - __popc(bits);
        rank += __shfl_sync(~0u, pre, 31);
        if (bits == 0u) continue;
        const int64_t v0 = vector_at(tw + i * 32) - row.lead;
        for (; bits != 0u && r < k; bits &= bits - 1u, ++r)
          push(base | (0xffffffffu - static_cast<uint32_t>(v0 + __ffs(static_cast<int>(bits)) - 1)));
      }
    }
    sync_warps<kWarps>();
  }
  int have = sh.count;
  fill_up(have);
  if (have <= kCand) {
    rank_all(sh, have, k, tid);
    sync_warps<kWarps>();
    return;
  }
  // More candidates than fit (a row in rising order, say): some words at a time, under a rising bound.
  constexpr int kStep = (kCand - HYLO_TOP_MAX) / (32 * VE) * 32;  // vectors
  uint64_t least = static_cast<uint64_t>(bound) << 32;  // candidates are not below it
  int best = 0;
  for (int t0 = 0; t0 < nv; t0 += kStep) {
    sync_warps<kWarps>();
    if (tid == 0) sh.count = best;
    for (int i = tid; i < best; i += kWarps * 32) sh.cand[i] = sh.top[i];
    sync_warps<kWarps>();
    for (int t = t0 + tid; t < min(nv, t0 + kStep); t += kWarps * 32) {
      const int64_t u = vector_at(t);
#pragma unroll 1
      for (int q = 0; q < VE; ++q) {
        if (!row.inside(u + q, u + q + 1)) continue;
        const uint64_t cd = cand_of(order_key(Elem<T>::get(row.base[u + q])), static_cast<int>(u + q - row.lead));
        if (cd >= least) sh.cand[atomicAdd(&sh.count, 1)] = cd;
      }
    }
    sync_warps<kWarps>();
    const int all = sh.count;
    rank_all(sh, all, k, tid);
    best = min(k, all);
    sync_warps<kWarps>();
    if (best == k) least = sh.top[k - 1];
  }
  sync_warps<kWarps>();
}

// Streams blocks blk0 .. blk1 of a row through warps 0 .. kWarps - 1: the lane's sums, and (kTop) the groups' maxima. A
// block is one vector of each lane of a warp.
template <typename T, int kWarps, bool kTop>
__device__ __forceinline__ Sums stream_row(const Row<T>& row, int blk0, int blk1, int vec_shift, float c, int warp, int lane,
                                           uint32_t* group_key) {
  constexpr int VE = Elem<T>::kVec;
  constexpr int kBlock = 32 * VE;  // words of a block
  constexpr int kBatch = 4;        // blocks a warp has in flight
  const int group_blocks = vec_shift > 5 ? 1 << (vec_shift - 5) : 1;
  const int run = max(kBatch, group_blocks);  // consecutive blocks of one warp
  Sums r{-INFINITY, 0.f, 0.f};
  bool masked = false;
  for (int b0 = blk0 + warp * run; b0 < blk1; b0 += kWarps * run) {
    const int b1 = min(blk1, b0 + run);
    float gm = -INFINITY;
    for (int b = b0; b < b1; b += kBatch) {
      const int64_t u0 = static_cast<int64_t>(b) * kBlock + lane * VE;
      uint4 v[kBatch];
      if (row.inside(static_cast<int64_t>(b) * kBlock, static_cast<int64_t>(b + kBatch) * kBlock)) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) v[i] = row.whole(u0 + i * kBlock);
      } else {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) v[i] = row.edge(u0 + i * kBlock);
      }
      float mx = r.mx;
      float bm[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        bm[i] = Elem<T>::vec_max(v[i]);
        mx = max_nan(mx, bm[i]);
      }
      if (kTop) {
        if (vec_shift == 6) {  // a group is two blocks; lane i stores pair i's
          const float m0 = warp_max_nan(max_nan(bm[0], bm[1])), m1 = warp_max_nan(max_nan(bm[2], bm[3]));
          if (lane < 2 && b + 2 * lane < b1) group_key[(b >> 1) + lane] = order_key(lane == 0 ? m0 : m1);
        } else if (vec_shift == 5) {  // a group is a block; lane i stores block i's
          float mine = -INFINITY;
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            const float m = warp_max_nan(bm[i]);
            mine = lane == i ? m : mine;
          }
          if (lane < kBatch && b + lane < b1) group_key[b + lane] = order_key(mine);
        } else if (vec_shift < 5) {  // several groups per block
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            float m = bm[i];
            for (int off = 1; off < (1 << vec_shift); off <<= 1) m = max_nan(m, __shfl_xor_sync(~0u, m, off));
            if (b + i < b1 && (lane & ((1 << vec_shift) - 1)) == 0)
              group_key[((b + i) << (5 - vec_shift)) + (lane >> vec_shift)] = order_key(m);
          }
        } else {  // a group is a batch, or a run of batches, of this warp
          gm = max_nan(gm, max_nan(max_nan(bm[0], bm[1]), max_nan(bm[2], bm[3])));
          if (((b + kBatch) & (group_blocks - 1)) == 0 || b + kBatch >= b1) {
            const float m = warp_max_nan(gm);
            if (lane == 0) group_key[b >> (vec_shift - 5)] = order_key(m);
            gm = -INFINITY;
          }
        }
      }
      if (mx != r.mx) rebase(r, mx, c);
      const float m0 = base_of(mx);
      float2 s = make_float2(0.f, 0.f), a = s;
      // The floor costs an operation per word in the busiest pipe, so it is left out until a masked word shows.
      if (!masked) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) fold<T, false>(v[i], m0, c, s, a);
        masked = isnan(a.x + a.y);
      }
      if (masked) {
        s = a = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) fold<T, true>(v[i], m0, c, s, a);
      }
      r.s += s.x + s.y;
      r.a += a.x + a.y;
    }
  }
  return join_lanes(r, 32, c);
}

// The logit of token t, if it is one.
template <typename T>
__device__ __forceinline__ float token_logit(const TokenRows& in, const Row<T>& row, int64_t t) {
  return t >= 0 && t < in.V ? Elem<T>::get(row.base[t + row.lead]) : 0.f;
}

// Row n's results but the alternatives, for its token t of logit zt; one thread.
__device__ __forceinline__ void write_row(const TokenRows& in, const TokenOut& out, int64_t n, int64_t t, float zt, const Sums& r,
                                          float log_s) {
  float lp = 0.f;
  if (t >= in.V)
    lp = __uint_as_float(0x7fffffffu);
  else if (t >= 0)
    lp = r.mx == -INFINITY ? -INFINITY : (zt - r.mx) * in.inv_tau - log_s;
  out.logp[n] = lp;
  if (out.entropy) out.entropy[n] = r.mx == -INFINITY ? 0.f : log_s - kLn2F * r.a / r.s;
  if (out.lse) out.lse[n] = r.mx == -INFINITY ? -INFINITY : r.mx * in.inv_tau + log_s;
  if (out.stats) out.stats[n] = make_float2(r.mx, log_s);
}

// Row n's alternatives from top[0..k); thread tid of `threads`.
__device__ __forceinline__ void write_top(const TokenRows& in, const TokenOut& out, int64_t n, const uint64_t* top,
                                          const Sums& r, float log_s, int tid, int threads) {
  for (int i = tid; i < out.k; i += threads) {
    const float z = key_value(static_cast<uint32_t>(top[i] >> 32));
    out.top_logp[n * out.k + i] = r.mx == -INFINITY ? -INFINITY : (z - r.mx) * in.inv_tau - log_s;
    out.top_ids[n * out.k + i] = cand_index(top[i]);
  }
}

template <typename T>
__device__ __forceinline__ Groups groups_of(const Row<T>& row, int vec_shift) {
  const int64_t vectors = (row.end + Elem<T>::kVec - 1) / Elem<T>::kVec;
  return Groups{vec_shift, static_cast<int>((vectors + (int64_t(1) << vec_shift) - 1) >> vec_shift)};
}

template <typename T>
__device__ __forceinline__ int blocks_of(const Row<T>& row) {
  return static_cast<int>((row.end + 32 * Elem<T>::kVec - 1) / (32 * Elem<T>::kVec));
}

template <int kWarps, bool kTop>
struct Shared {
  Sums warp_sums[kWarps];
  Sums cta_sums[kMaxSplit];                   // in the first CTA of a cluster: every CTA's
  alignas(16) uint32_t group_key[kTop ? kMaxGroups : 1];  // in the first CTA: the whole row's
  Choice<kTop ? kWarps : 1> choice;
};

// A cluster of S CTAs takes a row at a time, each CTA `span` consecutive blocks of it (row_split.h); the first CTA joins the
// results.
template <typename T, int kWarps, bool kTop>
__global__ void __launch_bounds__(kWarps * 32, 32 / kWarps)
token_logprobs_kernel(const TokenRows in, const TokenOut out, int span, int vec_shift) {
  __shared__ Shared<kWarps, kTop> sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t S = 1, q = 0;
  if (kWarps > 1) {
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(S));
    q = cluster_ctarank();
  }
  // Between an arrive and its wait the first CTA's shared memory is not written by the others: it may not
  // have started yet, or still be reading the previous row's.
  if (S > 1) cluster_arrive();

  for (int64_t n = blockIdx.x / S; n < in.N; n += gridDim.x / S) {
    const Row<T> row(in.z, n * in.ld, in.V);
    int64_t token = -1;  // thread 0's, early: its logit waits for it
    float zt = 0.f;
    if (tid == 0 && q == 0) {
      token = in.tokens[n];
      zt = token_logit(in, row, token);
    }
    const RowPart part = row_part(blocks_of(row), span, static_cast<int>(q), vec_shift);
    Sums r = stream_row<T, kWarps, kTop>(row, part.blk0, part.blk1, vec_shift, in.c, warp, lane, sh.group_key);
    if (kWarps > 1) {
      if (lane == 0) sh.warp_sums[warp] = r;
      __syncthreads();
      // every warp the same; lanes w, w + kWarps, ... take the same sums, so that all lanes end with the total
      r = join_lanes(sh.warp_sums[lane & (kWarps - 1)], kWarps, in.c);
    }
    if (S > 1) {  // the first CTA of the cluster joins the others' sums and maxima
      cluster_wait();
      if (tid == 0) {
        const uint32_t to = mapa_shared(smem_u32(&sh.cta_sums[q]), 0);
        st_cluster_u32(to, __float_as_uint(r.mx));
        st_cluster_u32(to + 4, __float_as_uint(r.s));
        st_cluster_u32(to + 8, __float_as_uint(r.a));
      }
      if (kTop && q != 0) {
        for (int g = part.g0 + tid; g < part.g1; g += kWarps * 32)
          st_cluster_u32(mapa_shared(smem_u32(&sh.group_key[g]), 0), sh.group_key[g]);
      }
      cluster_sync_all();
      if (q == 0) r = join_lanes(sh.cta_sums[lane & (S - 1)], static_cast<int>(S), in.c);
    }
    if (q == 0) {
      const float log_s = logf(r.s);
      if (tid == 0) write_row(in, out, n, token, zt, r, log_s);
      if constexpr (kTop) {
        __syncthreads();  // (one warp: its group maxima)
        best_words<T>(sh.choice, sh.group_key, row, groups_of(row, vec_shift), out.k, tid);
        write_top(in, out, n, sh.choice.top, r, log_s, tid, kWarps * 32);
      }
    }
    __syncthreads();  // this CTA's shared memory is free for the next row
    if (S > 1) cluster_arrive();
  }
  if (S > 1) cluster_wait();
}

constexpr int kStreamWarps = 8;  // warps of a CTA that shares a row

// Many whole rows with alternatives: eight warps stream row after row and never wait for a selection; a ninth warp joins
// each row's sums and chooses its alternatives while the next row streams. (8192 x 128256, 16 alternatives: with the eight
// warps choosing between rows, 489 us; so, 382 us.)
constexpr int kRowWarps = 8;
constexpr int kRowThreads = 32 * (kRowWarps + 1);
constexpr int kRowBlocks = 4;  // thread blocks per SM

__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" :: "r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void bar_arrive(int id, int threads) {
  asm volatile("bar.arrive %0, %1;" :: "r"(id), "r"(threads) : "memory");
}

template <typename T>
__global__ void __launch_bounds__(kRowThreads, kRowBlocks)
token_logprobs_rows_kernel(const TokenRows in, const TokenOut out, int vec_shift) {
  __shared__ Sums warp_sums[2][kRowWarps];
  __shared__ uint32_t group_key[2][kMaxGroups];
  __shared__ Choice<1> choice;
  __shared__ uint4 stage[kStage];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // Barriers 1, 2: buffer 0, 1 full; 3, 4: free again.
  int buf = 0;
  if (warp < kRowWarps) {
    bool first[2] = {true, true};
    for (int64_t n = blockIdx.x; n < in.N; n += gridDim.x, buf ^= 1) {
      const Row<T> row(in.z, n * in.ld, in.V);
      if (!(buf == 0 ? first[0] : first[1])) bar_sync(3 + buf, kRowThreads);
      (buf == 0 ? first[0] : first[1]) = false;
      const Sums r = stream_row<T, kRowWarps, true>(row, 0, blocks_of(row), vec_shift, in.c, warp, lane, group_key[buf]);
      if (lane == 0) warp_sums[buf][warp] = r;
      __threadfence_block();
      bar_arrive(1 + buf, kRowThreads);
    }
  } else {
    // A row's token is loaded two rows ahead and its logit one, so that neither load is waited for.
    const int64_t stride = gridDim.x;
    int64_t n0 = blockIdx.x, token = n0 < in.N ? in.tokens[n0] : -1, token1 = n0 + stride < in.N ? in.tokens[n0 + stride] : -1;
    float zt = n0 < in.N ? token_logit(in, Row<T>(in.z, n0 * in.ld, in.V), token) : 0.f;
    for (int64_t n = n0; n < in.N; n += stride, buf ^= 1) {
      const Row<T> row(in.z, n * in.ld, in.V);
      const int64_t token2 = n + 2 * stride < in.N ? in.tokens[n + 2 * stride] : -1;
      const float zt1 = n + stride < in.N ? token_logit(in, Row<T>(in.z, (n + stride) * in.ld, in.V), token1) : 0.f;
      bar_sync(1 + buf, kRowThreads);
      const Sums r = join_lanes(warp_sums[buf][lane & (kRowWarps - 1)], kRowWarps, in.c);
      const float log_s = logf(r.s);
      if (lane == 0) write_row(in, out, n, token, zt, r, log_s);
      best_words<T, 1, true>(choice, group_key[buf], row, groups_of(row, vec_shift), out.k, lane, stage);
      write_top(in, out, n, choice.top, r, log_s, lane, 32);
      token = token1, token1 = token2, zt = zt1;
      __syncwarp();
      if (n + 2 * static_cast<int64_t>(gridDim.x) < in.N) bar_arrive(3 + buf, kRowThreads);  // someone waits for it
    }
  }
}

constexpr int kBwdThreads = 256;
constexpr int kBwdVecs = 4;  // vectors a lane has in flight

// A warp takes pieces of 32 * kBwdVecs vectors, rows one after another.
template <typename T>
__global__ void __launch_bounds__(kBwdThreads) token_logprobs_bwd_kernel(const TokenRows in, const TokenGrad g,
                                                                         int pieces) {
  constexpr int VE = Elem<T>::kVec;
  constexpr int64_t kPiece = 32 * kBwdVecs * VE;
  const int lane = threadIdx.x & 31;
  const int64_t total = static_cast<int64_t>(in.N) * pieces, warps = static_cast<int64_t>(gridDim.x) * (kBwdThreads / 32);
  for (int64_t w = static_cast<int64_t>(blockIdx.x) * (kBwdThreads / 32) + (threadIdx.x >> 5); w < total; w += warps) {
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
    uint4 v[kBwdVecs];
    if (row.inside(u0, u0 + kPiece)) {
#pragma unroll
      for (int i = 0; i < kBwdVecs; ++i) v[i] = row.template whole<true>(u0 + (i * 32 + lane) * VE);
    } else {
#pragma unroll
      for (int i = 0; i < kBwdVecs; ++i) v[i] = row.template edge<true>(u0 + (i * 32 + lane) * VE);
    }
    const float2 nm = make_float2(-m0, -m0), c2 = make_float2(in.c, in.c), nl = make_float2(-l2, -l2),
                 A2 = make_float2(A, A), B2 = make_float2(B, B);
#pragma unroll
    for (int i = 0; i < kBwdVecs; ++i) {
      const int64_t u = u0 + (i * 32 + lane) * VE;
      float z[VE];
      Elem<T>::unpack(v[i], z);
#pragma unroll
      for (int j = 0; j < VE / 2; ++j) {
        float2 y = __ffma2_rn(__fadd2_rn(make_float2(z[2 * j], z[2 * j + 1]), nm), c2, nl);
        y.x = max_nan(y.x, kFloor);
        y.y = max_nan(y.y, kFloor);
        const float2 d = __fmul2_rn(make_float2(ex2_approx(y.x), ex2_approx(y.y)), __ffma2_rn(B2, y, A2));
        z[2 * j] = d.x;
        z[2 * j + 1] = d.y;
      }
      if (static_cast<uint64_t>(ut - u) < VE) {  // the row's token is in this vector
#pragma unroll
        for (int j = 0; j < VE; ++j)
          if (u + j == ut) z[j] += hit;
      }
      if (vec && row.inside(u, u + VE)) {
        __stcs(reinterpret_cast<uint4*>(dst + u), Elem<T>::pack(z));
      } else {
#pragma unroll
        for (int j = 0; j < VE; ++j)
          if (row.inside(u + j, u + j + 1)) dst[u + j] = Elem<T>::put(z[j]);
      }
    }
  }
}

// CTAs per row for the clusters of eight-warp CTAs: the power of two with the least
// ceil(rows / clusters at once) * (a CTA's blocks + what a row costs beside its words, in blocks).
int choose_split(int64_t N, int64_t blocks, int row_cost, const TokenOccupancy& occ) {
  int best = 1;
  int64_t best_cost = INT64_MAX;
  for (int S = 1, i = 0; S <= kMaxSplit && (S == 1 || blocks / S >= 32); S *= 2, ++i) {
    if (occ.clusters[i] < 1) continue;
    const int64_t cost = (N + occ.clusters[i] - 1) / occ.clusters[i] * ((blocks + S - 1) / S + row_cost);
    if (cost < best_cost) {
      best_cost = cost;
      best = S;
    }
  }
  return best;
}

cudaLaunchConfig_t split_config(cudaLaunchAttribute* attr, int S, int warps, int64_t rows, cudaStream_t stream) {
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(S);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows * S), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(warps * 32), 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

template <typename T, int kWarps, bool kTop>
cudaError_t launch_split(const TokenRows& in, const TokenOut& out, int S, int64_t at_once, int64_t blocks, int vec_shift,
                         cudaStream_t stream) {
  const int span = row_span(blocks, S, vec_shift);
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = split_config(attr, S, kWarps, in.N < at_once ? in.N : at_once, stream);
  return cudaLaunchKernelEx(&cfg, token_logprobs_kernel<T, kWarps, kTop>, in, out, span, vec_shift);
}

constexpr int kShortRow = 16;  // blocks

// What a row costs beside its words, in blocks of streaming (about 76 clocks each on a busy SM): the joins, and the
// selection of alternatives.
constexpr int kJoinCost = 40, kTopCost = 200;

template <typename T, bool kTop>
cudaError_t launch_fwd(const TokenRows& in, const TokenOut& out, const TokenOccupancy& occ, cudaStream_t stream) {
  constexpr int VE = Elem<T>::kVec;
  const int64_t blocks = (static_cast<int64_t>(in.V) + VE - 1 + 32 * VE - 1) / (32 * VE);
  int vec_shift = 0;  // the smallest groups that fit
  while (((blocks * 32 + (int64_t(1) << vec_shift) - 1) >> vec_shift) > kMaxGroups) ++vec_shift;
  if (blocks <= kShortRow && in.N >= 4 * occ.sms)
    return launch_split<T, 1, kTop>(in, out, 1, 32 * occ.sms, blocks, vec_shift, stream);
  const int S = choose_split(in.N, blocks, kTop ? kTopCost : kJoinCost, occ);
  const int whole = kRowBlocks * occ.sms;  // CTAs at once that take whole rows
  if (kTop && in.N > whole) {
    // whole rows, their alternatives chosen beside the streaming: a row costs its words alone
    int i = 0;
    while ((1 << i) < S) ++i;
    const int64_t split_cost = (in.N + occ.clusters[i] - 1) / occ.clusters[i] * ((blocks + S - 1) / S + kTopCost);
    if ((in.N + whole - 1) / whole * blocks + kTopCost <= split_cost) {
      token_logprobs_rows_kernel<T><<<whole, kRowThreads, 0, stream>>>(in, out, vec_shift);
      return cudaGetLastError();
    }
  }
  int i = 0;
  while ((1 << i) < S) ++i;
  return launch_split<T, kStreamWarps, kTop>(in, out, S, occ.clusters[i], blocks, vec_shift, stream);
}

template <typename T>
cudaError_t launch_bwd(const TokenRows& in, const TokenGrad& g, int sms, cudaStream_t stream) {
  const int64_t piece = 32 * kBwdVecs * Elem<T>::kVec;
  const int64_t pieces = (static_cast<int64_t>(in.V) + Elem<T>::kVec - 1 + piece - 1) / piece;
  const int64_t total = (pieces * in.N + kBwdThreads / 32 - 1) / (kBwdThreads / 32), cap = static_cast<int64_t>(sms) * 64;
  token_logprobs_bwd_kernel<T>
      <<<static_cast<int>(total < cap ? total : cap), kBwdThreads, 0, stream>>>(in, g, static_cast<int>(pieces));
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_fwd_any(const TokenRows& in, const TokenOut& out, const TokenOccupancy& occ, cudaStream_t stream) {
  return out.k > 0 ? launch_fwd<T, true>(in, out, occ, stream) : launch_fwd<T, false>(in, out, occ, stream);
}

template <typename T, bool kTop>
cudaError_t prepare_one(TokenOccupancy* occ) {
  cudaError_t e =
      cudaFuncSetAttribute(token_logprobs_kernel<T, kStreamWarps, kTop>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  for (int S = 1, i = 0; e == cudaSuccess && S <= kMaxSplit; S *= 2, ++i) {
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = split_config(attr, S, kStreamWarps, 1, nullptr);
    int n = 0;
    if ((e = cudaOccupancyMaxActiveClusters(&n, token_logprobs_kernel<T, kStreamWarps, kTop>, &cfg)) != cudaSuccess) break;
    n = n < 4 * occ->sms / S ? n : 4 * occ->sms / S;  // more per SM than the four planned for shares the same memory
    if (n < occ->clusters[i]) occ->clusters[i] = n;
  }
  return e;
}

template <typename T>
cudaError_t prepare(TokenOccupancy* occ) {
  const cudaError_t e = prepare_one<T, true>(occ);
  return e == cudaSuccess ? prepare_one<T, false>(occ) : e;
}

}  // namespace

cudaError_t token_logprobs_prepare(int sms, TokenOccupancy* occ) {
  occ->sms = sms;
  for (int& c : occ->clusters) c = 1 << 30;
  cudaError_t e = prepare<float>(occ);
  if (e == cudaSuccess) e = prepare<__nv_bfloat16>(occ);
  if (e == cudaSuccess) e = prepare<__half>(occ);
  if (e == cudaSuccess && occ->clusters[0] < 1) e = cudaErrorInvalidConfiguration;
  return e;
}

cudaError_t launch_token_logprobs(const TokenRows& in, const TokenOut& out, int dtype, const TokenOccupancy& occ,
                                  cudaStream_t stream) {
  switch (dtype) {
    case HYLO_F32: return launch_fwd_any<float>(in, out, occ, stream);
    case HYLO_BF16: return launch_fwd_any<__nv_bfloat16>(in, out, occ, stream);
    default: return launch_fwd_any<__half>(in, out, occ, stream);
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
