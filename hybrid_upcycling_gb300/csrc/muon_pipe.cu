// The Newton-Schulz steps X <- a X + (b A + c A^2) X, A = X X^T, of a group of matrices, on the tensor cores in one persistent launch.
//
// Three products a step: Gram forms A, Poly B = b A + c A^2, Apply the next X; the last Apply writes the results, or steps
// the parameters. A and B are symmetric, so only their 256 x 256 tiles on and above the diagonal are computed and stored. An
// operand block that lies below it is read as its mirror image: the tensor cores take either order of an operand ("major"), which
// is a bit of the instruction, set for each block. So half of the products of Gram and Poly are saved without a copy of the mirror
// image.
//
// Operands are fp16 scaled by powers of two (bf16 would round eight times coarser for the same time, and a matrix whose singular
// values are at most about 1 needs no more range); sums are fp32. X is kept as two fp16 terms, 22 bits: the products read the
// first one, a X both. So rounding X does not meet the factor a = 3.4 of the small singular values five times over (a matrix of
// low rank and noise: error 2e-2 with one term, 4e-4 with two).
//
// The tensor cores cut every product of a sum off at about 2^-24 of the sum so far, which carries it towards 0 (A of a row of
// 100 000 elements came out 3e-3 too small), so at most kMuonDepth k-blocks are summed there; longer sums go through fp32 numbers in
// the CTA's part of the workspace, rounded to nearest.
//
// Work items are 256 x 256 tiles, taken from a queue in the order step, product, matrix, tile. One
// may start once every earlier item of its matrix is done, which a counter per matrix tells: what it reads is then complete, and
// what it overwrites is no longer read. With several matrices the tail of one's product is filled with the next one's items;
// every item waits for earlier ones only, which running CTAs hold, so the launch cannot deadlock whatever the residency. Where whole
// tiles of a product would leave clusters idle, items are 256 x 128 and take little more than half as long, 296 cycles for a 64-deep
// block, a whole tile's 512 (the tensor cores' rate) to 590. (Eight stages of their size instead of six: the same or slower.)
//
// Long sums of few items of Gram are split among items of their own; their fp32 parts meet in the workspace, and each warp of the
// epilogue that finds all parts of its 32 rows there adds them up in a fixed order.
//
// A CTA pair takes an item: warp 2 of the even CTA fetches it, waits for its matrix and publishes it to both CTAs; warp 0 of each CTA
// loads by TMA; one thread of warp 1 of the even CTA issues the products; eight warps of each CTA take the sums out of TMEM, whose two
// halves alternate. These add X or A and write the next X, A or B, 32 rows and 32 columns at a time, the next ones on their way, with a
// lane to a row and 32 bytes, a whole sector, an access. (With 16 bytes an access and nothing ahead the tiles of Apply took twice as
// long; parts through shared memory by TMA are as fast as this where there is much to do and slower where there is little.)
//
// What bounds it: the tensor cores, at the clock that the power cap leaves. Four 2048 x 8192 matrices 1.38 ms, the tensor pipe 85 %
// active; an item of Gram, K = 8192, 66 200 cycles (65 500 at the tensor cores' rate), one of Apply, K = 2048, 17 800 (16 400), its
// epilogue 11 500 beside the next one's products. One 2048 x 2048: 0.22 ms, each product a chain of queue, copies, products and epilogue.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "muon.h"

namespace hylo {
namespace {

constexpr int kEpiWarps = 8, kEpiWarp0 = 4, kThreads = 32 * (kEpiWarp0 + kEpiWarps);
constexpr int kRegsControl = 96, kRegsEpilogue = 200;  // per thread of warpgroup 0, and of the two of the epilogue
static_assert(128 * kRegsControl + 256 * kRegsEpilogue <= kThreads * 168, "register split");
constexpr int A_BYTES = kBM * kBK * 2;      // 16 KB: this CTA's 128 rows of A
constexpr int STAGE_BYTES = 2 * A_BYTES;    // and 128 rows (columns) of B
constexpr int STAGES = 6;
constexpr int STAGING_BYTES = kEpiWarps * 4096;  // 32 x 32 fp32 numbers a warp
constexpr int kUnits = kMuonLoUnits;        // such parts of a warp's 32 rows x 128 columns
constexpr int kItemDepth = 2;
constexpr int ITEM_OFF = STAGES * STAGE_BYTES + STAGING_BYTES;
constexpr int BAR_OFF = ITEM_OFF + kItemDepth * 32;
constexpr int NBARS = 2 * STAGES + 4 + 2 * kItemDepth + 1;  // full, empty, tfull[2], tempty[2], ifull, iempty, drain
constexpr int SMEM = 1024 + BAR_OFF + NBARS * 8 + 16;
static_assert(SMEM <= 232448, "shared memory budget");
constexpr int kItemConsumers = 2 * (1 + kEpiWarps) + 1;  // producers and epilogue warps of both CTAs, the issuer
constexpr uint32_t kDone = 2 * kEpiWarps;                // what an item adds to its matrix's counter: one per epilogue warp

// fp16 A and B, fp32 sums.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
constexpr uint32_t kAMajor = 1u << 15, kBMajor = 1u << 16;

struct Item {
  int product;  // kMuonGram, kMuonPoly, kMuonApply, or -1: no more
  int step, mat;
  int i, j;     // 256-row tile, 256-column tile
  int half;     // -1, or 0 or 1: the tile's first or second 128 columns only
  unsigned need;  // the matrix's counter once all earlier items are done
  int part;       // of the sum of a split item
};
static_assert(sizeof(Item) == 32, "item size");

template <bool SPLIT>
__device__ __forceinline__ Item item_at(const MuonTable& tab, const MuonPipe& p, unsigned index) {
  unsigned counts[3], per_step = 0;
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    counts[k] = static_cast<unsigned>(p.items[k]) << p.half[k];
    per_step += counts[k];
  }
  Item it{};
  it.step = static_cast<int>(index / per_step);
  if (it.step >= p.steps) {
    it.product = -1;
    return it;
  }
  unsigned r = index - static_cast<unsigned>(it.step) * per_step;
  it.product = r < counts[0] ? kMuonGram : r < counts[0] + counts[1] ? kMuonPoly : kMuonApply;
  r -= it.product == kMuonGram ? 0u : it.product == kMuonPoly ? counts[0] : counts[0] + counts[1];
  const int halves = p.half[it.product], t = static_cast<int>(r >> halves);
  it.half = halves ? static_cast<int>(r & 1u) : -1;
  int lo = 0, hi = tab.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tab.t[mid].item0[it.product] <= t)
      lo = mid;
    else
      hi = mid - 1;
  }
  const MuonMat& m = tab.t[lo];
  it.mat = lo;
  int local = t - m.item0[it.product];
  if (it.product == kMuonApply) {
    it.j = local / m.mt;
    it.i = local - it.j * m.mt;
  } else {  // column by column of the upper triangle: j (j + 1) / 2 + i
    if (SPLIT && it.product == kMuonGram && m.splits > 1) {
      it.part = local % m.splits;
      local /= m.splits;
    }
    int j = static_cast<int>((sqrtf(8.f * static_cast<float>(local) + 1.f) - 1.f) * 0.5f);
    while (j * (j + 1) / 2 > local) --j;
    while ((j + 1) * (j + 2) / 2 <= local) ++j;
    it.j = j;
    it.i = local - j * (j + 1) / 2;
  }
  const unsigned sym = static_cast<unsigned>(m.mt * (m.mt + 1) / 2), poly = sym << p.half[1];
  const unsigned gram = (SPLIT ? sym * static_cast<unsigned>(m.splits) : sym) << p.half[0];
  const unsigned all = gram + poly + (static_cast<unsigned>(m.mt * m.nt) << p.half[2]);
  it.need = kDone * (static_cast<unsigned>(it.step) * all + (it.product == kMuonGram ? 0u : it.product == kMuonPoly ? gram : gram + poly));
  return it;
}

// The k-blocks of an item: [first, end).
struct Range {
  int first, end;
};
template <bool SPLIT>
__device__ __forceinline__ Range kblocks(const MuonMat& m, const Item& it) {
  if (it.product != kMuonGram) return Range{0, m.km};
  if (!SPLIT || m.splits == 1) return Range{0, m.kn};
  const int64_t kn = m.kn;
  return Range{static_cast<int>(kn * it.part / m.splits), static_cast<int>(kn * (it.part + 1) / m.splits)};
}
// Whether k-block kb of an operand of Poly or Apply comes from its mirror image: it lies left of 256-row tile `tile`.
__device__ __forceinline__ bool mirrored(int kb, int tile) { return (kb >> 2) < tile; }

__device__ __forceinline__ uint64_t slice_desc(bool mn, uint32_t base, int k) {
  return mn ? smem_desc_sw128(base + k * 2048, 8192, 1024) : smem_desc_sw128(base + k * 32, 0, 1024);
}

// One lane of a converged warp, the same every time. The compiler knows that code behind it runs in one thread; behind lane == 0 it does
// not, and each operand of the copies and products, which have to be uniform, costs a detour (one 2048 x 2048 matrix 262 us so, 223
// with the chosen lane; a 64-deep block of products of half a tile 546 cycles and 296).
__device__ __forceinline__ bool elect_one() {
  uint32_t is;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(is));
  return is != 0;
}

__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity, unsigned long long limit_ns) {
  const uint32_t a = smem_u32(bar);
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(a, parity)) {
    if (globaltimer_ns() - t0 > limit_ns) return;
  }
}

// Waits for *ctr >= target (acquire); false on abort or time-out.
__device__ __forceinline__ bool wait_count(const unsigned* ctr, unsigned target, volatile int* abort_flag, const WaitCtl& ctl) {
  if (target == 0u || ld_acquire_gpu(ctr) >= target) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    __nanosleep(32);
    if (ld_acquire_gpu(ctr) >= target) return true;
    if ((it & 7u) == 0) {
      if (*abort_flag) return false;
      if (globaltimer_ns() - t0 > ctl.limit_ns) {
        *abort_flag = 1;
        atomicCAS(ctl.status, 0, kDevTimeoutBase + 71);
        return false;
      }
    }
  }
}

// 128 rows (64 unless `both`) from `row` on and 64 columns from 64 kb on of a matrix whose panels have mp rows. mirror: the block is
// stored as its mirror image, 64 rows from 64 kb on and the columns `row`, ..., and arrives in MN-major order.
__device__ __forceinline__ void load_rows(uint8_t* dst, const CUtensorMap* map, uint32_t bar, uint32_t base, int mp, int row, int kb,
                                          bool mirror, bool both) {
  const int at = static_cast<int>(base) + (mirror ? row / 64 * mp + kb * 64 : kb * mp + row), next = mirror ? mp : 64;
  tma_load_2d_pair(dst, map, bar, 0, at);
  if (both) tma_load_2d_pair(dst + 8192, map, bar, 0, at + next);
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_f16x2(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
// 32 bytes, a whole sector, a lane. The load is coherent: the bytes may have been written on another SM.
__device__ __forceinline__ void ld_sector(const void* p, uint32_t* r) {
  asm volatile("ld.relaxed.gpu.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]) : "l"(p) : "memory");
}
__device__ __forceinline__ void st_sector(void* p, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
               :: "l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]) : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}

__device__ __forceinline__ float ld_shared_f32(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}

// Stores where `ok`, as one predicated access: behind a branch goes what is stored too, one element's work after another's (a bf16
// item of a tall matrix 32 800 cycles, so 28 900).
__device__ __forceinline__ void store_if(bool ok, uint16_t* p, uint32_t v) {
  asm volatile("{ .reg .pred q; setp.ne.u32 q, %2, 0; @q st.global.u16 [%0], %1; }"
               :: "l"(p), "h"(static_cast<uint16_t>(v)), "r"(static_cast<uint32_t>(ok)) : "memory");
}
__device__ __forceinline__ void store_if(bool ok, float* p, float v) {
  asm volatile("{ .reg .pred q; setp.ne.u32 q, %2, 0; @q st.global.f32 [%0], %1; }"
               :: "l"(p), "f"(v), "r"(static_cast<uint32_t>(ok)) : "memory");
}
__device__ __forceinline__ void store_if(bool ok, uint16_t* p, uint2 v) {
  asm volatile("{ .reg .pred q; setp.ne.u32 q, %3, 0; @q st.global.v2.b32 [%0], {%1, %2}; }"
               :: "l"(p), "r"(v.x), "r"(v.y), "r"(static_cast<uint32_t>(ok)) : "memory");
}
__device__ __forceinline__ void store_if(bool ok, float* p, const float* v) {
  asm volatile("{ .reg .pred q; setp.ne.u32 q, %5, 0; @q st.global.v4.f32 [%0], {%1, %2, %3, %4}; }"
               :: "l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "r"(static_cast<uint32_t>(ok)) : "memory");
}

// ---- what becomes of O
__device__ __forceinline__ uint32_t mix32(uint32_t x) {  // the finaliser of MurmurHash3
  x = (x ^ (x >> 16)) * 0x85EBCA6Bu;
  x = (x ^ (x >> 13)) * 0xC2B2AE35u;
  return x ^ (x >> 16);
}
// The step's random bits at positions lo0, lo0 + 1, ... (modulo 2^32, fewer than 2^32 of them): a key for lo0's upper 32 bits and one
// for those behind a carry.
struct RandomKeys {
  uint32_t lo0, first, second;
  __device__ __forceinline__ RandomKeys(uint32_t seed, uint64_t pos) : lo0(static_cast<uint32_t>(pos)) {
    const uint32_t hi = static_cast<uint32_t>(pos >> 32);
    first = mix32(seed + 0x9E3779B9u * (hi + 1u));
    second = mix32(seed + 0x9E3779B9u * (hi + 2u));
    asm("" : "+r"(first), "+r"(second));  // once, not for each element
  }
  __device__ __forceinline__ uint32_t at(uint32_t offset) const {  // to which the position's lower 32 bits, up to a carry, are added
    return lo0 + offset + (lo0 + offset < lo0 ? second : first);
  }
};
// bf16 of w, rounded up with the probability of the part cut off, in the upper 16 bits; the lower ones are left over. (No branch: elements
// would wait for one another.)
__device__ __forceinline__ uint32_t round_random(float w, uint32_t key) {
  const uint32_t bits = mix32(key) * 0x9E3779B1u, up = __float_as_uint(w) + (bits >> 16);
  return fabsf(w) < __int_as_float(0x7f800000) ? up : __float_as_uint(w + w);  // NaN becomes the one of arithmetic
}

// How 32 lanes share O's 32 rows from `row` on and 32 columns from `col` on (of X). Each has one row of it in registers. Where X is the
// transpose, the lanes already hold consecutive elements of the result: lane by lane 32 single elements, one below the other.
// Otherwise they change places through shared memory, for vectors of four elements (eight lanes a row, eight rows a lane),
// or, where the rows are not made of those, for single ones as before.
struct Place {
  bool single;
  int n;         // rows that exist
  uint32_t step;  // elements from one of a lane's rows to the next
  int64_t e;     // the lane's first element of the matrix
  __device__ __forceinline__ Place(const MuonMat& m, int row, int col, int lane) {
    single = m.tall || !m.dst_vec;
    const int r = m.tall ? col : single ? row : row + (lane >> 3), c = m.tall ? row + lane : single ? col + lane : col + 4 * (lane & 7);
    n = c >= m.cols || r >= m.rows ? 0 : single ? m.rows - r : (m.rows - r + 3) / 4;
    step = static_cast<uint32_t>(single ? m.cols : 4 * m.cols);
    e = static_cast<int64_t>(r) * m.cols + c;
  }
};
template <int OUT>
constexpr bool kStep = OUT == kMuonParamF32 || OUT == kMuonParamBf16 || OUT == kMuonParamMaster;
template <int OUT>
using Stored = typename std::conditional<OUT == kMuonParamBf16, uint16_t, float>::type;  // of a parameter's value before the step
template <int OUT>
__device__ __forceinline__ const Stored<OUT>* old_values(const MuonMat& m) {
  return static_cast<const Stored<OUT>*>(OUT == kMuonParamMaster ? m.master : m.dst);
}

// Asks for the old values of 32 rows and 32 `units` columns. (Without this, with a branch around each element's step and a hash more for it
// an item of the last product took 58 000 cycles in bf16 and 34 000 with masters; now 23 500 and 20 000, beside 15 000 to 19 000 for the
// products.)
template <int OUT>
__device__ __forceinline__ void prefetch_old(const MuonMat& m, int row, int col, int units, int lane) {
  constexpr int LINE = 128 / sizeof(Stored<OUT>);
  const Stored<OUT>* old = old_values<OUT>(m);
  const int c1 = min(m.cols, m.tall ? row + 32 : col + units * 32);
  for (int r = (m.tall ? col : row) + lane; r < min(m.rows, m.tall ? col + units * 32 : row + 32); r += 32) {
    for (int c = m.tall ? row : col; c < c1; c += LINE)
      asm volatile("prefetch.global.L2 [%0];" :: "l"(old + static_cast<int64_t>(r) * m.cols + c));
  }
}

// The old values of a lane's elements, as they lie in memory: 32 words, of vectors of bf16 two elements each. (No test around more than
// an access, here and below: what depends on a load would wait for it there, one row after another.)
template <int OUT>
__device__ __forceinline__ void load_old(const MuonMat& m, const Place& at, uint32_t (&w)[32]) {
  const Stored<OUT>* old = old_values<OUT>(m) + at.e;
#pragma unroll
  for (int j = 0; j < 32; ++j) w[j] = 0u;
  if (at.single) {
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      if (j < at.n) {
        if constexpr (OUT == kMuonParamBf16)
          w[j] = old[static_cast<uint32_t>(j) * at.step];
        else
          w[j] = __float_as_uint(old[static_cast<uint32_t>(j) * at.step]);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j < at.n) {
        if constexpr (OUT == kMuonParamBf16) {
          const uint2 v = *reinterpret_cast<const uint2*>(old + static_cast<uint32_t>(j) * at.step);
          w[2 * j] = v.x, w[2 * j + 1] = v.y;
        } else {
          const uint4 v = *reinterpret_cast<const uint4*>(old + static_cast<uint32_t>(j) * at.step);
          w[4 * j] = v.x, w[4 * j + 1] = v.y, w[4 * j + 2] = v.z, w[4 * j + 3] = v.w;
        }
      }
    }
  }
}

template <int OUT>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) { return OUT == kMuonOutF16 ? pack_f16x2(lo, hi) : pack_bf16x2(lo, hi); }

template <int OUT>
__device__ __forceinline__ void finish_part(const MuonMat& m, uint32_t seed, const Place& at, int lane, uint32_t staging,
                                            const uint32_t (&w)[32], float (&o)[32]) {
  const RandomKeys keys(seed, m.pos + static_cast<uint64_t>(at.e));
  float* f = (OUT == kMuonParamF32 ? static_cast<float*>(m.dst) : m.master) + at.e;  // written unless the results have 16 bits
  uint16_t* d = static_cast<uint16_t*>(m.dst) + at.e;                                // written unless OUT is kMuonParamF32
  if (!m.tall) {  // rows of 32 fp32 numbers, 16-byte chunks swizzled by the row
#pragma unroll
    for (int k = 0; k < 8; ++k)
      st_shared_v4(staging + lane * 128 + (k ^ (lane & 7)) * 16, __float_as_uint(o[4 * k]), __float_as_uint(o[4 * k + 1]),
                   __float_as_uint(o[4 * k + 2]), __float_as_uint(o[4 * k + 3]));
    __syncwarp();
  }
  if (at.single) {
    if (!m.tall) {
#pragma unroll
      for (int r = 0; r < 32; ++r) o[r] = ld_shared_f32(staging + r * 128 + ((lane >> 2) ^ (r & 7)) * 16 + (lane & 3) * 4);
    }
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const uint32_t off = static_cast<uint32_t>(j) * at.step;
      if constexpr (kStep<OUT>) o[j] = fmaf(__uint_as_float(OUT == kMuonParamBf16 ? w[j] << 16 : w[j]), m.decay, -m.step * o[j]);
      if constexpr (OUT == kMuonParamF32 || OUT == kMuonParamMaster) store_if(j < at.n, f + off, o[j]);
      if constexpr (OUT == kMuonParamBf16)
        store_if(j < at.n, d + off, round_random(o[j], keys.at(off)) >> 16);
      else if constexpr (OUT != kMuonParamF32)
        store_if(j < at.n, d + off, pack16<OUT>(o[j], 0.f));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int r = 4 * j + (lane >> 3);
      const uint32_t off = static_cast<uint32_t>(j) * at.step;
      const uint4 u = ld_shared_v4(staging + r * 128 + ((lane & 7) ^ (r & 7)) * 16);
      float v[4] = {__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w)};
      if constexpr (kStep<OUT>) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t x = OUT == kMuonParamBf16 ? (i & 1 ? w[2 * j + i / 2] & 0xffff0000u : w[2 * j + i / 2] << 16) : w[4 * j + i];
          v[i] = fmaf(__uint_as_float(x), m.decay, -m.step * v[i]);
        }
      }
      if constexpr (OUT == kMuonParamF32 || OUT == kMuonParamMaster) store_if(j < at.n, f + off, v);
      if constexpr (OUT == kMuonParamBf16) {
        const uint32_t key = keys.at(off);  // of all four: positions of vectors are multiples of four
        store_if(j < at.n, d + off, make_uint2(__byte_perm(round_random(v[0], key), round_random(v[1], key + 1), 0x7632),
                                               __byte_perm(round_random(v[2], key + 2), round_random(v[3], key + 3), 0x7632)));
      } else if constexpr (OUT != kMuonParamF32) {
        store_if(j < at.n, d + off, make_uint2(pack16<OUT>(v[0], v[1]), pack16<OUT>(v[2], v[3])));
      }
    }
  }
  __syncwarp();
}

// SPLIT: the group has split sums. Their code costs other groups up to 4 %.
template <int OUT, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
muon_pipe_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ MuonTable tab, const __grid_constant__ MuonPipe p,
                  const MuonHyper hyper) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* staging_all = smem + STAGES * STAGE_BYTES;
  Item* items = reinterpret_cast<Item*>(smem + ITEM_OFF);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + BAR_OFF);  // used in the even CTA
  uint64_t* empty = full + STAGES;                                // both CTAs
  uint64_t* tfull = empty + STAGES;                               // both CTAs: TMEM half written
  uint64_t* tempty = tfull + 2;                                   // even CTA: half read by both CTAs
  uint64_t* ifull = tempty + 2;                                   // both CTAs: item slot published
  uint64_t* iempty = ifull + kItemDepth;                          // even CTA: item slot released
  uint64_t* drain = iempty + kItemDepth;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    for (int h = 0; h < 2; ++h) {
      mbar_init(tfull + h, 1);
      mbar_init(tempty + h, 2 * kEpiWarps);
    }
    for (int k = 0; k < kItemDepth; ++k) {
      mbar_init(ifull + k, 1);
      mbar_init(iempty + k, kItemConsumers);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (threadIdx.x == 32) prefetch_tmap(&map);
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // barriers of both CTAs initialised before any cross-CTA signal
  tc_fence_after();
  grid_dep_wait();
  const uint32_t tmem_base = *tmem_slot;

  if (warp < kEpiWarp0) setmaxnreg_dec<kRegsControl>();  // each warpgroup changes its registers at once
  if (warp == 2) {
    // ------------------------------------------------------------------ scheduler (even CTA)
    if (lane == 0 && rank == 0) {
      const uint32_t peer_items = mapa_shared(smem_u32(items), 1), peer_ifull = mapa_shared(smem_u32(ifull), 1);
      for (int k = 0;; ++k) {
        const int slot = k % kItemDepth;
        const uint32_t par = static_cast<uint32_t>(k / kItemDepth) & 1u;
        if (!wait_bounded<true>(iempty + slot, par ^ 1u, abort_flag, p.ctl, 72)) break;
        const Item it = item_at<SPLIT>(tab, p, atomicAdd(p.ctrl, 1u));
        if (it.product >= 0 && !wait_count(p.ctrl + 1 + it.mat, it.need, abort_flag, p.ctl)) break;
        items[slot] = it;
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&it);
        for (int q = 0; q < 8; ++q) st_cluster_u32(peer_items + slot * 32 + q * 4, w[q]);
        mbar_arrive(ifull + slot);
        mbar_arrive_remote(peer_ifull + slot * 8);
        if (it.product < 0) break;
      }
    }
  } else if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer (both CTAs)
    if (elect_one()) {
      int stage = 0;
      uint32_t phase = 0, armed = 0;
      const uint32_t lead_iempty = mapa_shared(smem_u32(iempty), 0), full_lead = mapa_shared(smem_u32(full), 0);
      bool ok = true;
      for (int k = 0; ok; ++k) {
        const int slot = k % kItemDepth;
        const uint32_t par = static_cast<uint32_t>(k / kItemDepth) & 1u;
        if (!wait_bounded<true>(ifull + slot, par, abort_flag, p.ctl, 73)) break;
        const Item it = items[slot];
        if (rank == 0)
          mbar_arrive(iempty + slot);
        else
          mbar_arrive_remote(lead_iempty + slot * 8);
        if (it.product < 0) break;
        fence_proxy_async_global();  // what it reads was stored in other CTAs, or by the kernel before
        const MuonMat& m = tab.t[it.mat];
        const int mp = m.mt * 256, cur = it.step & 1;
        const Range range = kblocks<SPLIT>(m, it);
        const uint32_t abase = it.product == kMuonGram ? m.x[cur] : it.product == kMuonPoly ? m.a : m.b;
        const uint32_t bbase = it.product == kMuonPoly ? m.a : m.x[cur];
        const int pair = static_cast<int>(rank), arow = it.i * 256 + pair * kBM;
        const int brow = it.j * 256 + (it.half < 0 ? pair * kBM : it.half * 128 + pair * 64);
        const uint32_t bytes = it.half < 0 ? 2u * STAGE_BYTES : 2u * (A_BYTES + A_BYTES / 2);  // both CTAs'
        for (int kb = range.first; kb < range.end; ++kb) {
          if (!wait_bounded(empty + stage, phase ^ 1u, abort_flag, p.ctl, 74)) {
            ok = false;
            break;
          }
          uint8_t* sa = smem + stage * STAGE_BYTES;
          const uint32_t fb = full_lead + static_cast<uint32_t>(stage) * 8u;
          if (rank == 0) {
            mbar_arrive_expect_tx(full + stage, bytes);
            armed |= 1u << stage;
          }
          load_rows(sa, &map, fb, abase, mp, arow, kb, it.product != kMuonGram && mirrored(kb, it.i), true);
          // B of Apply is X, 64 of its rows and this CTA's columns, which lie like a mirror image's
          load_rows(sa + A_BYTES, &map, fb, bbase, mp, brow, kb,
                    it.product == kMuonApply || (it.product == kMuonPoly && mirrored(kb, it.j)), it.half < 0);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {  // let every armed load land before the CTA can exit
        for (int s = 0; s < STAGES; ++s)
          if (armed & (1u << s)) drain_wait(full + s, s < stage ? phase : (phase ^ 1u), 100000000ull);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ UMMA issuer (even CTA)
    if (rank == 0 && elect_one()) {
      int stage = 0, h = 0;
      uint32_t phase = 0, uses[2] = {0u, 0u};
      bool ok = true, issued = false;
      for (int k = 0; ok; ++k) {
        const int slot = k % kItemDepth;
        const uint32_t par = static_cast<uint32_t>(k / kItemDepth) & 1u;
        if (!wait_bounded(ifull + slot, par, abort_flag, p.ctl, 75)) {
          ok = false;
          break;
        }
        const Item it = items[slot];
        mbar_arrive(iempty + slot);
        if (it.product < 0) break;
        const Range range = kblocks<SPLIT>(tab.t[it.mat], it);
        const uint32_t idesc0 = idesc_f16_f32(2 * kBM, it.half < 0 ? 256 : 128);
        for (int from = range.first; ok && from < range.end; from += kMuonDepth) {
          if (!wait_bounded(tempty + h, (uses[h] & 1u) ^ 1u, abort_flag, p.ctl, 76)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem_base + static_cast<uint32_t>(h * 256);
          for (int kb = from; kb < min(range.end, from + kMuonDepth); ++kb) {
            if (!wait_bounded(full + stage, phase, abort_flag, p.ctl, 77)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t sa = smem_u32(smem + stage * STAGE_BYTES), sb = sa + A_BYTES;
            const bool amn = it.product != kMuonGram && mirrored(kb, it.i);
            const bool bmn = it.product == kMuonApply || (it.product == kMuonPoly && mirrored(kb, it.j));
            const uint32_t idesc = idesc0 | (amn ? kAMajor : 0u) | (bmn ? kBMajor : 0u);
            const uint64_t a0 = slice_desc(amn, sa, 0), b0 = slice_desc(bmn, sb, 0);
            const uint32_t astep = amn ? 2048 >> 4 : 32 >> 4, bstep = bmn ? 2048 >> 4 : 32 >> 4;
#pragma unroll
            for (int q = 0; q < kBK / 16; ++q)
              umma_bf16_pair(d, a0 + q * astep, b0 + q * bstep, idesc, (kb > from || q > 0) ? 1u : 0u);
            umma_commit_pair(empty + stage, 0x3);
            issued = true;
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (!ok) break;
          umma_commit_pair(tfull + h, 0x3);
          ++uses[h];
          h ^= 1;
        }
      }
      if (!ok && issued) {
        umma_commit_pair(drain, 0x1);
        drain_wait(drain, 0, 100000000ull);
      }
    }
  } else if (warp >= kEpiWarp0) {
    // ------------------------------------------------------------------ epilogue (both CTAs)
    setmaxnreg_inc<kRegsEpilogue>();
    const int e = warp - kEpiWarp0, q = warp & 3, hc = e >> 2;  // lane quarter, column half
    const uint32_t lead_tempty = mapa_shared(smem_u32(tempty), 0), lead_iempty = mapa_shared(smem_u32(iempty), 0);
    const uint32_t staging = smem_u32(staging_all + e * STAGING_BYTES / kEpiWarps);
    uint32_t uses[2] = {0u, 0u};
    int h = 0;
    bool skip = false;  // a Muon step whose norm is not finite changes nothing
    if (hyper.norm != nullptr) skip = !isfinite(hyper.norm[0]);
    for (int k = 0;; ++k) {
      const int slot = k % kItemDepth;
      const uint32_t par = static_cast<uint32_t>(k / kItemDepth) & 1u;
      bool got = wait_bounded<true>(ifull + slot, par, abort_flag, p.ctl, 78);
      if (!__all_sync(0xffffffffu, got)) break;
      const Item it = items[slot];
      __syncwarp();
      if (lane == 0) {
        if (rank == 0)
          mbar_arrive(iempty + slot);
        else
          mbar_arrive_remote(lead_iempty + slot * 8);
      }
      if (it.product < 0) break;
      const MuonMat& m = tab.t[it.mat];
      const Range range = kblocks<SPLIT>(m, it);
      const int mp = m.mt * 256, nk = range.end - range.first, cur = it.step & 1;
      const bool apply = it.product == kMuonApply, last = apply && it.step + 1 == p.steps;
      const uint32_t out = it.product == kMuonGram ? m.a : it.product == kMuonPoly ? m.b : m.x[cur ^ 1];
      const uint32_t add = it.product == kMuonPoly ? m.a : m.x[cur];
      const int row = it.i * 256 + static_cast<int>(rank) * kBM + q * 32;
      // This warp's columns of the accumulator and of the matrix: 128, or 64 of half a tile.
      const int units = it.half < 0 ? kUnits : kUnits / 2, acc0 = hc * 32 * units;
      const int col0 = it.j * 256 + (it.half < 0 ? 0 : it.half * 128) + acc0;
      // Rows and columns behind the last 64-deep k-block are never read as such: their parts are left out.
      const int wide = (apply ? m.kn : m.km) * 64 - col0;
      int nu = row >= m.km * 64 || wide <= 0 ? 0 : wide >= 32 * units ? units : wide / 32;
      // X's second term, which only the epilogue of the same tile reads again, lies in the order of its lanes.
      const int64_t sector =
          muon_lo_sector(it.j * m.mt + it.i, static_cast<int>(rank), q + (col0 >> 7 & 1) * 4) + (col0 >> 5 & 3) * 64 + lane;
      uint8_t* lo = hyper.ws + static_cast<size_t>(m.lo) * 128 + sector * 32;
      auto part = [&](uint32_t base, int u) {  // this lane's row of part u
        return hyper.ws + (static_cast<size_t>(base) + static_cast<size_t>(col0 / 64 + u / 2) * mp + row + lane) * 128 + (u & 1) * 64;
      };
      uint32_t hi1[16], lo1[16];  // of the next part
      auto read_ahead = [&](int u) {
        if (it.product != kMuonGram && u < nu) {
          const uint8_t* a = part(add, u);
          ld_sector(a, hi1);
          ld_sector(a + 32, hi1 + 8);
          if (apply) {
            ld_sector(lo + u * 2048, lo1);
            ld_sector(lo + u * 2048 + 1024, lo1 + 8);
          }
        }
      };
#pragma unroll
      for (int j = 0; j < 16; ++j) hi1[j] = lo1[j] = 0u;
      read_ahead(0);
      if constexpr (kStep<OUT>)
        if (last && !skip && nu > 0) prefetch_old<OUT>(m, row, col0, nu, lane);
      // Of a long sum all but the last stretch, added up in the workspace: [kUnits][8][32 lanes] of this warp.
      const bool deep = nk > kMuonDepth;
      float4* scratch = nullptr;
      if (deep)
        scratch = reinterpret_cast<float4*>(p.scratch + blockIdx.x * static_cast<size_t>(kMuonScratch) +
                                            static_cast<size_t>(e) * (kMuonScratch / kEpiWarps)) + lane;
      const uint32_t lanes = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
      for (int from = 0; from + kMuonDepth < nk; from += kMuonDepth) {
        got = __all_sync(0xffffffffu, wait_bounded(tfull + h, uses[h] & 1u, abort_flag, p.ctl, 79));
        if (!got) break;
        tc_fence_after();
        for (int c = 0; c < units; ++c) {
          float v[32];
          tmem_ld32(lanes + static_cast<uint32_t>(h * 256 + acc0 + c * 32), v);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float4 x = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
            if (from > 0) {
              const float4 y = scratch[(c * 8 + j) * 32];
              x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
            }
            scratch[(c * 8 + j) * 32] = x;
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(lead_tempty + h * 8);
        ++uses[h];
        h ^= 1;
      }
      if (!got) break;
      got = wait_bounded(tfull + h, uses[h] & 1u, abort_flag, p.ctl, 80);
      if (!__all_sync(0xffffffffu, got)) break;
      tc_fence_after();
      // A part of a split sum goes to the workspace; the warp that comes last adds all parts up, in their order.
      const float4* all = nullptr;  // this lane's place in the first part
      if (SPLIT && it.product == kMuonGram && m.splits > 1 && nu > 0) {
        const int tile = it.j * (it.j + 1) / 2 + it.i;
        uint8_t* at = p.parts + ((static_cast<size_t>(m.part0) + static_cast<size_t>(tile) * m.splits) * 2 + rank) * kMuonScratch +
                      e * (kMuonScratch / kEpiWarps);
        float4* own = reinterpret_cast<float4*>(at + static_cast<size_t>(it.part) * 2 * kMuonScratch) + lane;
        all = reinterpret_cast<const float4*>(at) + lane;
        for (int u = 0; u < nu; ++u) {
          float v[32];
          tmem_ld32(lanes + static_cast<uint32_t>(h * 256 + acc0 + u * 32), v);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float4 x = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
            if (deep) {
              const float4 y = scratch[(u * 8 + j) * 32];
              x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
            }
            own[(u * 8 + j) * 32] = x;
          }
        }
        __syncwarp();
        unsigned done = 0;
        if (lane == 0) {
          __threadfence();  // every lane's stores, ordered before it by the barrier
          done = atomicAdd(p.ctrl + kMuonCtrlWords + (m.split0 + tile) * 16 + rank * kEpiWarps + e, 1u) + 1u;
          __threadfence();
        }
        done = __shfl_sync(0xffffffffu, done, 0);
        __syncwarp();
        if (done % static_cast<unsigned>(m.splits) != 0u) nu = 0;  // others are to come
      }
      const float acc = p.acc[it.step][it.product], fac = p.add[it.step][it.product];
#pragma unroll 1
      for (int u = 0; u < nu; ++u) {
        uint32_t w[16], l[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) w[j] = hi1[j], l[j] = lo1[j];
        read_ahead(u + 1);
        uint32_t old[32];
        if constexpr (kStep<OUT>)
          if (last && !skip) load_old<OUT>(m, Place(m, row, col0 + u * 32, lane), old);
        float v[32];
        if (SPLIT && all != nullptr) {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = 0.f;
          for (int part = 0; part < m.splits; part += 2) {  // two on their way at a time
            const float4* a = all + static_cast<size_t>(part) * 2 * (kMuonScratch / 16);
            const float4* b = part + 1 < m.splits ? a + 2 * (kMuonScratch / 16) : nullptr;
            float4 x[8], y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {  // written on other SMs: not from L1
              x[j] = __ldcg(a + (u * 8 + j) * 32);
              y[j] = b != nullptr ? __ldcg(b + (u * 8 + j) * 32) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              v[4 * j] = v[4 * j] + x[j].x + y[j].x, v[4 * j + 1] = v[4 * j + 1] + x[j].y + y[j].y;
              v[4 * j + 2] = v[4 * j + 2] + x[j].z + y[j].z, v[4 * j + 3] = v[4 * j + 3] + x[j].w + y[j].w;
            }
          }
        } else {
          tmem_ld32(lanes + static_cast<uint32_t>(h * 256 + acc0 + u * 32), v);
          tmem_ld_wait();
          if (deep) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float4 y = scratch[(u * 8 + j) * 32];
              v[4 * j] += y.x, v[4 * j + 1] += y.y, v[4 * j + 2] += y.z, v[4 * j + 3] += y.w;
            }
          }
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) {  // A has nothing added: its w and l are zeros
          const float2 f = unpack_f16x2(w[j]), g = unpack_f16x2(l[j]);
          v[2 * j] = fmaf(f.x + g.x, fac, v[2 * j] * acc);
          v[2 * j + 1] = fmaf(f.y + g.y, fac, v[2 * j + 1] * acc);
          w[j] = pack_f16x2(v[2 * j], v[2 * j + 1]);
        }
        if (last) {
#pragma unroll
          for (int j = 0; j < 16; ++j) {  // O as orthogonalize gives it in fp16, in every type: 1e-4 of its norm beside the products' 1e-3
            const float2 f = unpack_f16x2(w[j]);
            v[2 * j] = f.x * hyper.unscale;
            v[2 * j + 1] = f.y * hyper.unscale;
          }
          if (!skip) finish_part<OUT>(m, hyper.seed, Place(m, row, col0 + u * 32, lane), lane, staging, old, v);
          continue;
        }
        uint8_t* dst = part(out, u);
        st_sector(dst, w);
        st_sector(dst + 32, w + 8);
        if (apply) {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float2 f = unpack_f16x2(w[j]);
            l[j] = pack_f16x2(v[2 * j] - f.x, v[2 * j + 1] - f.y);
          }
          st_sector(lo + u * 2048, l);
          st_sector(lo + u * 2048 + 1024, l + 8);
        }
      }
      tc_fence_before();  // the half is free for the next item but one
      if (!last) fence_proxy_async_global();  // what this lane has stored will be loaded by TMA
      __syncwarp();
      if (lane == 0) {
        mbar_arrive_remote(lead_tempty + h * 8);
        if (!last) red_release_gpu_add(p.ctrl + 1 + it.mat, 1u);  // every lane's stores are ordered before it by the barrier
      }
      ++uses[h];
      h ^= 1;
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // no cross-CTA signal may target a CTA that has exited
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

cudaLaunchConfig_t pipe_config(cudaLaunchAttribute* attr, int clusters, cudaStream_t stream) {
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // see grid_dep_wait()
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * clusters, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cfg;
}

template <bool SPLIT>
const void* kernel_for(int out) {
  switch (out) {
    case kMuonOutBf16: return reinterpret_cast<const void*>(muon_pipe_kernel<kMuonOutBf16, SPLIT>);
    case kMuonOutF16: return reinterpret_cast<const void*>(muon_pipe_kernel<kMuonOutF16, SPLIT>);
    case kMuonParamF32: return reinterpret_cast<const void*>(muon_pipe_kernel<kMuonParamF32, SPLIT>);
    case kMuonParamBf16: return reinterpret_cast<const void*>(muon_pipe_kernel<kMuonParamBf16, SPLIT>);
    default: return reinterpret_cast<const void*>(muon_pipe_kernel<kMuonParamMaster, SPLIT>);
  }
}
const void* kernel_for(int out, bool split) { return split ? kernel_for<true>(out) : kernel_for<false>(out); }

}  // namespace

cudaError_t muon_pipe_prepare(int* max_clusters) {
  *max_clusters = kMaxClusters;
  for (int k = 0; k <= 2 * kMuonParamMaster + 1; ++k) {
    const void* f = kernel_for(k / 2, k % 2 != 0);
    cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = pipe_config(attr, 1, nullptr);
    cfg.numAttrs = 1;  // occupancy: the cluster shape only
    int n = 0;
    if ((e = cudaOccupancyMaxActiveClusters(&n, f, &cfg)) != cudaSuccess) return e;
    if (n < *max_clusters) *max_clusters = n;
  }
  return cudaSuccess;
}

cudaError_t launch_muon_pipe(const CUtensorMap& load, const MuonTable& t, const MuonPipe& p, const MuonHyper& h, int out,
                             bool split, int clusters, cudaStream_t stream) {
  int most = 0;  // items that can run at once
  for (int k = 0; k < 3; ++k) most = p.items[k] << p.half[k] > most ? p.items[k] << p.half[k] : most;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = pipe_config(attr, most < clusters ? most : clusters, stream);
  void* args[] = {const_cast<CUtensorMap*>(&load), const_cast<MuonTable*>(&t), const_cast<MuonPipe*>(&p), const_cast<MuonHyper*>(&h)};
  return cudaLaunchKernelExC(&cfg, kernel_for(out, split), args);
}

}  // namespace hylo
