// The products of the Newton-Schulz steps X <- a X + (b A + c A^2) X, A = X X^T, over a group of matrices, on the tensor cores.
//
// Three launches a step: kMuonGram forms A, kMuonPoly B = b A + c A^2, kMuonApply the next X. A and B are symmetric, so only
// their 256 x 256 tiles on and above the diagonal are computed and stored. An operand block that lies below it is read as its
// mirror image: the tensor cores take either order of an operand ("major"), which is a bit of the instruction, set for each
// block. So half of the products of the first two launches are saved without a copy of the mirror image.
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
// A CTA pair computes 256 x BN tiles one after another: one warp of each CTA loads by TMA, one thread of the even CTA issues the
// products, eight warps of each CTA take the sums out of TMEM, whose two halves alternate.
#include <cuda_fp16.h>

#include "muon.h"

namespace hylo {
namespace {

constexpr int kEpiWarps = 8, kEpiWarp0 = 4, kThreads = 32 * (kEpiWarp0 + kEpiWarps);
constexpr int A_BYTES = kBM * kBK * 2;  // 16 KB: this CTA's 128 rows of A

template <int BN>
struct Cfg {
  static constexpr int HB = BN / 2;                // B rows staged per CTA
  static constexpr int B_BYTES = HB * kBK * 2;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int STAGES = BN == 256 ? 6 : 8;  // 192 KB
  static constexpr int BAR_OFF = STAGES * STAGE_BYTES;
  static constexpr int NBARS = 2 * STAGES + 4 + 1;  // full, empty, tfull[2], tempty[2], drain
  static constexpr int SMEM = 1024 + BAR_OFF + NBARS * 8 + 16;
  static_assert(SMEM <= 232448, "shared memory budget");
};

// fp16 A and B, fp32 sums.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
constexpr uint32_t kAMajor = 1u << 15, kBMajor = 1u << 16;

// A 256 x BN tile of the phase: matrix, 256-row tile, BN-column tile.
struct Tile {
  int mat, i, j;
};

template <int PHASE, int BN>
__device__ __forceinline__ Tile tile_of(const MuonGemmParams& p, int index) {
  const int t = index / (256 / BN), sub = index % (256 / BN);
  int lo = 0, hi = p.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((PHASE == kMuonApply ? p.t[mid].rect0 : p.t[mid].sym0) <= t)
      lo = mid;
    else
      hi = mid - 1;
  }
  const MuonGemmMat& m = p.t[lo];
  Tile r;
  r.mat = lo;
  int big;  // 256-column tile
  if (PHASE == kMuonApply) {
    const int local = t - m.rect0;
    big = local / m.mt;
    r.i = local - big * m.mt;
  } else {  // column by column of the upper triangle: local = big (big + 1) / 2 + i
    const int local = t - m.sym0;
    big = static_cast<int>((sqrtf(8.f * static_cast<float>(local) + 1.f) - 1.f) * 0.5f);
    while (big * (big + 1) / 2 > local) --big;
    while ((big + 1) * (big + 2) / 2 <= local) ++big;
    r.i = local - big * (big + 1) / 2;
  }
  r.j = big * (256 / BN) + sub;
  return r;
}

__device__ __forceinline__ uint64_t slice_desc(bool mn, uint32_t base, int k) {
  return mn ? smem_desc_sw128(base + k * 2048, 8192, 1024) : smem_desc_sw128(base + k * 32, 0, 1024);
}

__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity, unsigned long long limit_ns) {
  const uint32_t a = smem_u32(bar);
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(a, parity)) {
    if (globaltimer_ns() - t0 > limit_ns) return;
  }
}

// `rows` (64 or 128) rows from `row` on and 64 columns from 64 kb on of a symmetric matrix, or of X (`mirror` false).
// mirror: the block is stored as its mirror image, columns of 64 kb .. rows, which arrives in MN-major order.
template <int ROWS>
__device__ __forceinline__ void load_rows(uint8_t* dst, const CUtensorMap* map, uint32_t bar, uint32_t base, int mp, int row, int kb, bool mirror) {
#pragma unroll
  for (int h = 0; h < ROWS / 64; ++h) {
    const int r = mirror ? static_cast<int>(base) + (row / 64 + h) * mp + kb * 64 : static_cast<int>(base) + kb * mp + row + h * 64;
    tma_load_2d_pair(dst + h * 8192, map, bar, 0, r);
  }
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_f16x2(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }

template <int PHASE, int BN>
__global__ void __launch_bounds__(kThreads, 1)
muon_gemm_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ MuonGemmParams p) {
  using C = Cfg<BN>;
  constexpr int STAGES = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);  // used in the even CTA
  uint64_t* empty = full + STAGES;                                   // both CTAs
  uint64_t* tfull = empty + STAGES;                                  // both CTAs: TMEM half written
  uint64_t* tempty = tfull + 2;                                      // even CTA: half read by both CTAs
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1, tiles = p.tiles * (256 / BN);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    for (int h = 0; h < 2; ++h) {
      mbar_init(tfull + h, 1);
      mbar_init(tempty + h, 2 * kEpiWarps);
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
  grid_dep_launch();
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer (both CTAs)
    if (lane == 0) {
      fence_proxy_async_global();  // the operands were stored by the kernel before
      int stage = 0;
      uint32_t phase = 0, armed = 0;
      const uint32_t full_lead = mapa_shared(smem_u32(full), 0);
      bool ok = true;
      for (int t = first; ok && t < tiles; t += step) {
        const Tile tile = tile_of<PHASE, BN>(p, t);
        const MuonGemmMat& m = p.t[tile.mat];
        const int mp = m.mt * 256, nk = PHASE == kMuonGram ? m.kn : m.km;
        const uint32_t abase = PHASE == kMuonGram ? m.x[p.cur] : PHASE == kMuonPoly ? m.a : m.b;
        const uint32_t bbase = PHASE == kMuonPoly ? m.a : m.x[p.cur];
        const int arow = tile.i * 256 + static_cast<int>(rank) * kBM, brow = tile.j * BN + static_cast<int>(rank) * C::HB;
        const int big_j = tile.j / (256 / BN);
        for (int kb = 0; kb < nk; ++kb) {
          if (!wait_bounded(empty + stage, phase ^ 1u, abort_flag, p.ctl, 41)) {
            ok = false;
            break;
          }
          uint8_t* sa = smem + stage * C::STAGE_BYTES;
          const uint32_t fb = full_lead + static_cast<uint32_t>(stage) * 8u;
          if (rank == 0) {
            mbar_arrive_expect_tx(full + stage, 2 * C::STAGE_BYTES);  // both CTAs' bytes
            armed |= 1u << stage;
          }
          load_rows<kBM>(sa, &map, fb, abase, mp, arow, kb, PHASE != kMuonGram && (kb >> 2) < tile.i);
          // kMuonApply: B is X, 64 of its rows and this CTA's columns; its panels lie like a mirror image's
          load_rows<C::HB>(sa + A_BYTES, &map, fb, bbase, mp, brow, kb, PHASE == kMuonApply || (PHASE == kMuonPoly && (kb >> 2) < big_j));
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
    if (lane == 0 && rank == 0) {
      constexpr uint32_t kIdesc = idesc_f16_f32(2 * kBM, BN);
      int stage = 0, h = 0;
      uint32_t phase = 0, uses[2] = {0u, 0u};
      bool ok = true, issued = false;
      for (int t = first; ok && t < tiles; t += step) {
        const Tile tile = tile_of<PHASE, BN>(p, t);
        const MuonGemmMat& m = p.t[tile.mat];
        const int nk = PHASE == kMuonGram ? m.kn : m.km, big_j = tile.j / (256 / BN);
        for (int from = 0; ok && from < nk; from += kMuonDepth) {
          if (!wait_bounded(tempty + h, (uses[h] & 1u) ^ 1u, abort_flag, p.ctl, 42)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem_base + static_cast<uint32_t>(h * 256);
          for (int kb = from; kb < min(nk, from + kMuonDepth); ++kb) {
            if (!wait_bounded(full + stage, phase, abort_flag, p.ctl, 43)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t sa = smem_u32(smem + stage * C::STAGE_BYTES), sb = sa + A_BYTES;
            const bool amn = PHASE != kMuonGram && (kb >> 2) < tile.i;
            const bool bmn = PHASE == kMuonApply || (PHASE == kMuonPoly && (kb >> 2) < big_j);
            const uint32_t idesc = kIdesc | (amn ? kAMajor : 0u) | (bmn ? kBMajor : 0u);
#pragma unroll
            for (int q = 0; q < kBK / 16; ++q)
              umma_bf16_pair(d, slice_desc(amn, sa, q), slice_desc(bmn, sb, q), idesc, (kb > from || q > 0) ? 1u : 0u);
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
    const int q = warp & 3, hc = (warp - kEpiWarp0) >> 2;  // lane quarter, column half
    const uint32_t lead_tempty = mapa_shared(smem_u32(tempty), 0);
    uint32_t uses[2] = {0u, 0u};
    int h = 0;
    for (int t = first; t < tiles; t += step) {
      const Tile tile = tile_of<PHASE, BN>(p, t);
      const MuonGemmMat& m = p.t[tile.mat];
      const int mp = m.mt * 256;
      const int nk = PHASE == kMuonGram ? m.kn : m.km;
      const bool deep = nk > kMuonDepth;
      float4* scratch = nullptr;  // of this lane: [BN / 64][8][32 lanes] per warp
      if (deep)
        scratch = reinterpret_cast<float4*>(p.scratch + (static_cast<size_t>(blockIdx.x) * kEpiWarps + warp - kEpiWarp0) * (BN / 64) * 4096) + lane;
      bool got = true;
      for (int from = 0; from + kMuonDepth < nk; from += kMuonDepth) {  // all but the last stretch of the sum
        got = __all_sync(0xffffffffu, wait_bounded(tfull + h, uses[h] & 1u, abort_flag, p.ctl, 45));
        if (!got) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < BN / 64; ++c) {
          float v[32];
          tmem_ld32(tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(h * 256 + hc * (BN / 2) + c * 32), v);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            float4 x = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
            if (from > 0) {
              const float4 y = scratch[(c * 8 + k) * 32];
              x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
            }
            scratch[(c * 8 + k) * 32] = x;
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(lead_tempty + h * 8);
        ++uses[h];
        h ^= 1;
      }
      if (!got) break;
      got = wait_bounded(tfull + h, uses[h] & 1u, abort_flag, p.ctl, 44);
      if (!__all_sync(0xffffffffu, got)) break;
      tc_fence_after();
      const uint32_t out = PHASE == kMuonGram ? m.a : PHASE == kMuonPoly ? m.b : m.x[p.cur ^ 1];
      const uint32_t add = PHASE == kMuonPoly ? m.a : m.x[p.cur];
      const int row = tile.i * 256 + static_cast<int>(rank) * kBM + q * 32 + lane;
#pragma unroll
      for (int c = 0; c < BN / 64; ++c) {
        const int col = tile.j * BN + hc * (BN / 2) + c * 32;
        const size_t at = (static_cast<size_t>(col >> 6) * mp + row) * 128 + (col & 63) * 2;
        float v[32];
        tmem_ld32(tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(h * 256 + hc * (BN / 2) + c * 32), v);
        tmem_ld_wait();
        if (c == BN / 64 - 1) {  // the half is free for the next tile but one
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_remote(lead_tempty + h * 8);
        }
        if (deep) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float4 y = scratch[(c * 8 + k) * 32];
            v[4 * k] += y.x, v[4 * k + 1] += y.y, v[4 * k + 2] += y.z, v[4 * k + 3] += y.w;
          }
        }
        uint4* dst = reinterpret_cast<uint4*>(p.ws + static_cast<size_t>(out) * 128 + at);
        const uint4* hi = reinterpret_cast<const uint4*>(p.ws + static_cast<size_t>(add) * 128 + at);
        uint4* lo = reinterpret_cast<uint4*>(p.ws + static_cast<size_t>(m.lo) * 128 + at);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float x[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = v[8 * k + j] * p.acc;
          if (PHASE != kMuonGram) {
            const uint4 w = hi[k];
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
            uint32_t ll[4] = {0u, 0u, 0u, 0u};
            if (PHASE == kMuonApply) {
              const uint4 l = lo[k];
              ll[0] = l.x, ll[1] = l.y, ll[2] = l.z, ll[3] = l.w;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float2 f = unpack_f16x2(ww[j]);
              if (PHASE == kMuonApply) {
                const float2 g = unpack_f16x2(ll[j]);
                f.x += g.x;
                f.y += g.y;
              }
              x[2 * j] = fmaf(f.x, p.add, x[2 * j]);
              x[2 * j + 1] = fmaf(f.y, p.add, x[2 * j + 1]);
            }
          }
          uint32_t o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) o[j] = pack_f16x2(x[2 * j], x[2 * j + 1]);
          dst[k] = make_uint4(o[0], o[1], o[2], o[3]);
          if (PHASE == kMuonApply && p.want_lo) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 f = unpack_f16x2(o[j]);
              o[j] = pack_f16x2(x[2 * j] - f.x, x[2 * j + 1] - f.y);
            }
            lo[k] = make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
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

cudaLaunchConfig_t gemm_config(cudaLaunchAttribute* attr, int clusters, int smem, cudaStream_t stream) {
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // see grid_dep_wait()
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * clusters, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cfg;
}

template <int PHASE, int BN>
cudaError_t prepare_one(int* max_clusters) {
  cudaError_t e = cudaFuncSetAttribute(muon_gemm_kernel<PHASE, BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<BN>::SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = gemm_config(attr, 1, Cfg<BN>::SMEM, nullptr);
  cfg.numAttrs = 1;  // occupancy: the cluster shape only
  int n = 0;
  e = cudaOccupancyMaxActiveClusters(&n, muon_gemm_kernel<PHASE, BN>, &cfg);
  if (e == cudaSuccess && n < *max_clusters) *max_clusters = n;
  return e;
}

template <int PHASE, int BN>
cudaError_t launch_one(const CUtensorMap& ws, const MuonGemmParams& p, int clusters, cudaStream_t stream) {
  const int tiles = p.tiles * (256 / BN);
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = gemm_config(attr, tiles < clusters ? tiles : clusters, Cfg<BN>::SMEM, stream);
  return cudaLaunchKernelEx(&cfg, muon_gemm_kernel<PHASE, BN>, ws, p);
}

}  // namespace

cudaError_t muon_gemm_prepare(int* max_clusters) {
  *max_clusters = kMaxClusters;
  cudaError_t e = prepare_one<kMuonGram, 256>(max_clusters);
  if (e == cudaSuccess) e = prepare_one<kMuonPoly, 256>(max_clusters);
  if (e == cudaSuccess) e = prepare_one<kMuonApply, 256>(max_clusters);
  if (e == cudaSuccess) e = prepare_one<kMuonGram, 128>(max_clusters);
  if (e == cudaSuccess) e = prepare_one<kMuonPoly, 128>(max_clusters);
  if (e == cudaSuccess) e = prepare_one<kMuonApply, 128>(max_clusters);
  return e;
}

cudaError_t launch_muon_gemm(int phase, const CUtensorMap& ws, const MuonGemmParams& p, int clusters, cudaStream_t stream) {
  // 256-wide tiles read fewer operands per product, 128-wide ones leave fewer SMs idle: the rounds of tiles decide, a narrow one
  // counting 5/8 of a wide one.
  const int64_t wide = (p.tiles + clusters - 1) / clusters, narrow = (2 * static_cast<int64_t>(p.tiles) + clusters - 1) / clusters;
  if (5 * narrow < 8 * wide) {
    if (phase == kMuonGram) return launch_one<kMuonGram, 128>(ws, p, clusters, stream);
    if (phase == kMuonPoly) return launch_one<kMuonPoly, 128>(ws, p, clusters, stream);
    return launch_one<kMuonApply, 128>(ws, p, clusters, stream);
  }
  if (phase == kMuonGram) return launch_one<kMuonGram, 256>(ws, p, clusters, stream);
  if (phase == kMuonPoly) return launch_one<kMuonPoly, 256>(ws, p, clusters, stream);
  return launch_one<kMuonApply, 256>(ws, p, clusters, stream);
}

}  // namespace hylo
