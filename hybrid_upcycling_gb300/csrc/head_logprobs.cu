// Log-probabilities of given tokens and entropies straight from hidden states and an LM head, on
// sm_103a: one persistent, warp-specialised kernel computes the logit tiles z = h W^T on the
// tensor cores (tcgen05 UMMA on CTA pairs, TMA-fed 128-byte-swizzled operands, fp32 accumulators
// in TMEM) and folds each tile into running softmax sums, so that logits are never stored:
//   mx = max z, s = sum e^((z - mx)/tau), a = sum e^((z - mx)/tau) (z - mx)/tau, and z_t itself;
//   a small kernel joins the partial sums: logp = (z_t - mx)/tau - log s, entropy = log s - a/s.
// (The gradient recomputes the tiles: kl_bwd_pipe.cu.)
//
// Roles (384 threads per CTA): warp 0 issues the TMA loads, warp 1 of the even CTA owns TMEM and
// issues the UMMAs for the pair, warps 4..11 are the epilogue: warp w reads TMEM lanes
// 32 (w % 4) .. + 31, one token row per thread, warps 4..7 columns 0..127 of a 256-column tile,
// warps 8..11 the other half. TMEM holds two tiles, so that one is read while the next is
// computed. A deep hidden dimension is accumulated in parts (kLogitDepth), one TMEM tile after another, which the
// epilogue adds up in registers before it folds them (hence setmaxnreg: 56 registers per thread for warpgroup 0, 224 for
// the others). Every (token, vocabulary segment, column half) writes its sums to a slot of
// its own; nothing is added in an order that could change.
#include "hylo_ops_internal.h"

namespace hylo {
namespace {

constexpr float kLog2eF = 1.4426950408889634f;
constexpr float kLn2F = 0.6931471805599453f;

constexpr int kEpiWarps = 8;
constexpr int kEpiWarp0 = 4;
constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);
constexpr int kRegsControl = 56;         // per thread, warpgroup 0 (TMA, UMMA)
constexpr int kRegsEpilogue = 224;       // per thread, warpgroups 1 and 2
static_assert(128 * kRegsControl + 256 * kRegsEpilogue <= kThreads * 168, "register split of the launch's 168 per thread");
constexpr int BN = 256;                 // vocabulary columns of a pair tile
constexpr int HB = BN / 2;              // W rows staged per CTA; columns per epilogue warp
constexpr int A_BYTES = kBM * kBK * 2;
constexpr int B_BYTES = HB * kBK * 2;
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int STAGES = (232448 - 1024 - 256) / STAGE_BYTES;
constexpr int BAR_OFF = STAGES * STAGE_BYTES;
constexpr int NBARS = 2 * STAGES + 4 + 1;  // full, empty, tfull[2], tempty[2], drain
constexpr int SMEM = 1024 + BAR_OFF + NBARS * 8 + 16;
static_assert(SMEM <= 232448, "shared memory budget");

__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity, unsigned long long limit_ns) {
  const uint32_t a = smem_u32(bar);
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(a, parity)) {
    if (globaltimer_ns() - t0 > limit_ns) return;
  }
}

struct Sums {
  float mx, s, a;  // as above, a and exponents in units of log 2
};

__device__ __forceinline__ void rebase(Sums& r, float mx, float c) {
  const float d = fmaxf((r.mx - mx) * c, -200.f);  // the first columns: mx was -inf
  const float w = ex2_approx(d);
  r.a = w * fmaf(r.s, d, r.a);
  r.s *= w;
  r.mx = mx;
}

// Adds 32 columns of a TMEM tile.
__device__ __forceinline__ void add32(float (&z)[32], uint32_t taddr) {
  float v[32];
  tmem_ld32(taddr, v);
  tmem_ld_wait();
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float2 s = __fadd2_rn(make_float2(z[2 * j], z[2 * j + 1]), make_float2(v[2 * j], v[2 * j + 1]));
    z[2 * j] = s.x;
    z[2 * j + 1] = s.y;
  }
}

// Folds 32 logits; MASKED: only the first `valid` of them exist.
template <bool MASKED>
__device__ __forceinline__ void fold32(Sums& r, const float (&z)[32], int valid, float c) {
  float mx = r.mx;
#pragma unroll
  for (int j = 0; j < 32; ++j)
    if (!MASKED || j < valid) mx = fmaxf(mx, z[j]);
  rebase(r, mx, c);
  const float2 c2 = make_float2(c, c), nm = make_float2(-mx, -mx);  // the difference first: it is exact where it matters
  float2 s = make_float2(0.f, 0.f), a = s;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    float2 y = __fmul2_rn(__fadd2_rn(make_float2(z[2 * j], z[2 * j + 1]), nm), c2);
    if (MASKED) {
      if (2 * j >= valid) y.x = -1024.f;  // 2^-1024 is 0
      if (2 * j + 1 >= valid) y.y = -1024.f;
    }
    const float2 e = make_float2(ex2_approx(y.x), ex2_approx(y.y));
    s = __fadd2_rn(s, e);
    a = __ffma2_rn(e, y, a);
  }
  r.s += s.x + s.y;
  r.a += a.x + a.y;
}

// Work unit u: 256-token tile u % token_tiles of segment u / token_tiles (segments ascend, so the clusters
// at work share few segments: their W rows come from DRAM once and from L2 for the others).
__device__ __forceinline__ void unit_range(const HeadParams& p, int u, int& row0, int& vt0, int& vt1, int& seg) {
  seg = u / p.token_tiles;
  row0 = (u - seg * p.token_tiles) * 2 * kBM;
  vt0 = static_cast<int>((static_cast<long long>(seg) * p.vtiles) / p.nseg);
  vt1 = static_cast<int>((static_cast<long long>(seg + 1) * p.vtiles) / p.nseg);
}

__global__ void __launch_bounds__(kThreads, 1)
head_logprobs_kernel(const __grid_constant__ CUtensorMap tm_h, const __grid_constant__ CUtensorMap tm_W,
                     const HeadParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + BAR_OFF);  // used in the even CTA
  uint64_t* empty = full + STAGES;                                // both CTAs: stage free
  uint64_t* tfull = empty + STAGES;                               // both CTAs: TMEM half complete
  uint64_t* tempty = tfull + 2;                                   // even CTA: half read by both CTAs
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();  // 0: issues the UMMAs
  const int cid = blockIdx.x >> 1;
  const int ncl = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull + b, 1);
      mbar_init(tempty + b, 2 * kEpiWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (threadIdx.x == 32) {
    prefetch_tmap(&tm_h);
    prefetch_tmap(&tm_W);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // barriers of both CTAs initialised before any cross-CTA signal
  tc_fence_after();
  grid_dep_wait();  // the workspace may be shared with the previous kernel in the stream
  grid_dep_launch();
  const uint32_t tmem_base = *tmem_slot;
  const int my_rows = static_cast<int>(rank) * kBM;

  if (warp < kEpiWarp0) setmaxnreg_dec<kRegsControl>();  // each warpgroup changes its registers at once
  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer (both CTAs)
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, armed = 0;
      bool ok = true;
      const uint32_t full_lead = mapa_shared(smem_u32(full), 0);
      const int copy = cid % p.copies;
      for (int u = cid; ok && u < p.units; u += ncl) {
        int row0, vt0, vt1, seg;
        unit_range(p, u, row0, vt0, vt1, seg);
        for (int vt = vt0; ok && vt < vt1; ++vt) {
          const int brow = vt * BN + static_cast<int>(rank) * HB;
          for (int kb = 0; kb < p.kb; ++kb) {
            if (!wait_bounded(empty + stage, phase ^ 1u, abort_flag, p.ctl, 41)) {
              ok = false;
              break;
            }
            uint8_t* sa = smem + stage * STAGE_BYTES;
            const uint32_t fbar = full_lead + static_cast<uint32_t>(stage) * 8u;
            if (rank == 0) {
              mbar_arrive_expect_tx(full + stage, 2 * STAGE_BYTES);  // both CTAs' bytes
              armed |= 1u << stage;
            }
            tma_load_3d_pair(sa, &tm_h, fbar, kb * kBK, row0 + my_rows, copy);
            tma_load_2d_pair(sa + A_BYTES, &tm_W, fbar, kb * kBK, brow);
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
      }
      if (!ok) {
        // Let every armed load land before the CTA can exit: the latest armed phase of stage s
        // has parity `phase` for stages below the current one and `phase ^ 1` otherwise.
        for (int s = 0; s < STAGES; ++s) {
          if (armed & (1u << s)) drain_wait(full + s, s < stage ? phase : (phase ^ 1u), 100000000ull);
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ UMMA issuer (even CTA)
    if (lane == 0 && rank == 0) {
      constexpr uint32_t kIdesc = idesc_bf16_f32(2 * kBM, BN, false, false);
      int stage = 0;
      uint32_t phase = 0;
      int lt = 0;
      bool ok = true, issued = false;
      for (int u = cid; ok && u < p.units; u += ncl) {
        int row0, vt0, vt1, seg;
        unit_range(p, u, row0, vt0, vt1, seg);
        for (int i = vt0 * p.depths; ok && i < vt1 * p.depths; ++i, ++lt) {
          const int h = lt & 1;
          if (!wait_bounded(tempty + h, (static_cast<uint32_t>(lt >> 1) & 1u) ^ 1u, abort_flag, p.ctl, 42)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem_base + static_cast<uint32_t>(h * BN);
          const int depth = min(kLogitDepth, p.kb - i % p.depths * kLogitDepth);
          for (int kb = 0; kb < depth; ++kb) {
            if (!wait_bounded(full + stage, phase, abort_flag, p.ctl, 43)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t sa = smem_u32(smem + stage * STAGE_BYTES);
            const uint32_t sb = sa + A_BYTES;
#pragma unroll
            for (int k = 0; k < kBK / 16; ++k) {
              umma_bf16_pair(d, smem_desc_sw128(sa + k * 32, 0, 1024), smem_desc_sw128(sb + k * 32, 0, 1024), kIdesc,
                             (kb > 0 || k > 0) ? 1u : 0u);
            }
            umma_commit_pair(empty + stage, 0x3);
            issued = true;
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (!ok) break;
          umma_commit_pair(tfull + h, 0x3);
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
    const int q = warp & 3;                 // TMEM lane quarter this warp may access
    const int hc = (warp - kEpiWarp0) >> 2;  // column half
    const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(hc * HB);
    const uint32_t lead_tempty = mapa_shared(smem_u32(tempty), 0);
    int lt = 0;
    bool ok = true;
    for (int u = cid; ok && u < p.units; u += ncl) {
      int row0, vt0, vt1, seg;
      unit_range(p, u, row0, vt0, vt1, seg);
      const int token = row0 + my_rows + q * 32 + lane;
      const int64_t want = token < p.N ? p.tokens[token] : -1;
      // the row's own column of this warp's half, relative to vocabulary column 0 of the half
      const int tcol = want >= 0 && want < p.V ? static_cast<int>(want) : -1;
      Sums r{-INFINITY, 0.f, 0.f};
      for (int vt = vt0; ok && vt < vt1; ++vt) {
        float z[HB / 32][32] = {};  // this row's logits, the sum of its parts
#pragma unroll 1
        for (int part = 0; part < p.depths; ++part, ++lt) {
          const int h = lt & 1;
          const bool w = wait_bounded(tfull + h, static_cast<uint32_t>(lt >> 1) & 1u, abort_flag, p.ctl, 44);
          if (!__all_sync(0xffffffffu, w)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t half = lane_base + static_cast<uint32_t>(h * BN);
#pragma unroll
          for (int ch = 0; ch < HB / 32; ++ch) add32(z[ch], half + ch * 32);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_remote(lead_tempty + h * 8);
        }
        if (!ok) break;
        const int col_base = vt * BN + hc * HB;
#pragma unroll
        for (int ch = 0; ch < HB / 32; ++ch) {
          const int col = col_base + ch * 32;
          const int valid = p.V - col;
          if (valid <= 0) continue;
          const int rel = tcol - col;
          if (__any_sync(0xffffffffu, rel >= 0 && rel < 32)) {
            float zt = 0.f;
#pragma unroll
            for (int j = 0; j < 32; ++j) zt = j == rel ? z[ch][j] : zt;
            if (rel >= 0 && rel < 32) p.z_token[token] = zt;
          }
          if (valid >= 32)
            fold32<false>(r, z[ch], 32, p.c);
          else
            fold32<true>(r, z[ch], valid, p.c);
        }
      }
      if (!ok) break;
      if (token < p.N)
        p.part[static_cast<int64_t>(token) * p.slots + 2 * seg + hc] = make_float4(r.mx, r.s, r.a, 0.f);
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

// ---- A few tokens (one decoding step): the LM head's bytes are the cost, and the tensor cores would spend their
// 256-row tiles on them. Every warp takes kRows words at a time, its lanes walk the hidden dimension with
// 16-byte loads of W and the tokens' states in fp32 from shared memory, and the dot products end in
// a warp reduction; lane t keeps token t's running sums. fp32 multiply-adds: no drift of
// long tensor-core accumulations. Measured beside the tensor-core path (128256 words; d = 4096 177 us and d = 2048 95 us
// for three or four tokens): one token 147 us (7.1 TB/s) and 78; two tokens 152 and 90; four tokens 172 at d = 4096,
// where the multiply-adds and not the loads set the time. So it takes one or two.
constexpr int kFewThreads = 512;
constexpr int kFewWarps = kFewThreads / 32;
constexpr int kRows = 4;

template <int NT>
__global__ void __launch_bounds__(kFewThreads, 1)
head_few_kernel(const uint16_t* __restrict__ h, const uint16_t* __restrict__ W, int d, const HeadParams p) {
  extern __shared__ float hs[];  // [NT][d]
  __shared__ Sums sums[kFewWarps][NT];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < NT * d; i += kFewThreads)
    hs[i] = i < p.N * d ? __uint_as_float(static_cast<uint32_t>(h[i]) << 16) : 0.f;
  __syncthreads();
  const int64_t want = lane < p.N ? p.tokens[lane] : -1;
  Sums r{-INFINITY, 0.f, 0.f};
  const int nvec = d / 8;
  const int64_t groups = (static_cast<int64_t>(p.V) + kRows - 1) / kRows;
  for (int64_t g = static_cast<int64_t>(blockIdx.x) * kFewWarps + warp; g < groups; g += static_cast<int64_t>(gridDim.x) * kFewWarps) {
    const int64_t v0 = g * kRows;
    const uint4* row[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) row[k] = reinterpret_cast<const uint4*>(W + min(v0 + k, static_cast<int64_t>(p.V) - 1) * d);
    float2 acc[kRows][NT];
#pragma unroll
    for (int k = 0; k < kRows; ++k)
#pragma unroll
      for (int t = 0; t < NT; ++t) acc[k][t] = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int i = lane; i < nvec; i += 32) {
      uint4 w[kRows];
#pragma unroll
      for (int k = 0; k < kRows; ++k) w[k] = __ldcs(row[k] + i);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float4 a = *reinterpret_cast<const float4*>(hs + t * d + i * 8), b = *reinterpret_cast<const float4*>(hs + t * d + i * 8 + 4);
        const float2 x[4] = {make_float2(a.x, a.y), make_float2(a.z, a.w), make_float2(b.x, b.y), make_float2(b.z, b.w)};
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
          const uint32_t q[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            acc[k][t] = __ffma2_rn(make_float2(__uint_as_float(q[j] << 16), __uint_as_float(q[j] & 0xffff0000u)), x[j], acc[k][t]);
        }
      }
    }
    float z[kRows];  // this lane's token's logits (lanes from NT on: token 0's)
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      z[k] = 0.f;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float s = acc[k][t].x + acc[k][t].y;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(~0u, s, off);
        z[k] = t == 0 || lane == t ? s : z[k];
      }
    }
    const int rows = static_cast<int>(min(static_cast<int64_t>(kRows), p.V - v0));
    float mx = r.mx;
#pragma unroll
    for (int k = 0; k < kRows; ++k)
      if (k < rows) mx = fmaxf(mx, z[k]);
    rebase(r, mx, p.c);
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      if (k < rows) {
        const float y = (z[k] - mx) * p.c;
        const float e = ex2_approx(y);
        r.s += e;
        r.a = fmaf(e, y, r.a);
        if (want == v0 + k) p.z_token[lane] = z[k];
      }
    }
  }
  if (lane < NT) sums[warp][lane] = r;
  __syncthreads();
  if (tid < NT && tid < p.N) {
    Sums total = sums[0][tid];
    for (int w = 1; w < kFewWarps; ++w) {
      Sums o = sums[w][tid];
      if (o.mx == -INFINITY) continue;  // a warp without words
      const float m = fmaxf(total.mx, o.mx);
      rebase(total, m, p.c);
      rebase(o, m, p.c);
      total.s += o.s;
      total.a += o.a;
    }
    p.part[static_cast<int64_t>(tid) * p.slots + blockIdx.x] = make_float4(total.mx, total.s, total.a, 0.f);
  }
}

// One warp per token joins its partial sums (a fixed tree).
__global__ void __launch_bounds__(256) head_combine_kernel(const HeadParams p, float* logp, float* entropy, float* lse) {
  const int lane = threadIdx.x & 31;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (n >= p.N) return;
  const int slots = p.slots;
  Sums r{-INFINITY, 0.f, 0.f};
  auto add = [&](float mx, float s, float a) {
    if (mx == -INFINITY) return;  // a half without columns (the vocabulary ends before it)
    const float m = fmaxf(r.mx, mx);
    Sums o{mx, s, a};
    rebase(r, m, p.c);
    rebase(o, m, p.c);
    r.s += o.s;
    r.a += o.a;
  };
  for (int i = lane; i < slots; i += 32) {
    const float4 v = p.part[n * slots + i];
    add(v.x, v.y, v.z);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const float mx = __shfl_xor_sync(~0u, r.mx, off), s = __shfl_xor_sync(~0u, r.s, off), a = __shfl_xor_sync(~0u, r.a, off);
    add(mx, s, a);
  }
  if (lane != 0) return;
  const float inv_tau = p.inv_tau, log_s = logf(r.s);
  const int64_t t = p.tokens[n];
  logp[n] = t < 0 ? 0.f : t >= p.V ? __uint_as_float(0x7fffffffu) : (p.z_token[n] - r.mx) * inv_tau - log_s;
  if (entropy) entropy[n] = log_s - kLn2F * r.a / r.s;
  if (lse) lse[n] = r.mx * inv_tau + log_s;
}

// Eight values per thread and step.
template <bool BF16>
__global__ void __launch_bounds__(256) join_parts_kernel(const float4* __restrict__ x, int parts, void* __restrict__ y, int64_t n8) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n8; i += static_cast<int64_t>(gridDim.x) * 256) {
    float4 a = __ldcs(x + 2 * i), b = __ldcs(x + 2 * i + 1);
#pragma unroll 4
    for (int k = 1; k < parts; ++k) {
      const float4 c = __ldcs(x + 2 * (k * n8 + i)), d = __ldcs(x + 2 * (k * n8 + i) + 1);
      a = make_float4(a.x + c.x, a.y + c.y, a.z + c.z, a.w + c.w);
      b = make_float4(b.x + d.x, b.y + d.y, b.z + d.z, b.w + d.w);
    }
    if (BF16) {
      static_cast<uint4*>(y)[i] = make_uint4(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w), pack_bf16x2(b.x, b.y), pack_bf16x2(b.z, b.w));
    } else {
      static_cast<float4*>(y)[2 * i] = a;
      static_cast<float4*>(y)[2 * i + 1] = b;
    }
  }
}

// `copies` copies of x [n], one behind the other.
__global__ void __launch_bounds__(256) head_copy_kernel(const uint4* __restrict__ x, uint4* __restrict__ y, int n, int copies) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  const uint4 v = x[i];
  for (int c = 0; c < copies; ++c) y[c * n + i] = v;
}

cudaLaunchConfig_t head_config(cudaLaunchAttribute* attr, int clusters, cudaStream_t stream) {
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
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

}  // namespace

cudaError_t launch_join_parts(const float* x, int parts, void* y, bool bf16, int64_t n, int sms, cudaStream_t stream) {
  const int64_t want = (n / 8 + 255) / 256, cap = static_cast<int64_t>(sms) * 8;
  const int grid = static_cast<int>(want < cap ? want : cap);
  const float4* x4 = reinterpret_cast<const float4*>(x);
  if (bf16)
    join_parts_kernel<true><<<grid, 256, 0, stream>>>(x4, parts, y, n / 8);
  else
    join_parts_kernel<false><<<grid, 256, 0, stream>>>(x4, parts, y, n / 8);
  return cudaGetLastError();
}

cudaError_t head_few_prepare();

cudaError_t head_prepare(int* max_clusters) {
  cudaError_t e = head_few_prepare();
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(head_logprobs_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = head_config(attr, 1, nullptr);
  cfg.numAttrs = 1;  // occupancy: the cluster shape only
  return cudaOccupancyMaxActiveClusters(max_clusters, head_logprobs_kernel, &cfg);
}

cudaError_t launch_head_copy(const uint16_t* h, void* copies, int64_t n, int count, cudaStream_t stream) {
  const int n8 = static_cast<int>(n / 8);
  head_copy_kernel<<<(n8 + 255) / 256, 256, 0, stream>>>(reinterpret_cast<const uint4*>(h), static_cast<uint4*>(copies), n8, count);
  return cudaGetLastError();
}

constexpr int kFewTokens = 2;
constexpr size_t kFewSmem = 200 * 1024;

template <int NT>
cudaError_t launch_few(const uint16_t* h, const uint16_t* W, int d, const HeadParams& p, int ctas, cudaStream_t stream) {
  head_few_kernel<NT><<<ctas, kFewThreads, static_cast<size_t>(NT) * d * sizeof(float), stream>>>(h, W, d, p);
  return cudaGetLastError();
}

bool head_few_fits(int64_t N, int64_t d) { return N <= kFewTokens && static_cast<size_t>(N) * d * sizeof(float) <= kFewSmem; }

cudaError_t head_few_prepare() {
  const void* kernels[] = {reinterpret_cast<const void*>(head_few_kernel<1>), reinterpret_cast<const void*>(head_few_kernel<2>)};
  for (const void* k : kernels) {
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kFewSmem));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_head_few(const uint16_t* h, const uint16_t* W, int d, const HeadParams& p, float* logp, float* entropy,
                            float* lse, cudaStream_t stream) {
  const cudaError_t e = p.N == 1 ? launch_few<1>(h, W, d, p, p.slots, stream) : launch_few<2>(h, W, d, p, p.slots, stream);
  if (e != cudaSuccess) return e;
  head_combine_kernel<<<(p.N + 7) / 8, 256, 0, stream>>>(p, logp, entropy, lse);
  return cudaGetLastError();
}

cudaError_t launch_head_logprobs(const CUtensorMap& h, const CUtensorMap& W, const HeadParams& p, float* logp,
                                 float* entropy, float* lse, int clusters, cudaStream_t stream) {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = head_config(attr, clusters, stream);
  cudaError_t e = cudaLaunchKernelEx(&cfg, head_logprobs_kernel, h, W, p);
  if (e != cudaSuccess) return e;
  head_combine_kernel<<<(p.N + 7) / 8, 256, 0, stream>>>(p, logp, entropy, lse);
  return cudaGetLastError();
}

}  // namespace hylo
