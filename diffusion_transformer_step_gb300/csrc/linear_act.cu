// Linear layer with bias, activation and residual in its epilogue: out = act(a w^T + bias) + res, bf16
// operands, fp32 from the accumulator to the one rounding of the output.
//
//   linear_act_wide_kernel   the pair kernel of the step's products: CTA pairs, 256 x 256 tiles, seven stages of
//                            64-deep blocks, two accumulators, so that a tile's epilogue runs beside the next
//                            tile's main loop.  Where tiles leave pairs idle, the depth is split over
//                            a cluster of up to four pairs.
//   linear_act_few_kernel    few rows, where reading the weights bounds the time: 128 rows of weights take the
//                            MMA's row side and the activation rows its column side, the depth split over
//                            a cluster of up to eight CTAs.
//
// Splits add up through distributed shared memory, in rank order: each CTA leaves its part in its own shared
// memory (the ring has been read), then finishes its share of the rows from all parts.
#include <math.h>

#include <atomic>

#include "cta_pair.cuh"
#include "runtime.h"

namespace dit {

namespace {

enum : uint32_t { kSiteEmpty = 0xa01, kSiteFull, kSiteAccEmpty, kSiteAccFull };

struct alignas(64) Params {
  CUtensorMap a_map, w_map;
  LinearActArgs a;
  int kblocks, m_tiles, tiles, splits;
};

// ---- epilogue --------------------------------------------------------------------------------

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two values at a time: packed fp32 arithmetic, exponentials and reciprocals of the special unit.
template <int kAct>
__device__ __forceinline__ float2 activate(float2 z) {
  auto f2 = [](float v) { return make_float2(v, v); };
  if constexpr (kAct == 1) return make_float2(z.x < 0.f ? 0.f : z.x, z.y < 0.f ? 0.f : z.y);
  if constexpr (kAct == 2) {
    // Phi(-|z|) = erfc(|z| / sqrt 2) / 2 by Abramowitz and Stegun 7.1.26 (within 0.75e-7):
    // t (a1 + t (a2 + ...)) exp(-z^2 / 2) / 2, t = 1 / (1 + p |z| / sqrt 2)
    const float2 x = make_float2(fabsf(z.x), fabsf(z.y));
    const float2 d = __ffma2_rn(x, f2(0.3275911f * 0.70710678f), f2(1.0f));
    const float2 t = make_float2(rcp_approx(d.x), rcp_approx(d.y));
    float2 h = __ffma2_rn(t, f2(0.5f * 1.061405429f), f2(0.5f * -1.453152027f));
    h = __ffma2_rn(t, h, f2(0.5f * 1.421413741f));
    h = __ffma2_rn(t, h, f2(0.5f * -0.284496736f));
    h = __ffma2_rn(t, h, f2(0.5f * 0.254829592f));
    const float2 e = __fmul2_rn(__fmul2_rn(z, f2(-0.72134752f)), z);
    h = __fmul2_rn(__fmul2_rn(t, h), make_float2(ex2_approx(e.x), ex2_approx(e.y)));
    return __fmul2_rn(z, make_float2(z.x < 0.f ? h.x : 1.0f - h.x, z.y < 0.f ? h.y : 1.0f - h.y));
  }
  if constexpr (kAct == 3 || kAct == 4) {
    // z / (1 + 2^(-u)), u = z log2 e, or 2 sqrt(2 / pi) log2 e (z + 0.044715 z^3)
    float2 u = __fmul2_rn(z, f2(kAct == 4 ? -1.4426950408889634f : -2.3022081986f));
    if constexpr (kAct == 3) u = __ffma2_rn(__fmul2_rn(z, z), __fmul2_rn(u, f2(0.044715f)), u);
    const float2 d = __fadd2_rn(make_float2(ex2_approx(u.x), ex2_approx(u.y)), f2(1.0f));
    return __fmul2_rn(z, make_float2(rcp_approx(d.x), rcp_approx(d.y)));
  }
  return z;
}

constexpr int kAnyAct = -1;  // looked up at run time

template <int kAct>
__device__ __forceinline__ void activate4(float2& a, float2& b, int act) {
  if constexpr (kAct != kAnyAct) {
    a = activate<kAct>(a);
    b = activate<kAct>(b);
  } else if (act != 0) {
    if (act == 1) activate4<1>(a, b, 1);
    else if (act == 2) activate4<2>(a, b, 2);
    else if (act == 3) activate4<3>(a, b, 3);
    else activate4<4>(a, b, 4);
  }
}

// Four neighbouring values [c, c + 4) of a row of n, c % 4 == 0 and c < n: rows are 16-byte aligned, so that only
// the last group of a row may need single ones.
__device__ __forceinline__ uint2 load4(const bf16* row, int c, int n) {
  if (c + 4 <= n) return *reinterpret_cast<const uint2*>(row + c);
  const uint16_t* s = reinterpret_cast<const uint16_t*>(row + c);
  uint2 u = make_uint2(s[0], 0u);
  if (c + 1 < n) u.x |= (uint32_t)s[1] << 16;
  if (c + 2 < n) u.y = s[2];
  return u;
}

// Sums v of columns [c, c + 4) of row r to the output; bias and res as load4 gives them.
template <int kAct>
__device__ __forceinline__ void finish4(const LinearActArgs& p, long long r, int c, float4 v, uint2 bias, uint2 res) {
  const bool whole = c + 4 <= p.n;
  float2 lo = make_float2(v.x, v.y), hi = make_float2(v.z, v.w);
  if (p.bias) {
    lo = __fadd2_rn(lo, unpack_bf16x2(bias.x));
    hi = __fadd2_rn(hi, unpack_bf16x2(bias.y));
  }
  activate4<kAct>(lo, hi, p.act);
  if (p.res) {
    lo = __fadd2_rn(lo, unpack_bf16x2(res.x));
    hi = __fadd2_rn(hi, unpack_bf16x2(res.y));
  }
  if (p.out_f32) {
    float* o = reinterpret_cast<float*>(p.out) + r * p.ld_out + c;
    if (whole) {
      *reinterpret_cast<float4*>(o) = make_float4(lo.x, lo.y, hi.x, hi.y);
    } else {
      o[0] = lo.x;
      if (c + 1 < p.n) o[1] = lo.y;
      if (c + 2 < p.n) o[2] = hi.x;
    }
  } else {
    bf16* o = reinterpret_cast<bf16*>(p.out) + r * p.ld_out + c;
    const uint2 u = make_uint2(pack_bf16x2(lo.x, lo.y), pack_bf16x2(hi.x, hi.y));
    if (whole) {
      *reinterpret_cast<uint2*>(o) = u;
    } else {
      uint16_t* h = reinterpret_cast<uint16_t*>(o);
      h[0] = (uint16_t)u.x;
      if (c + 1 < p.n) h[1] = (uint16_t)(u.x >> 16);
      if (c + 2 < p.n) h[2] = (uint16_t)u.y;
    }
  }
}

// 32 columns [c, c + 32) of one row, all below n; res: that piece of the residual.
template <int kAct>
__device__ __forceinline__ void finish32(const LinearActArgs& p, long long r, int c, const uint32_t (&v)[32],
                                         const uint4 (&res)[4]) {
  auto eight = [](const uint4& u, float2 (&f)[4]) {
    f[0] = unpack_bf16x2(u.x), f[1] = unpack_bf16x2(u.y), f[2] = unpack_bf16x2(u.z), f[3] = unpack_bf16x2(u.w);
  };
  float2 o[16];
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    float2 b[4];
    if (p.bias) eight(__ldg(reinterpret_cast<const uint4*>(p.bias + c + g * 8)), b);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 z = make_float2(__uint_as_float(v[g * 8 + 2 * i]), __uint_as_float(v[g * 8 + 2 * i + 1]));
      if (p.bias) z = __fadd2_rn(z, b[i]);
      o[g * 4 + i] = activate<kAct>(z);
    }
  }
  if (p.res) {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      float2 x[4];
      eight(res[g], x);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[g * 4 + i] = __fadd2_rn(o[g * 4 + i], x[i]);
    }
  }
  if (p.out_f32) {
    float4* dst = reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + r * p.ld_out + c);
#pragma unroll
    for (int i = 0; i < 8; ++i) dst[i] = make_float4(o[2 * i].x, o[2 * i].y, o[2 * i + 1].x, o[2 * i + 1].y);
  } else {
    uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<bf16*>(p.out) + r * p.ld_out + c);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      dst[i] = make_uint4(pack_bf16x2(o[4 * i].x, o[4 * i].y), pack_bf16x2(o[4 * i + 1].x, o[4 * i + 1].y),
                          pack_bf16x2(o[4 * i + 2].x, o[4 * i + 2].y), pack_bf16x2(o[4 * i + 3].x, o[4 * i + 3].y));
  }
}

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// The rows r0, r0 + step, ... below `rows` (of the output: m0 further), four columns from c on per thread; part(r, k) is what
// rank k's shared memory holds of them, added in rank order.  Parts and residual of one row are fetched ahead of the
// arithmetic of the row before.  Not unrolled further: a loop that runs a few times waits for its code as
// much as for its data (128 rows of one block of depth, eight rows at once: 8.8 us, two 6.4).
template <int K, typename Part>
__device__ __forceinline__ void finish_rows(const Params& P, int r0, int step, int rows, int m0, int c, Part part) {
  const LinearActArgs& p = P.a;
  struct Row {
    float4 v[K];
    uint2 res;
  };
  auto load = [&](int r, Row& x) {
    x.res = make_uint2(0, 0);
    if (r < rows && p.res) x.res = load4(p.res + (long long)(m0 + r) * p.ld_res, c, p.n);
#pragma unroll
    for (int k = 0; k < K; ++k)
      x.v[k] = r < rows && (K == 1 || k < P.splits) ? part(r, k) : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  const uint2 bias = p.bias ? load4(p.bias, c, p.n) : make_uint2(0, 0);
  auto finish = [&](int r, const Row& x) {
    float4 sum = x.v[0];
#pragma unroll
    for (int k = 1; k < K; ++k) sum.x += x.v[k].x, sum.y += x.v[k].y, sum.z += x.v[k].z, sum.w += x.v[k].w;
    if (r < rows) finish4<kAnyAct>(p, m0 + r, c, sum, bias, x.res);
  };
  Row one, two;
  load(r0, one);
#pragma unroll 1
  for (int r = r0; r < rows; r += 2 * step) {
    load(r + step, two);
    finish(r, one);
    load(r + 2 * step, one);
    finish(r + step, two);
  }
}

// ---- many rows -------------------------------------------------------------------------------

constexpr int kWideStages = 7, kWideThreads = 320;
constexpr uint32_t kWideTile = 128 * 128, kWideStage = 2 * kWideTile;
constexpr size_t kWideBytes = 1024 + (size_t)kWideStages * kWideStage + 256;
static_assert(kWideStages * kWideStage >= 128 * 256 * 4, "a split's part reuses the ring");

// Pair `pair` of a cluster (rank = 2 pair + half) takes the depth blocks [K pair / S, K (pair + 1) / S) of its cluster's
// tiles; with splits a cluster has one tile.  Roles as in the step's products: warp 0 loads, warp 1 issues (the
// pair's first CTA), warps 2 to 9 finish, one thread per row of 128 columns.
template <int kAct, bool kSplit>
__global__ void __launch_bounds__(kWideThreads, 1) linear_act_wide_kernel(const __grid_constant__ Params P) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sW = smem + kWideStages * kWideTile;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kWideStages * kWideStage);
  uint64_t* empty = full + kWideStages;
  uint64_t* acc_full = empty + kWideStages;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t crank = cta_rank(), leader = crank & ~1u, half = crank & 1u;
  const int S = kSplit ? P.splits : 1, split = kSplit ? (int)(crank >> 1) : 0;
  const int first = blockIdx.x / (2 * S), step = gridDim.x / (2 * S);
  const int kb0 = kSplit ? (int)((long long)P.kblocks * split / S) : 0;
  const int kb1 = kSplit ? (int)((long long)P.kblocks * (split + 1) / S) : P.kblocks;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kWideStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 16);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&P.a_map);
    tma_prefetch_desc(&P.w_map);
  }
  __syncwarp();
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  cluster_sync_all();  // barriers and Tensor Memory of every CTA of the cluster are there
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtx wc{P.a.status, abort_flag, kWaitLimitNs};
  grid_dependency_wait();
  allow_dependents();

  if (warp == 0) {
    if (lane == 0) {
      uint32_t stage = 0, phase = 0;
      long long issued = 0;
      bool ok = true;
      for (int t = first; t < P.tiles && ok; t += step) {
        const int nt = t / P.m_tiles, mt = t - nt * P.m_tiles;
        const int arow = mt * 256 + (int)half * 128, wrow = nt * 256 + (int)half * 128;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (mt == 0 && kb + 8 < kb1) pf_l2(&P.w_map, (kb + 8) * 64, wrow);  // one prefetcher per weight column
          if (!mbar_wait_sleep(&empty[stage], phase ^ 1u, wc, kSiteEmpty)) {
            ok = false;
            break;
          }
          const uint32_t fb = map_to_rank(smem_u32(&full[stage]), leader);
          if (half == 0) mbar_arrive_expect_tx(&full[stage], 2 * kWideStage);
          tma2_2sm(sA + stage * kWideTile, &P.a_map, fb, kb * 64, arow);
          tma2_2sm(sW + stage * kWideTile, &P.w_map, fb, kb * 64, wrow);
          ++issued;
          if (++stage == kWideStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok && half == 0) {
        // Unwinding: let copies in flight land (bounded) before the pair exits.
        const long long outstanding = issued < kWideStages ? issued : kWideStages;
        for (long long i = 0; i < outstanding; ++i) {
          if (stage == 0) {
            stage = kWideStages;
            phase ^= 1u;
          }
          --stage;
          const uint64_t t0 = global_timer_ns();
          while (!mbar_try(&full[stage], phase) && global_timer_ns() - t0 < 100000000ull) {
          }
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && half == 0) {
      const uint32_t idesc = make_idesc_bf16(256, 256, false);
      const uint16_t both = (uint16_t)(3u << leader);
      auto commit = [&](uint64_t* bar) {
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                smem_u32(bar)),
            "h"(both)
            : "memory");
      };
      const uint64_t a0 = make_sdesc_sw128(smem_u32(sA), 16, 1024), w0 = make_sdesc_sw128(smem_u32(sW), 16, 1024);
      uint32_t stage = 0, phase = 0;
      int local = 0;
      bool ok = true;
      for (int t = first; t < P.tiles && ok; t += step, ++local) {
        const int acc = local & 1;
        if (!mbar_wait(&acc_empty[acc], ((uint32_t)(local >> 1) & 1u) ^ 1u, wc, kSiteAccEmpty)) break;
        tc_fence_after();
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait(&full[stage], phase, wc, kSiteFull)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t ad = desc_advance(a0, stage * (kWideTile >> 4)), wd = desc_advance(w0, stage * (kWideTile >> 4));
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma2(tmem + (uint32_t)(acc * 256), desc_advance(ad, kk * 2), desc_advance(wd, kk * 2), idesc,
                  kb > kb0 || kk ? 1u : 0u);
          commit(&empty[stage]);
          if (++stage == kWideStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (ok) commit(&acc_full[acc]);
      }
      asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(drain))
                   : "memory");
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try(drain, 0) && global_timer_ns() - t0 < 1000000000ull) {
      }
    }
  } else {
    const int q = warp & 3, eh = (warp - 2) >> 2;  // rows [32 q, 32 q + 32) of this CTA, columns [128 eh, 128 eh + 128)
    const uint32_t free0 = map_to_rank(smem_u32(acc_empty), leader);
    int local = 0;
    for (int t = first; t < P.tiles; t += step, ++local) {
      const int acc = local & 1;
      const int nt = t / P.m_tiles, mt = t - nt * P.m_tiles;
      const int r = q * 32 + lane, row = mt * 256 + (int)half * 128 + r, col = nt * 256 + eh * 128;
      // the residual's pieces one ahead, the first before the accumulator is waited for
      uint4 ahead[4];
      auto fetch = [&](int c) {
        if (kSplit || !P.a.res || row >= P.a.rows || c + 32 > P.a.n) return;
        const uint4* src = reinterpret_cast<const uint4*>(P.a.res + row * P.a.ld_res + c);
#pragma unroll
        for (int i = 0; i < 4; ++i) ahead[i] = src[i];
      };
      fetch(col);
      bool ok = mbar_wait_sleep(&acc_full[acc], (uint32_t)(local >> 1) & 1u, wc, kSiteAccFull);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const uint32_t tb = tmem + (uint32_t)(acc * 256 + eh * 128) + ((uint32_t)(q * 32) << 16);
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        const int cc = col + c * 32;
        if (cc >= P.a.n) break;
        uint4 res[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) res[i] = ahead[i];
        if (c < 3) fetch(cc + 32);
        uint32_t v[32];
        tmem_load32(tb + c * 32, v);
        if (kSplit) {
          // 16-byte pieces of a row are turned by the row's number, so that eight rows lie in different banks
          float4* part = reinterpret_cast<float4*>(smem) + r * 64;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            part[(eh * 32 + c * 8 + i) ^ (r & 7)] =
                make_float4(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]), __uint_as_float(v[4 * i + 2]),
                            __uint_as_float(v[4 * i + 3]));
        } else if (row < P.a.rows) {
          if (cc + 32 <= P.a.n) {
            finish32<kAct>(P.a, row, cc, v, res);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (cc + 4 * i < P.a.n) {
                uint2 b4 = make_uint2(0, 0), r4 = b4;
                if (P.a.bias) b4 = load4(P.a.bias, cc + 4 * i, P.a.n);
                if (P.a.res) r4 = load4(P.a.res + row * P.a.ld_res, cc + 4 * i, P.a.n);
                finish4<kAct>(P.a, row, cc + 4 * i, make_float4(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]),
                                                                __uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3])),
                              b4, r4);
              }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_cluster(free0 + (uint32_t)(acc * 8));
    }
  }

  __syncwarp();
  if (kSplit) {
    tc_fence_before();
    cluster_sync_all();  // all parts are written
    const int nt = first / P.m_tiles, mt = first - nt * P.m_tiles;
    if (warp >= 2 && first < P.tiles && !*abort_flag) {
      // this CTA's share of its half's rows: 128 columns of one row per warp
      const int m0 = mt * 256 + (int)half * 128, h = warp & 1, c = nt * 256 + h * 128 + lane * 4;
      auto at = [&](int r) { return smem_u32(smem) + (uint32_t)(r * 64 + ((h * 32 + lane) ^ (r & 7))) * 16; };
      if (c < P.a.n)
        finish_rows<4>(P, split + ((warp - 2) >> 1) * S, 4 * S, min(128, P.a.rows - m0), m0, c, [&](int r, int k) {
          return ld_cluster_f32x4(map_to_rank(at(r), 2 * k + half));
        });
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();  // no MMA, load, remote arrive or read of the cluster is still in flight
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// ---- few rows --------------------------------------------------------------------------------

template <int T>  // activation rows, rounded up
struct Few {
  static constexpr uint32_t kW = 128 * 128, kA = T * 128, kStage = kW + kA;
  static constexpr int kResident = T <= 64 ? 2 : 1;
  static constexpr int kStages = (kResident == 2 ? 110 * 1024 : 220 * 1024) / (int)kStage;
  static constexpr int kThreads = 256;  // loader, issuer, two to share the finishing, four that read Tensor Memory
  static constexpr uint32_t kTmem = T < 32 ? 32 : T;
  static constexpr size_t kBytes = 1024 + (size_t)kStages * kStage + 256;
  static_assert((size_t)kStages * kStage >= (size_t)T * 128 * 4, "the part reuses the ring");
  static_assert(kThreads == 256, "eight warps finish");
};

__device__ __forceinline__ void umma1(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* m, uint64_t* bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void tmem_load16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

// One cluster of S CTAs per 128 output columns; rank r takes the depth blocks [K r / S, K (r + 1) / S).
template <int T>
__global__ void __launch_bounds__(Few<T>::kThreads, Few<T>::kResident)
    linear_act_few_kernel(const __grid_constant__ Params P) {
  using L = Few<T>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sW = smem;
  uint8_t* sA = smem + L::kStages * L::kW;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kStages * L::kStage);
  uint64_t* empty = full + L::kStages;
  uint64_t* done = empty + L::kStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, S = P.splits;
  const int rank = blockIdx.x % S, nb = blockIdx.x / S;
  const int kb0 = (int)((long long)P.kblocks * rank / S), n = (int)((long long)P.kblocks * (rank + 1) / S) - kb0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&P.a_map);
    tma_prefetch_desc(&P.w_map);
  }
  __syncwarp();
  if (warp == 1) {
    tmem_alloc(tmem_slot, L::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtx wc{P.a.status, abort_flag, kWaitLimitNs};
  grid_dependency_wait();
  allow_dependents();

  if (warp == 0) {
    if (lane == 0) {
      int issued = 0;
      bool ok = true;
      for (int i = 0; i < n; ++i) {
        const int s = i % L::kStages;
        if (!mbar_wait_sleep(&empty[s], ((uint32_t)(i / L::kStages) & 1u) ^ 1u, wc, kSiteEmpty)) {
          ok = false;
          break;
        }
        mbar_arrive_expect_tx(&full[s], L::kStage);
        tma_load_2d(sW + s * L::kW, &P.w_map, &full[s], (kb0 + i) * 64, nb * 128);
        tma_load_2d(sA + s * L::kA, &P.a_map, &full[s], (kb0 + i) * 64, 0);
        issued = i + 1;
      }
      if (!ok) {
        const uint64_t t0 = global_timer_ns();
        for (int i = issued > L::kStages ? issued - L::kStages : 0; i < issued; ++i)
          while (!mbar_try(&full[i % L::kStages], (uint32_t)(i / L::kStages) & 1u) &&
                 global_timer_ns() - t0 < 200000000ull) {
          }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = make_idesc_bf16(128, T, false);
      const uint64_t w0 = make_sdesc_sw128(smem_u32(sW), 16, 1024), a0 = make_sdesc_sw128(smem_u32(sA), 16, 1024);
      for (int i = 0; i < n; ++i) {
        const int s = i % L::kStages;
        if (!mbar_wait(&full[s], (uint32_t)(i / L::kStages) & 1u, wc, kSiteFull)) break;
        tc_fence_after();
        const uint64_t wd = desc_advance(w0, s * (L::kW >> 4)), ad = desc_advance(a0, s * (L::kA >> 4));
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma1(tmem, desc_advance(wd, kk * 2), desc_advance(ad, kk * 2), idesc, i | kk ? 1u : 0u);
        umma_commit(&empty[s]);
      }
      umma_commit(done);  // also after a wait that gave up: every MMA issued has ended when it arrives
    }
  }
  // Every rank leaves its part [row][column] in its own shared memory: all loads have landed and all MMAs read them
  // when `done` arrives.
  float* part = reinterpret_cast<float*>(smem);
  __syncwarp();
  bool ok = mbar_wait_sleep(done, 0, wc, kSiteAccFull);
  ok = __all_sync(0xffffffffu, ok);
  tc_fence_after();
  if (ok && !*abort_flag) {
    // warp w reads the columns [16, 32, ...) of its half, of the rows of its quarter
    const int q = warp & 3;
#pragma unroll 1
    for (int c = (warp >> 2) * 16; c < T && c < P.a.rows; c += 32) {
      uint32_t v[16];
      tmem_load16(tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)c, v);
#pragma unroll
      for (int e = 0; e < 16; ++e) part[(c + e) * 128 + q * 32 + lane] = __uint_as_float(v[e]);
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();
  const int c = nb * 128 + lane * 4;
  if (c < P.a.n && !*abort_flag) {
    // a row per warp, every S-th row a rank's
    const float* at = part + lane * 4;
    auto remote = [&](int r, int k) { return ld_cluster_f32x4(map_to_rank(smem_u32(at + r * 128), k)); };
    if (S == 1)
      finish_rows<1>(P, warp, 8, P.a.rows, 0, c, [&](int r, int) { return *reinterpret_cast<const float4*>(at + r * 128); });
    else if (S <= 4) finish_rows<4>(P, rank + warp * S, 8 * S, P.a.rows, 0, c, remote);
    else finish_rows<8>(P, rank + warp * S, 8 * S, P.a.rows, 0, c, remote);
  }
  __syncwarp();
  cluster_sync_all();  // no rank leaves while another reads its part
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kTmem);
  }
}

// ---- launching -------------------------------------------------------------------------------

bool encode(Params& P, const LinearActArgs& a, uint32_t a_box) {
  memset(&P, 0, sizeof(P));
  P.a = a;
  P.kblocks = (a.k + 63) / 64;
  const uint64_t ad[2] = {(uint64_t)a.k, (uint64_t)a.rows}, wd[2] = {(uint64_t)a.k, (uint64_t)a.n};
  const uint64_t as[1] = {(uint64_t)a.lda * 2}, ws[1] = {(uint64_t)a.ldw * 2};
  const uint32_t ab[2] = {64, a_box}, wb[2] = {64, 128};
  return encode_tmap_bf16(&P.a_map, a.a, 2, ad, as, ab) && encode_tmap_bf16(&P.w_map, a.w, 2, wd, ws, wb);
}

using Kernel = void (*)(Params);

struct Shape {
  Kernel kernel;
  int id, threads, cluster;
  size_t smem;
};

cudaLaunchConfig_t config(const Shape& k, unsigned ctas, cudaStream_t s, cudaLaunchAttribute (&attr)[2]) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3((unsigned)k.threads);
  cfg.dynamicSmemBytes = k.smem;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)k.cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  return cfg;
}

constexpr int kKernels = 16;

cudaError_t raise_smem(const Shape& k) {
  static std::atomic<bool> done[16 * kKernels];  // (device, kernel)
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 16 && done[dev * kKernels + k.id].load(std::memory_order_acquire)) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute((const void*)k.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)k.smem);
  if (e == cudaSuccess && dev < 16) done[dev * kKernels + k.id].store(true, std::memory_order_release);
  return e;
}

// Clusters that the current device runs at once; it depends on which SMs each of its processing clusters
// has.  Asked once per (device, kernel, cluster size).
int clusters_at_once(const Shape& k) {
  static std::atomic<int> known[16 * kKernels * 9];
  int dev = 0, n = 0;
  cudaGetDevice(&dev);
  std::atomic<int>* slot = dev < 16 ? &known[(dev * kKernels + k.id) * 9 + k.cluster] : nullptr;
  if (slot) n = slot->load(std::memory_order_relaxed);
  if (n > 0) return n;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = config(k, (unsigned)k.cluster, nullptr, attr);
  cfg.numAttrs = 1;
  if (raise_smem(k) != cudaSuccess || cudaOccupancyMaxActiveClusters(&n, (const void*)k.kernel, &cfg) != cudaSuccess || n < 1) {
    cudaGetLastError();
    return sm_count() / k.cluster / 2 > 0 ? sm_count() / k.cluster / 2 : 1;
  }
  if (slot) slot->store(n, std::memory_order_relaxed);
  return n;
}

// A split tile is finished by finish4, which looks the activation up.
Shape wide_shape(int act, int splits) {
  static const Kernel kernels[5] = {linear_act_wide_kernel<0, false>, linear_act_wide_kernel<1, false>,
                                    linear_act_wide_kernel<2, false>, linear_act_wide_kernel<3, false>,
                                    linear_act_wide_kernel<4, false>};
  if (splits > 1) return Shape{linear_act_wide_kernel<0, true>, 5, kWideThreads, 2 * splits, kWideBytes};
  return Shape{kernels[act], act, kWideThreads, 2, kWideBytes};
}

template <int T>
Shape few_shape(int splits) {
  return Shape{linear_act_few_kernel<T>, T == 16 ? 6 : T == 32 ? 7 : T == 64 ? 8 : T == 128 ? 9 : 10, Few<T>::kThreads,
               splits, Few<T>::kBytes};
}

Shape few_shape_of(int rows, int splits) {
  return rows <= 16 ? few_shape<16>(splits) : rows <= 32 ? few_shape<32>(splits) : rows <= 64 ? few_shape<64>(splits)
       : rows <= 128 ? few_shape<128>(splits) : few_shape<256>(splits);
}

// Splits of the depth: as many as still run at once, of two blocks at least.  (The clusters that the runtime says run
// at once count one CTA per SM; two are placed where they fit.)
int few_splits(int rows, int n, int kblocks) {
  const int blocks = (n + 127) / 128, most = kblocks / 2;
  int S = most < 8 ? most : 8;
  const int start = S;
  while (S > 1 && blocks > clusters_at_once(few_shape_of(rows, S))) --S;
  if (S < 3 && rows <= 64)  // two CTAs per SM
    for (S = start; S > 1 && blocks > 2 * clusters_at_once(few_shape_of(rows, S));) --S;
  return S > 1 ? S : 1;
}

cudaError_t launch_few(const LinearActArgs& a, cudaStream_t s) {
  Params P;
  if (!encode(P, a, a.rows <= 16 ? 16u : a.rows <= 32 ? 32u : a.rows <= 64 ? 64u : a.rows <= 128 ? 128u : 256u))
    return cudaErrorInvalidValue;
  P.splits = few_splits(a.rows, a.n, P.kblocks);
  const Shape k = few_shape_of(a.rows, P.splits);
  const cudaError_t e = raise_smem(k);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = config(k, (unsigned)((a.n + 127) / 128 * P.splits), s, attr);
  LaunchScope scope(kClsLinearAct, s);
  return cudaLaunchKernelEx(&cfg, k.kernel, P);
}

// Splits only where all tiles' splits run at once, of eight blocks at least.
int wide_splits(int tiles, int kblocks) {
  const int most = kblocks / 8;
  for (int S = most < 4 ? most : 4; S > 1; --S)
    if (tiles <= clusters_at_once(wide_shape(0, S))) return S;
  return 1;
}

cudaError_t launch_wide(const LinearActArgs& a, cudaStream_t s) {
  Params P;
  if (!encode(P, a, 128)) return cudaErrorInvalidValue;
  P.m_tiles = (a.rows + 255) / 256;
  P.tiles = P.m_tiles * ((a.n + 255) / 256);
  P.splits = wide_splits(P.tiles, P.kblocks);
  const Shape k = wide_shape(a.act, P.splits);
  const cudaError_t e = raise_smem(k);
  if (e != cudaSuccess) return e;
  const int most = sm_count() / 2, pairs = P.splits > 1 ? P.tiles * P.splits : P.tiles < most ? P.tiles : most;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = config(k, (unsigned)(2 * pairs), s, attr);
  LaunchScope scope(kClsLinearAct, s);
  return cudaLaunchKernelEx(&cfg, k.kernel, P);
}

}  // namespace

size_t linear_act_parts_bytes(int, int, int) { return 0; }

cudaError_t launch_linear_act(const LinearActArgs& a, cudaStream_t s) {
  if (a.rows <= 128 || (a.rows <= 256 && few_splits(a.rows, a.n, (a.k + 63) / 64) >= 4)) return launch_few(a, s);
  return launch_wide(a, s);
}

}  // namespace dit
