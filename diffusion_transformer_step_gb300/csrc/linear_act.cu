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
// Splits add up through distributed shared memory, in rank order: each CTA sends its part of a row to the CTA that will
// finish it (whose ring has been read), and finishes its own share of the rows from the parts that have come. (Left where
// they were made and fetched by the one that finishes them, every row waited for another SM's memory: 777 x 1544 x 5160 with
// all three 33.9 us, so 26.6.) Wide tiles go by one bulk copy per receiver, 24 KB to 64 KB (stores of 16 bytes: 300 x 1000 x
// 9000 22.3 us, so 21.6).
//
// Loads and MMAs are issued by a thread that elect.sync chose: chosen by its lane number, the compiler guards every such
// instruction against more than one, and a block of depth takes 0.28 us whatever its tile's columns (elected: 0.27, 0.20 and
// 0.14 us for 256, 192 and 128).  Then loads bound the narrow tiles, and all where rows do not start on lines of 128 bytes:
// 777 x 1544 x 5120 16.5 us, 5152 19.0, 5136 20.1, 5160 24.6.
//
// Measured (bursts of twenty calls on different weights): 8192 x 12288 x 4096 432 to 438 us, 1880 to 1905 TFLOP/s (0.97 to 0.98
// of the measured burst); call after call 505 to 530, at the clocks that power leaves, with any epilogue (0.93 of the
// measured sustained rate). 4096 x 4096 x 4096 76 to 78 us, 512 x 4096 x 4096 15.4; 1 x 12288 x 4096 18.7 (5.4 TB/s of weights),
// 1 x 2560 x 4096 7.1, 64 x 4096 x 4096 11.4, 777 x 1544 x 5160 24.6 without epilogue. A call has about 3.5 us besides its
// loads (launch, first load, last rows), and a split of wide tiles 5.5 more.
// Measured and left: accumulators through shared memory to whole lines of the output, at six stages instead of seven (8192 x
// 12288 x 4096 455 -> 476 us: the MMAs and the loads take all of shared memory's cycles); the first weights sent to L2 before the
// kernel before has ended (1 x 2560 x 4096 7.3 -> 7.9: every line crosses the copy unit twice); two CTAs of three stages per
// SM for 128 rows (11.8 -> 13.8); a first pass through the finishing code while the loads are on their way (no change); a
// tile's residual sent to L2 while it is worked on, or fetched two pieces ahead (4096 x 4096 x 1024 31.4 -> 33.4 and 32.7).
#include <math.h>

#include <atomic>

#include "cta_pair.cuh"
#include "linear_act_plan.h"
#include "runtime.h"

namespace dit {

namespace {

enum : uint32_t { kSiteEmpty = 0xa01, kSiteFull, kSiteAccEmpty, kSiteAccFull, kSiteParts };

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

// Two values at a time: packed fp32 arithmetic, exponentials and reciprocals of the special unit. Where the reciprocal is below fp32's
// normal numbers (z below -87) an output is zero instead of under 2^-119.
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

template <int kAct, int N>
__device__ __forceinline__ void activate_all(float2 (&z)[N], int act) {
  if constexpr (kAct != kAnyAct) {
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = activate<kAct>(z[i]);
  } else if (act != 0) {
    if (act == 1) activate_all<1>(z, 1);
    else if (act == 2) activate_all<2>(z, 2);
    else if (act == 3) activate_all<3>(z, 3);
    else activate_all<4>(z, 4);
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

// Sums v of columns [c, c + 4) of N rows r[i] to the output, of those below `rows`; bias and res as load4 gives them.
template <int kAct, int N>
__device__ __forceinline__ void finish4(const LinearActArgs& p, const int (&r)[N], int rows, int m0, int c,
                                        const float4 (&v)[N], uint2 bias, const uint2 (&res)[N]) {
  const bool whole = c + 4 <= p.n;
  float2 z[2 * N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    z[2 * i] = make_float2(v[i].x, v[i].y);
    z[2 * i + 1] = make_float2(v[i].z, v[i].w);
    if (p.bias) {
      z[2 * i] = __fadd2_rn(z[2 * i], unpack_bf16x2(bias.x));
      z[2 * i + 1] = __fadd2_rn(z[2 * i + 1], unpack_bf16x2(bias.y));
    }
  }
  activate_all<kAct>(z, p.act);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (r[i] >= rows) continue;
    float2 lo = z[2 * i], hi = z[2 * i + 1];
    if (p.res) {
      lo = __fadd2_rn(lo, unpack_bf16x2(res[i].x));
      hi = __fadd2_rn(hi, unpack_bf16x2(res[i].y));
    }
    const long long at = (long long)(m0 + r[i]) * p.ld_out + c;
    if (p.out_f32) {
      float* o = reinterpret_cast<float*>(p.out) + at;
      if (whole) {
        *reinterpret_cast<float4*>(o) = make_float4(lo.x, lo.y, hi.x, hi.y);
      } else {
        o[0] = lo.x;
        if (c + 1 < p.n) o[1] = lo.y;
        if (c + 2 < p.n) o[2] = hi.x;
      }
    } else {
      bf16* o = reinterpret_cast<bf16*>(p.out) + at;
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
}

// Four lanes that hold four pieces of a row each, to each holding one piece of all four rows, and back.
__device__ __forceinline__ void transpose4(uint4 (&x)[4], int lane) {
#pragma unroll
  for (int by = 1; by < 4; by *= 2) {
    const bool up = lane & by;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & by) continue;
      uint4 &lo = x[i], &hi = x[i + by];
      const uint4 give = up ? lo : hi;
      uint4 take;
      take.x = __shfl_xor_sync(0xffffffffu, give.x, by);
      take.y = __shfl_xor_sync(0xffffffffu, give.y, by);
      take.z = __shfl_xor_sync(0xffffffffu, give.z, by);
      take.w = __shfl_xor_sync(0xffffffffu, give.w, by);
      if (up) lo = take;
      else hi = take;
    }
  }
}

// 32 columns [c, c + 32) of the warp's rows, row `row` of this lane's, all below n. Memory is read and written with four
// lanes to a row's 64 bytes, eight rows at once, which takes as many lines of an instruction as rows: 4096 x 4096 x 1024
// 30.4 -> 25.0 us, with bias, GELU and residual 47.4 -> 40.0, to fp32 48.7 -> 36.7 (each lane its own row before). res[i] is
// piece lane % 4 of the residual of the i-th of the four rows, bias what the columns add.
template <int kAct>
__device__ __forceinline__ void finish32(const LinearActArgs& p, int row, int c, const uint32_t (&v)[32], const uint4 (&bias)[4],
                                         uint4 (&res)[4], int lane) {
  auto eight = [](const uint4& u, float2 (&f)[4]) {
    f[0] = unpack_bf16x2(u.x), f[1] = unpack_bf16x2(u.y), f[2] = unpack_bf16x2(u.z), f[3] = unpack_bf16x2(u.w);
  };
  float2 o[16];
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    float2 b[4];
    if (p.bias) eight(bias[g], b);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 z = make_float2(__uint_as_float(v[g * 8 + 2 * i]), __uint_as_float(v[g * 8 + 2 * i + 1]));
      if (p.bias) z = __fadd2_rn(z, b[i]);
      o[g * 4 + i] = activate<kAct>(z);
    }
  }
  if (p.res) {
    transpose4(res, lane);
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      float2 x[4];
      eight(res[g], x);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[g * 4 + i] = __fadd2_rn(o[g * 4 + i], x[i]);
    }
  }
  const int r0 = row - (lane & 3);
  if (p.out_f32) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint4 x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[i] = make_uint4(__float_as_uint(o[8 * h + 2 * i].x), __float_as_uint(o[8 * h + 2 * i].y),
                          __float_as_uint(o[8 * h + 2 * i + 1].x), __float_as_uint(o[8 * h + 2 * i + 1].y));
      transpose4(x, lane);
      float* dst = reinterpret_cast<float*>(p.out) + r0 * p.ld_out + c + h * 16 + (lane & 3) * 4;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (r0 + i < p.rows) *reinterpret_cast<uint4*>(dst + i * p.ld_out) = x[i];
    }
  } else {
    uint4 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[i] = make_uint4(pack_bf16x2(o[4 * i].x, o[4 * i].y), pack_bf16x2(o[4 * i + 1].x, o[4 * i + 1].y),
                        pack_bf16x2(o[4 * i + 2].x, o[4 * i + 2].y), pack_bf16x2(o[4 * i + 3].x, o[4 * i + 3].y));
    transpose4(x, lane);
    bf16* dst = reinterpret_cast<bf16*>(p.out) + r0 * p.ld_out + c + (lane & 3) * 8;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (r0 + i < p.rows) *reinterpret_cast<uint4*>(dst + i * p.ld_out) = x[i];
  }
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void st_cluster(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// Of the rows first, first + stride, ... below `rows` (of the output: m0 further) every step-th from number i0 on, four
// columns from c on per thread; part(i, k) is what split k has sent of row number i, added in split order. R rows go
// side by side, the residual of the next R ahead. A loop that runs a few times waits for its code as much as for its data: 1
// x 2560 x 64 with one, two, four rows at once 2.3, 2.5, 2.7 us, 64 x 4096 x 4096 with everything 12.5, 12.1, 12.8, 777 x 1544 x
// 5160 with everything 30.9, 28.0, 27.3 (26.6 with the steps after this one).
template <int K, int R, typename Part>
__device__ __forceinline__ void finish_rows(const Params& P, int i0, int step, int first, int stride, int rows, int m0, int c,
                                            Part part) {
  const LinearActArgs& p = P.a;
  const uint2 none = make_uint2(0, 0), bias = p.bias ? load4(p.bias, c, p.n) : none;
  auto residual = [&](int r) { return r < rows && p.res ? load4(p.res + (long long)(m0 + r) * p.ld_res, c, p.n) : none; };
  auto sum = [&](int i) {
    float4 x = part(i, 0);
#pragma unroll
    for (int k = 1; k < K; ++k)
      if (k < P.splits) {
        const float4 v = part(i, k);
        x.x += v.x, x.y += v.y, x.z += v.z, x.w += v.w;
      }
    return x;
  };
  const int r0 = first + i0 * stride, by = step * stride;
  uint2 res[R];
#pragma unroll
  for (int u = 0; u < R; ++u) res[u] = residual(r0 + u * by);
#pragma unroll 1
  for (int r = r0, i = i0; r < rows; r += R * by, i += R * step) {
    int all[R];
    float4 v[R];
    uint2 now[R];
#pragma unroll
    for (int u = 0; u < R; ++u) {
      all[u] = r + u * by;
      v[u] = sum(r + u * by < rows ? i + u * step : i);
      now[u] = res[u];
      res[u] = residual(r + (R + u) * by);
    }
    finish4<kAnyAct>(p, all, rows, m0, c, v, bias, now);
  }
}

// ---- many rows -------------------------------------------------------------------------------

// One thread of a converged warp, so chosen that the compiler knows that it is one.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}

constexpr int kWideThreads = 320;
template <int BN>  // columns of a pair's tile: 128, 192 or 256
struct Wide {
  static constexpr uint32_t kA = 128 * 128, kW = BN / 2 * 128, kStage = kA + kW;
  static constexpr int kStages = 229376 / (int)kStage;
  static constexpr size_t kBytes = 1024 + (size_t)kStages * kStage + 256;
  static_assert(kStages * kStage >= (128 + 96) * BN * 4, "the splits' parts, at most of four, reuse the ring");
};

// Pair `pair` of a cluster (rank = 2 pair + half) takes the depth blocks [K pair / S, K (pair + 1) / S) of its cluster's
// tiles; with splits a cluster has one tile.  Roles as in the step's products: warp 0 loads, warp 1 issues (the
// pair's first CTA), warps 2 to 9 finish, one thread per row of 128 columns.
template <int kAct, bool kSplit, int BN>
__global__ void __launch_bounds__(kWideThreads, 1) linear_act_wide_kernel(const __grid_constant__ Params P) {
  using L = Wide<BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sW = smem + L::kStages * L::kA;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kStages * L::kStage);
  uint64_t* empty = full + L::kStages;
  uint64_t* acc_full = empty + L::kStages;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;
  uint64_t* come = drain + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(come + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t crank = cta_rank(), leader = crank & ~1u, half = crank & 1u;
  const int S = kSplit ? P.splits : 1, split = kSplit ? (int)(crank >> 1) : 0;
  const int first = blockIdx.x / (2 * S), step = gridDim.x / (2 * S);
  const int kb0 = kSplit ? (int)((long long)P.kblocks * split / S) : 0;
  const int kb1 = kSplit ? (int)((long long)P.kblocks * (split + 1) / S) : P.kblocks;
  // Splits: split s finishes the rows s, s + S, ... of each half, their number, and room for it.
  [[maybe_unused]] const int per = (127 + S) / S, m0 = first % P.m_tiles * 256 + (int)half * 128;
  [[maybe_unused]] auto share = [&](int s) { return (max(min(128, P.a.rows - m0), 0) + S - 1 - s) / S; };
  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 16);
    }
    mbar_init(drain, 1);
    mbar_init(come, 1);
    *abort_flag = 0;
    fence_mbar_init();
    if (kSplit) mbar_arrive_expect_tx(come, (uint32_t)((S - 1) * share(split) * BN * 4));
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
    if (elect_one()) {
      uint32_t stage = 0, phase = 0;
      long long issued = 0;
      bool ok = true;
      for (int t = first; t < P.tiles && ok; t += step) {
        const int nt = t / P.m_tiles, mt = t - nt * P.m_tiles;
        const int arow = mt * 256 + (int)half * 128, wrow = nt * BN + (int)half * (BN / 2);
        for (int kb = kb0; kb < kb1; ++kb) {
          if (mt == 0 && kb + 8 < kb1) pf_l2(&P.w_map, (kb + 8) * 64, wrow);  // one prefetcher per weight column
          if (!mbar_wait_sleep(&empty[stage], phase ^ 1u, wc, kSiteEmpty)) {
            ok = false;
            break;
          }
          const uint32_t fb = map_to_rank(smem_u32(&full[stage]), leader);
          if (half == 0) mbar_arrive_expect_tx(&full[stage], 2 * L::kStage);
          tma2_2sm(sA + stage * L::kA, &P.a_map, fb, kb * 64, arow);
          tma2_2sm(sW + stage * L::kW, &P.w_map, fb, kb * 64, wrow);
          ++issued;
          if (++stage == L::kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok && half == 0) {
        // Unwinding: let copies in flight land (bounded) before the pair exits.
        const long long outstanding = issued < L::kStages ? issued : L::kStages;
        for (long long i = 0; i < outstanding; ++i) {
          if (stage == 0) {
            stage = L::kStages;
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
    if (half == 0 && elect_one()) {
      const uint32_t idesc = make_idesc_bf16(256, BN, false);
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
          const uint64_t ad = desc_advance(a0, stage * (L::kA >> 4)), wd = desc_advance(w0, stage * (L::kW >> 4));
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma2(tmem + (uint32_t)(acc * BN), desc_advance(ad, kk * 2), desc_advance(wd, kk * 2), idesc,
                  kb > kb0 || kk ? 1u : 0u);
          commit(&empty[stage]);
          if (++stage == L::kStages) {
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
    const int q = warp & 3, eh = (warp - 2) >> 2;  // rows [32 q, 32 q + 32) of this CTA, half the columns
    const int r = q * 32 + lane;
    if constexpr (kSplit) {
      bool ok = mbar_wait_sleep(&acc_full[0], 0, wc, kSiteAccFull);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
      cluster_arrive();  // this CTA's ring has been read
      // Rows by the split that finishes them, 16-byte pieces turned by the row, so that eight rows lie in different banks.
      float4* mine = reinterpret_cast<float4*>(smem) + ((r % S) * per + r / S) * (BN / 4);
#pragma unroll 1
      for (int c = 0; c < BN / 64 && ok; ++c) {
        uint32_t v[32];
        tmem_load32(tmem + (uint32_t)(eh * (BN / 2) + c * 32) + ((uint32_t)(q * 32) << 16), v);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          mine[(eh * (BN / 8) + c * 8 + i) ^ (r & 7)] = make_float4(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]),
                                                                   __uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3]));
      }
      fence_proxy_async_smem();
      cluster_wait();  // every CTA's ring has been read
      asm volatile("bar.sync 1, 256;" ::: "memory");
      const int to = warp - 2;
      if (to < S && to != split && lane == 0 && share(to) > 0) {
        const uint32_t dst = smem_u32(smem) + (uint32_t)(S * per + (split < to ? split : split - 1) * per) * (BN * 4);
        asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                         map_to_rank(dst, (uint32_t)(2 * to) + half)),
                     "r"(smem_u32(smem) + (uint32_t)(to * per) * (BN * 4)), "r"((uint32_t)(share(to) * BN * 4)),
                     "r"(map_to_rank(smem_u32(come), (uint32_t)(2 * to) + half))
                     : "memory");
      }
    } else {
      const uint32_t free0 = map_to_rank(smem_u32(acc_empty), leader);
      int local = 0;
      for (int t = first; t < P.tiles; t += step, ++local) {
        const int acc = local & 1;
        const int nt = t / P.m_tiles, mt = t - nt * P.m_tiles;
        const int row = mt * 256 + (int)half * 128 + r, col = nt * BN + eh * (BN / 2);
        // the residual's pieces one ahead, the first before the accumulator is waited for
        uint4 ahead[4];
        auto fetch = [&](int c) {
          if (!P.a.res || c + 32 > P.a.n) return;
          const int r0 = row - (lane & 3);
          const bf16* src = P.a.res + r0 * P.a.ld_res + c + (lane & 3) * 8;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            ahead[i] = r0 + i < P.a.rows ? *reinterpret_cast<const uint4*>(src + i * P.a.ld_res) : make_uint4(0u, 0u, 0u, 0u);
        };
        fetch(col);
        bool ok = mbar_wait_sleep(&acc_full[acc], (uint32_t)(local >> 1) & 1u, wc, kSiteAccFull);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint32_t tb = tmem + (uint32_t)(acc * BN + eh * (BN / 2)) + ((uint32_t)(q * 32) << 16);
#pragma unroll 1
        for (int c = 0; c < BN / 64; ++c) {
          const int cc = col + c * 32;
          if (cc >= P.a.n) break;
          uint4 res[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) res[i] = ahead[i];
          if (c + 1 < BN / 64) fetch(cc + 32);
          uint4 bias[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (P.a.bias && cc + 32 <= P.a.n) bias[i] = __ldg(reinterpret_cast<const uint4*>(P.a.bias + cc + i * 8));
          uint32_t v[32];
          tmem_load32(tb + c * 32, v);
          if (cc + 32 <= P.a.n) {
            finish32<kAct>(P.a, row, cc, v, bias, res, lane);
          } else if (row < P.a.rows) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (cc + 4 * i < P.a.n) {
                uint2 b4 = make_uint2(0, 0), r4 = b4;
                if (P.a.bias) b4 = load4(P.a.bias, cc + 4 * i, P.a.n);
                if (P.a.res) r4 = load4(P.a.res + row * P.a.ld_res, cc + 4 * i, P.a.n);
                const int r1[1] = {row};
                const uint2 x1[1] = {r4};
                const float4 f[1] = {make_float4(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]),
                                                 __uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3]))};
                finish4<kAct>(P.a, r1, P.a.rows, 0, cc + 4 * i, f, b4, x1);
              }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_cluster(free0 + (uint32_t)(acc * 8));
      }
    }
  }

  __syncwarp();
  auto free_tmem = [&] {
    if (warp == 1) {
      tc_fence_after();
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
  };
  if constexpr (kSplit) {
    if (warp < 2) {
      cluster_arrive();
      cluster_wait();
    }
    const int nt = first / P.m_tiles;
    if (warp >= 2) {
      bool ok = mbar_wait_sleep(come, 0, wc, kSiteParts);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_before();
      cluster_arrive();  // what was sent here has come; no load or remote arrive is still in flight, with the others'
      // this pair's share of its half's rows: half the columns of one row per warp
      const int piece = (warp & 1) * (BN / 8) + lane, c = nt * BN + piece * 4;
      const float4* parts = reinterpret_cast<const float4*>(smem);
      if (ok && !*abort_flag && lane < BN / 8 && c < P.a.n && P.a.rows > m0 + split)
        finish_rows<4, 4>(P, (warp - 2) >> 1, 4, split, S, min(128, P.a.rows - m0), m0, c, [&](int i, int k) {
          const int slot = (k == split ? split : S + (k < split ? k : k - 1)) * per + i;
          return parts[slot * (BN / 4) + (piece ^ ((split + i * S) & 7))];
        });
      __syncwarp();
    } else {
      tc_fence_before();
      cluster_arrive();
    }
    cluster_wait();
    free_tmem();
  } else {
    tc_fence_before();
    cluster_sync_all();  // no MMA, load or remote arrive of the pair is still in flight
    free_tmem();
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
  static_assert((size_t)kStages * kStage >= (size_t)(T + 7) * 128 * 4, "the parts reuse the ring");
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
    if (elect_one()) {
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
    if (elect_one()) {
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
  // All loads have landed and all MMAs read them when `done` arrives; then, over the cluster, no ring is in use any more.
  // Every rank sends row r of its part to rank r % S, which finishes it.
  float* parts = reinterpret_cast<float*>(smem);  // [split][row / S][column]
  const int per = (T + S - 1) / S;
  __syncwarp();
  bool ok = mbar_wait_sleep(done, 0, wc, kSiteAccFull);
  ok = __all_sync(0xffffffffu, ok);
  tc_fence_after();
  if (S > 1) cluster_sync_all();
  if (ok && !*abort_flag) {
    // warp w reads the columns [16, 32, ...) of its half, of the rows of its quarter
    const int q = warp & 3;
#pragma unroll 1
    for (int c = (warp >> 2) * 16; c < T && c < P.a.rows; c += 32) {
      uint32_t v[16];
      tmem_load16(tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)c, v);
      if (S == 1) {
#pragma unroll
        for (int e = 0; e < 16; ++e) parts[(c + e) * 128 + q * 32 + lane] = __uint_as_float(v[e]);
      } else {
        int to = c % S, at = rank * per + c / S;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          if (c + e < P.a.rows) st_cluster(map_to_rank(smem_u32(parts + at * 128 + q * 32 + lane), to), __uint_as_float(v[e]));
          if (++to == S) to = 0, ++at;
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  if (S > 1) cluster_sync_all();  // all parts have come
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kTmem);
  }
  const int c = nb * 128 + lane * 4;
  if (c < P.a.n && !*abort_flag) {
    // a row per warp, every S-th row a rank's
    auto part = [&](int i, int k) { return *reinterpret_cast<const float4*>(parts + (k * per + i) * 128 + lane * 4); };
    constexpr int R = T <= 16 ? 1 : 2;
    if (S == 1) finish_rows<1, R>(P, warp, 8, 0, 1, P.a.rows, 0, c, part);
    else finish_rows<8, R>(P, warp, 8, rank, S, P.a.rows, 0, c, part);
  }
}

// ---- launching -------------------------------------------------------------------------------

bool encode(Params& P, const LinearActArgs& a, uint32_t a_box, uint32_t w_box) {
  memset(&P, 0, sizeof(P));
  P.a = a;
  P.kblocks = (a.k + 63) / 64;
  const uint64_t ad[2] = {(uint64_t)a.k, (uint64_t)a.rows}, wd[2] = {(uint64_t)a.k, (uint64_t)a.n};
  const uint64_t as[1] = {(uint64_t)a.lda * 2}, ws[1] = {(uint64_t)a.ldw * 2};
  const uint32_t ab[2] = {64, a_box}, wb[2] = {64, w_box};
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

constexpr int kKernels = 22;

cudaError_t raise_smem(const Shape& k) {
  static std::atomic<bool> done[16 * kKernels];  // (device, kernel)
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 16 && done[dev * kKernels + k.id].load(std::memory_order_acquire)) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute((const void*)k.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)k.smem);
  if (e == cudaSuccess && dev < 16) done[dev * kKernels + k.id].store(true, std::memory_order_release);
  return e;
}

// A split tile is finished by finish4, which looks the activation up.
template <int BN>
Shape wide_shape(int act, int splits) {
  static const Kernel kernels[5] = {linear_act_wide_kernel<0, false, BN>, linear_act_wide_kernel<1, false, BN>,
                                    linear_act_wide_kernel<2, false, BN>, linear_act_wide_kernel<3, false, BN>,
                                    linear_act_wide_kernel<4, false, BN>};
  constexpr int id = BN == 256 ? 0 : BN == 192 ? 6 : 12;
  if (splits > 1) return Shape{linear_act_wide_kernel<0, true, BN>, id + 5, kWideThreads, 2 * splits, Wide<BN>::kBytes};
  return Shape{kernels[act], id + act, kWideThreads, 2, Wide<BN>::kBytes};
}

Shape wide_shape_of(int bn, int act, int splits) {
  return bn == 256 ? wide_shape<256>(act, splits) : bn == 192 ? wide_shape<192>(act, splits) : wide_shape<128>(act, splits);
}

template <int T>
Shape few_shape(int splits) {
  return Shape{linear_act_few_kernel<T>, T == 16 ? 18 : T == 32 ? 19 : T == 64 ? 20 : 21, Few<T>::kThreads, splits,
               Few<T>::kBytes};
}

Shape few_shape_of(int rows, int splits) {
  return rows <= 16 ? few_shape<16>(splits) : rows <= 32 ? few_shape<32>(splits) : rows <= 64 ? few_shape<64>(splits)
                                                                                   : few_shape<128>(splits);
}

cudaError_t launch_few(const LinearActArgs& a, LinearActPlan plan, cudaStream_t s) {
  Params P;
  if (!encode(P, a, a.rows <= 16 ? 16u : a.rows <= 32 ? 32u : a.rows <= 64 ? 64u : 128u, 128))
    return cudaErrorInvalidValue;
  P.splits = plan.splits;
  const Shape k = few_shape_of(a.rows, P.splits);
  const cudaError_t e = raise_smem(k);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = config(k, (unsigned)((a.n + 127) / 128 * P.splits), s, attr);
  LaunchScope scope(kClsLinearAct, s);
  return cudaLaunchKernelEx(&cfg, k.kernel, P);
}

cudaError_t launch_wide(const LinearActArgs& a, LinearActPlan plan, cudaStream_t s) {
  Params P;
  if (!encode(P, a, 128, (uint32_t)plan.bn / 2)) return cudaErrorInvalidValue;
  P.m_tiles = (a.rows + 255) / 256;
  P.tiles = P.m_tiles * ((a.n + plan.bn - 1) / plan.bn);
  P.splits = plan.splits;
  const Shape k = wide_shape_of(plan.bn, a.act, P.splits);
  const cudaError_t e = raise_smem(k);
  if (e != cudaSuccess) return e;
  const int most = sm_count() / 2, pairs = P.splits > 1 ? P.tiles * P.splits : P.tiles < most ? P.tiles : most;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = config(k, (unsigned)(2 * pairs), s, attr);
  LaunchScope scope(kClsLinearAct, s);
  return cudaLaunchKernelEx(&cfg, k.kernel, P);
}

}  // namespace

cudaError_t launch_linear_act(const LinearActArgs& a, cudaStream_t s) {
  const bool lines = (a.lda | a.ldw) % 64 == 0 && ((reinterpret_cast<uintptr_t>(a.a) | reinterpret_cast<uintptr_t>(a.w)) & 127) == 0;
  const LinearActPlan plan = linear_act_plan(a.rows, a.n, (a.k + 63) / 64, lines);
  return plan.bn == 0 ? launch_few(a, plan, s) : launch_wide(a, plan, s);
}

}  // namespace dit
