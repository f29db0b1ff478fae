// e4m3 operands with one fp32 scale per block of 128: quantisation and the product
//   out[r, c] = sum_b sa[r, b] sw[c / 128, b] (a_b . w_b).
//
// The scales are any fp32 numbers, so the tensor cores sum one block of 128 depths at a time into
// Tensor Memory and the threads that own an accumulator row fold it into fp32 registers:
// acc += part * (sa sw), one packed fp32x2 FMA per two columns.  A block's MMAs run while the
// blocks before it are folded.
//
//   linear_fp8_wide_kernel   more than 64 rows: persistent CTA pairs, 256 x 128 tiles, the operands'
//                            ring of the bf16 product (128-byte rows hold one block of depth).
//   linear_fp8_few_kernel    up to 64 rows, where reading the weights bounds the time: the weights'
//                            rows take the MMA's 128-row side and the few activation rows its column
//                            side, the depth split over a cluster whose CTAs add their parts
//                            through distributed shared memory, in rank order.  (128 rows so: 16.9 us
//                            at 8192 x 4096, as wide tiles 12.7.)
//
// On random values, with the pass that quantises the rows, the wide kernel takes 362 us at 8192 x 12288 x 4096
// in a burst of twenty (the product 349, 2.36 PFLOP/s) and 386 to 395 call after call for a second, at the
// clocks that power leaves (2.1 PFLOP/s with the quantising); 79 us at 4096 x 4864 x 4096 in a burst
// (73): 0.6 of the e4m3 rate (twice the measured bf16 burst).  A 128-column block takes ~546 cycles: the MMAs'
// operands and the loads take 437 of them from shared memory at 128 bytes per cycle, and the fold's scale
// loads, one line per row, share that path.  256-column tiles read 40 % less shared memory per product but leave two
// accumulators, between which commit, fold, hand-back and issue (~1900 cycles) do not hide.
//
// Forms were compared on products of zeros, which draw less power and do not wait for the clock.  The
// product of 8192 x 12288 x 4096 took 339 us so, 290 without its fold, and 215 in 256-column tiles without
// theirs (3.8 PFLOP/s); measured and left: 256 columns 363, 160 columns in three accumulators 356, one CTA per
// tile with the weights by multicast 353, scales 16 blocks ahead through shared memory 390, scales of a block in
// one line 375.
#include <cuda_fp8.h>

#include <atomic>

#include "cta_pair.cuh"
#include "runtime.h"

namespace dit {

namespace {

constexpr float kAmaxFloor = 448.0f * 0x1p-118f;  // keeps 448 / max finite
constexpr int kSMs = 152;

// ---- quantisation ------------------------------------------------------------------------

__device__ __forceinline__ float absmax8(const uint4& u, float m) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = unpack_bf16x2(w[j]);
    m = fmaxf(m, fmaxf(fabsf(f.x), fabsf(f.y)));
  }
  return m;
}

__device__ __forceinline__ uint2 codes8(const uint4& u, float inv) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  uint32_t q[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = unpack_bf16x2(w[j]);
    q[j] = __nv_cvt_float2_to_fp8x2(make_float2(f.x * inv, f.y * inv), __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
}

// A scale per row and 128 columns: eight threads of 16 values each per block, so a row's read
// and write are whole 16-byte accesses of neighbouring threads.  blockDim = (8 x blocks of one
// row, up to 256; rows).  8192 x 4096: 16.7 us, 6.05 TB/s; 512 x 4096, which L2 holds, 2.1 us.
__global__ void __launch_bounds__(256) quantize_row_blocks_kernel(const bf16* __restrict__ x, long long ld, int rows,
                                                                  int cols, uint8_t* __restrict__ q,
                                                                  float* __restrict__ scale) {
  grid_dependency_wait();
  allow_dependents();
  const int row = blockIdx.x * blockDim.y + threadIdx.y;
  const int c = (blockIdx.y * blockDim.x + threadIdx.x) * 16;
  const bool ok = row < rows && c < cols;
  uint4 u[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
  if (ok) {
    const uint4* p = reinterpret_cast<const uint4*>(x + row * ld + c);
    u[0] = p[0];
    u[1] = p[1];
  }
  float m = absmax8(u[1], absmax8(u[0], kAmaxFloor));
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (!ok) return;
  const float inv = 448.0f / m;
  const uint2 lo = codes8(u[0], inv), hi = codes8(u[1], inv);
  *reinterpret_cast<uint4*>(q + (long long)row * cols + c) = make_uint4(lo.x, lo.y, hi.x, hi.y);
  if (c % 128 == 0) scale[(long long)row * ((cols + 127) / 128) + c / 128] = m / 448.0f;
}

// A scale per 128 x 128 block: one CTA each, the block held in registers.  12288 x 4096: 24.9 us, 6.05 TB/s.
__global__ void __launch_bounds__(256) quantize_square_blocks_kernel(const bf16* __restrict__ x, long long ld, int rows,
                                                                     int cols, uint8_t* __restrict__ q,
                                                                     float* __restrict__ scale) {
  grid_dependency_wait();
  allow_dependents();
  const int c = blockIdx.y * 128 + (threadIdx.x & 15) * 8, r0 = blockIdx.x * 128 + (threadIdx.x >> 4);
  uint4 u[8];
  float m = kAmaxFloor;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    u[i] = make_uint4(0, 0, 0, 0);
    if (r0 + 16 * i < rows && c < cols) u[i] = *reinterpret_cast<const uint4*>(x + (r0 + 16 * i) * ld + c);
    m = absmax8(u[i], m);
  }
  __shared__ float red[8];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, red[i]);
  const float inv = 448.0f / m;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (r0 + 16 * i < rows && c < cols)
      *reinterpret_cast<uint2*>(q + (long long)(r0 + 16 * i) * cols + c) = codes8(u[i], inv);
  if (threadIdx.x == 0) scale[(long long)blockIdx.x * gridDim.y + blockIdx.y] = m / 448.0f;
}

// ---- product, many rows ------------------------------------------------------------------

enum : uint32_t { kSiteEmpty = 0x701, kSiteFull, kSiteAccEmpty, kSiteAccFull };

struct alignas(64) Params {
  CUtensorMap a_map, w_map, out_map;  // out_map: the output, or the splits' parts
  LinearFp8Args a;
  int kblocks, m_tiles, items, splits;
};

// Work item t of the wide kernel: a tile, and a run [kb0, kb1) of its blocks of depth.
struct Item {
  int mt, nt, split, kb0, kb1;
};
template <bool kSplit>
__device__ __forceinline__ Item item_of(const Params& P, int t) {
  Item it;
  if (!kSplit) {
    it.nt = t / P.m_tiles;
    it.mt = t - it.nt * P.m_tiles;
    it.split = it.kb0 = 0;
    it.kb1 = P.kblocks;
    return it;
  }
  const int tile = t / P.splits;
  it.split = t - tile * P.splits;
  it.nt = tile / P.m_tiles;
  it.mt = tile - it.nt * P.m_tiles;
  it.kb0 = (int)((long long)P.kblocks * it.split / P.splits);
  it.kb1 = (int)((long long)P.kblocks * (it.split + 1) / P.splits);
  return it;
}

// Arrival at the leader's barrier that publishes no memory: the accumulator's reads are complete
// (tcgen05.wait::ld) and ordered by tcgen05.fence.  With release semantics at cluster scope each of the
// sixteen arrivals per block waited ~600 cycles for a memory barrier.
__device__ __forceinline__ void arrive_cluster_relaxed(uint32_t caddr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(caddr) : "memory");
}

// A box of the output from shared memory (128-byte swizzle), and the wait until every box of this
// thread has been read out of it.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* m, const void* src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void tma_store_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

// One block of depth: D = A W^T over four K = 32 MMAs, descriptors 32 bytes apart, in one statement.
__device__ __forceinline__ void umma2_f8x4(uint32_t d, uint64_t a, uint64_t w, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred pf, pt;\n\t.reg .b64 a1, a2, a3, w1, w2, w3;\n\t"
      "setp.ne.b32 pf, %4, %4;\n\tsetp.eq.b32 pt, %4, %4;\n\t"
      "add.s64 a1, %1, 2;\n\tadd.s64 w1, %2, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 w2, %2, 4;\n\t"
      "add.s64 a3, %1, 6;\n\tadd.s64 w3, %2, 6;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, pf;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a1, w1, %3, pt;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a2, w2, %3, pt;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a3, w3, %3, pt;\n\t}" ::"r"(d),
      "l"(a), "l"(w), "r"(idesc), "r"(0)
      : "memory");
}

// A stage and an accumulator always come back to the same issuer (both counts are even), whose
// parity waits are thereby never more than one phase behind.
constexpr int kIssuers = 2;

struct Wide {
  static constexpr int BN = 128;
  static constexpr uint32_t kA = 128 * 128, kW = BN / 2 * 128, kStage = kA + kW;
  static constexpr int kStages = 8;
  static constexpr int kBufs = 512 / BN;  // accumulators in Tensor Memory
  // folding warps: one per 32 rows and 64 columns, so that accumulators leave room in the registers
  static constexpr int kWarps = BN / 16, kThreads = 128 + kWarps * 32;
  // behind the ring: 4 KB per folding warp, 32 rows x 64 columns of output on their way to a TMA store
  static constexpr uint32_t kOut = kStages * kStage, kBar = kOut + kWarps * 4096;
  static constexpr size_t kBytes = 1024 + kBar + 256;
  static_assert(kStages % kIssuers == 0 && kBufs % kIssuers == 0, "see kIssuers");
};

// Warp 0 loads, warps 1 and 2 issue (leader CTA) every second block of depth each, the others from
// warp 4 fold and store, BN / 64 per row quarter with 64 columns each.  An issuing thread needs
// ~500 cycles per block for its waits, MMAs and commit, more than the MMAs themselves: two of them take a product
// of zeros of 8192 x 12288 x 4096 from 506 to 346 us, sleeping instead of spinning folders to 339.  Per block
// there is one commit, on the accumulator; the stage it frees is handed back by a folding thread of each CTA.
template <bool kSplit>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Wide::kThreads, 1)
    linear_fp8_wide_kernel(const __grid_constant__ Params P) {
  using L = Wide;
  constexpr int BN = L::BN;
  constexpr int kCols = 64;  // columns of a folding warp
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sW = smem + L::kStages * L::kA;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint64_t* empty = full + L::kStages;
  uint64_t* acc_full = empty + L::kStages;
  uint64_t* acc_empty = acc_full + L::kBufs;
  uint64_t* drain = acc_empty + L::kBufs;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cta_rank();
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < L::kBufs; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 2 * L::kWarps);
    }
    mbar_init(drain, kIssuers);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&P.a_map);
    tma_prefetch_desc(&P.w_map);
    tma_prefetch_desc(&P.out_map);
  }
  __syncwarp();
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  cluster_sync_all();  // barriers of both CTAs initialised, TMEM allocated in both
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtx wc{P.a.status, abort_flag, kWaitLimitNs};
  grid_dependency_wait();
  allow_dependents();

  if (warp < 4) {
    if (warp == 0) {
      if (lane == 0) {
        uint32_t stage = 0, phase = 0;
        long long issued = 0;
        bool ok = true;
        for (int t = pair; t < P.items && ok; t += npairs) {
          const Item it = item_of<kSplit>(P, t);
          const int arow = it.mt * 256 + (int)rank * 128, wrow = it.nt * BN + (int)rank * (BN / 2);
          for (int kb = it.kb0; kb < it.kb1; ++kb) {
            if (!mbar_wait_sleep(&empty[stage], phase ^ 1u, wc, kSiteEmpty)) {
              ok = false;
              break;
            }
            const uint32_t fb = map_to_rank(smem_u32(&full[stage]), 0);
            if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * L::kStage);
            tma2_2sm(sA + stage * L::kA, &P.a_map, fb, kb * 128, arow);
            tma2_2sm(sW + stage * L::kW, &P.w_map, fb, kb * 128, wrow);
            ++issued;
            if (++stage == L::kStages) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
        if (!ok && rank == 0) {
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
    } else if (warp <= kIssuers) {
      if (lane == 0 && rank == 0) {
        const uint32_t idesc = make_idesc_e4m3(256, BN);
        const uint64_t a0 = make_sdesc_sw128(smem_u32(sA), 16, 1024), w0 = make_sdesc_sw128(smem_u32(sW), 16, 1024);
        // Every kIssuers-th block of depth over all of this pair's items.
        uint32_t blocks = (uint32_t)((P.items - pair + npairs - 1) / npairs) * (uint32_t)P.kblocks;
        if (kSplit) {
          blocks = 0;
          for (int t = pair; t < P.items; t += npairs) {
            const Item it = item_of<kSplit>(P, t);
            blocks += (uint32_t)(it.kb1 - it.kb0);
          }
        }
        for (uint32_t i = warp - 1; i < blocks; i += kIssuers) {
          const uint32_t stage = i % L::kStages, buf = i % L::kBufs;
          if (!mbar_wait(&acc_empty[buf], ((i / L::kBufs) & 1u) ^ 1u, wc, kSiteAccEmpty) ||
              !mbar_wait(&full[stage], (i / L::kStages) & 1u, wc, kSiteFull))
            break;
          tc_fence_after();
          umma2_f8x4(tmem + buf * BN, desc_advance(a0, stage * (L::kA >> 4)), desc_advance(w0, stage * (L::kW >> 4)),
                     idesc);
          commit_both(&acc_full[buf]);
        }
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(drain))
                     : "memory");
        const uint64_t t0 = global_timer_ns();
        while (!mbar_try(drain, 0) && global_timer_ns() - t0 < 1000000000ull) {
        }
      }
    }
  } else {
    const int q = warp & 3, eh = (warp - 4) >> 2;
    const bool releaser = warp == 4 && lane == 0;
    const uint32_t acc_empty0 = map_to_rank(smem_u32(&acc_empty[0]), 0);
    const uint32_t trow = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(eh * kCols);
    uint8_t* staged = smem + L::kOut + (warp - 4) * 4096;
    uint32_t stage = 0, buf = 0, buf_phase = 0;
    bool ok = true;
    for (int t = pair; t < P.items && ok; t += npairs) {
      const Item it = item_of<kSplit>(P, t);
      const int row = it.mt * 256 + (int)rank * 128 + q * 32 + lane;
      const int col = it.nt * BN + eh * kCols;
      // rows and column blocks past the end: any scale of the matrix does, nothing is stored
      const float* sa = P.a.a_scale + (long long)min(row, P.a.rows - 1) * P.kblocks;
      const float* sw = P.a.w_scale + (long long)(min(col, P.a.n - 1) / 128) * P.kblocks;
      float2 acc[kCols / 2];
#pragma unroll
      for (int i = 0; i < kCols / 2; ++i) acc[i] = make_float2(0.f, 0.f);
      // scales of this block and the next; the one after is in flight while this one is folded
      const int last = it.kb1 - 1, k1 = min(it.kb0 + 1, last);
      float sa0 = __ldg(sa + it.kb0), sw0 = __ldg(sw + it.kb0), sa1 = __ldg(sa + k1), sw1 = __ldg(sw + k1);
      for (int kb = it.kb0; kb < it.kb1; ++kb) {
        const float s = sa0 * sw0;
        const float2 s2 = make_float2(s, s);
        sa0 = sa1;
        sw0 = sw1;
        sa1 = __ldg(sa + min(kb + 2, last));
        sw1 = __ldg(sw + min(kb + 2, last));
        ok = mbar_wait_sleep(&acc_full[buf], buf_phase, wc, kSiteAccFull);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (releaser) mbar_arrive(&empty[stage]);  // the block's MMAs have read the stage
        tc_fence_after();
        const uint32_t tb = trow + buf * BN;
#pragma unroll
        for (int c = 0; c < kCols / 32; ++c) {
          uint32_t v[32];
          tmem_load32(tb + c * 32, v);
          if (c + 1 == kCols / 32) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_cluster_relaxed(acc_empty0 + buf * 8);
          }
#pragma unroll
          for (int i = 0; i < 16; ++i)
            acc[c * 16 + i] =
                __ffma2_rn(make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), s2, acc[c * 16 + i]);
        }
        if (++stage == L::kStages) stage = 0;
        if (++buf == L::kBufs) {
          buf = 0;
          buf_phase ^= 1u;
        }
      }
      if (!ok) break;
      // Through this warp's staging rows (128-byte swizzle) to a TMA store, which clips rows and columns
      // past the matrix: 64 columns of bf16, or twice 32 of a split's fp32.
      if (lane == 0) tma_store_wait_read();
      __syncwarp();
      if (!kSplit) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2* f = acc + i * 4;
          *reinterpret_cast<uint4*>(staged + lane * 128 + ((i ^ (lane & 7)) << 4)) =
              make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y), pack_bf16x2(f[2].x, f[2].y),
                         pack_bf16x2(f[3].x, f[3].y));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && col < P.a.n && row < P.a.rows) tma_store_3d(&P.out_map, staged, col, row, 0);
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h > 0) {
            if (lane == 0) tma_store_wait_read();
            __syncwarp();
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2* f = acc + h * 16 + i * 2;
            *reinterpret_cast<float4*>(staged + lane * 128 + ((i ^ (lane & 7)) << 4)) =
                make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && col + h * 32 < P.a.n && row < P.a.rows)
            tma_store_3d(&P.out_map, staged, col + h * 32, row, it.split);
        }
      }
    }
    if (lane == 0) tma_store_wait_read();
  }

  tc_fence_before();
  cluster_sync_all();  // no MMA, load or remote arrive of the pair is still in flight
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// Adds the splits' parts [split][row][column] up, in split order: eight columns per thread.
__global__ void __launch_bounds__(256) linear_fp8_join_kernel(const float* __restrict__ parts, int splits, int rows,
                                                              int n, bf16* __restrict__ out, int ld_out) {
  grid_dependency_wait();
  allow_dependents();
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const int per_row = n / 8;
  if (i >= (long long)rows * per_row) return;
  const int row = (int)(i / per_row), c = (int)(i - (long long)row * per_row) * 8;
  const float4* p = reinterpret_cast<const float4*>(parts + (long long)row * n + c);
  const long long step = (long long)rows * n / 4;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
#pragma unroll 4
  for (int s = 0; s < splits; ++s) {
    const float4 a = p[s * step], b = p[s * step + 1];
    x.x += a.x, x.y += a.y, x.z += a.z, x.w += a.w;
    y.x += b.x, y.y += b.y, y.z += b.z, y.w += b.w;
  }
  *reinterpret_cast<uint4*>(out + (long long)row * ld_out + c) =
      make_uint4(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w), pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
}

// Splits of the depth: only where the tiles leave pairs idle, one item per pair, at least eight blocks
// each (2.1 us; a split costs ~3, its part's store and the join).  489 x 1168 x 9616: 28.5 us without,
// 15.5 with three (20 tiles, 76 blocks).
int wide_splits(int rows, int n, int k) {
  const int tiles = ((rows + 255) / 256) * ((n + Wide::BN - 1) / Wide::BN), kb = (k + 127) / 128;
  if (tiles > kSMs / 4) return 1;
  const int s = kSMs / 2 / tiles, most = kb / 8;
  return s < most ? s : most > 1 ? most : 1;
}

// ---- product, few rows -------------------------------------------------------------------

template <int T>  // activation rows, rounded up: 16, 32 or 64
struct Few {
  static constexpr uint32_t kW = 128 * 128, kA = T * 128, kStage = kW + kA;
  // Two CTAs per SM up to 32 rows.  64 rows fill an SM's folding with one, and a deeper ring then
  // beats two CTAs of four stages (150 x 128 columns, k 8192: 32.1 us against 38.0).
  static constexpr int kResident = T <= 32 ? 2 : 1;
  static constexpr int kStages = T == 16 ? 6 : T == 32 ? 5 : 8;
  static constexpr int kBufs = 4;  // accumulators in Tensor Memory
  static constexpr uint32_t kTmem = kBufs * T;     // 64 .. 256 columns
  static constexpr int kFold = T / 32 > 0 ? T / 32 : 1;  // folding warps per 32 output columns
  static constexpr int kMine = T / kFold;                // activation rows of a folding warp
  static constexpr int kThreads = 128 + kFold * 128;
  static constexpr size_t kBytes = 1024 + (size_t)kStages * kStage + 256 + 4 * T * 4;
  static_assert((size_t)kStages * kStage >= (size_t)T * 128 * 4, "the parts reuse the ring");
  // An issuer that waits for an accumulator knows every block before the one that held it folded, so
  // the stage's last use too: its parity waits are never more than one phase behind.
  static_assert(kBufs % kIssuers == 0 && kBufs <= kStages, "see above");
};

__device__ __forceinline__ void umma1_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
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
__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// One cluster per 128 output columns (one row block of w_scale); rank r of S takes the depth
// blocks [K r / S, K (r + 1) / S).  Warp 0 loads, warps 1 and 2 issue every second block each, the
// others from warp 4 fold: thread = one output column, registers = up to 32 activation rows.
template <int T>
__global__ void __launch_bounds__(Few<T>::kThreads, Few<T>::kResident) linear_fp8_few_kernel(const __grid_constant__ Params P, int S) {
  using L = Few<T>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sW = smem;
  uint8_t* sA = smem + L::kStages * L::kW;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kStages * L::kStage);
  uint64_t* empty = full + L::kStages;
  uint64_t* acc_full = empty + L::kStages;
  uint64_t* acc_empty = acc_full + L::kBufs;
  uint64_t* drain = acc_empty + L::kBufs;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x % S, nb = blockIdx.x / S;
  const int kb0 = (int)((long long)P.kblocks * rank / S), kb1 = (int)((long long)P.kblocks * (rank + 1) / S);
  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < L::kBufs; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 4 * L::kFold);
    }
    mbar_init(drain, kIssuers);
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

  constexpr int M = L::kMine;
  const int q = warp & 3, eh = (warp - 4) >> 2;  // folding warps: their 32 columns and their rows [eh M, eh M + M)
  float2 acc[M / 2];
#pragma unroll
  for (int i = 0; i < M / 2; ++i) acc[i] = make_float2(0.f, 0.f);
  const int n = kb1 - kb0;
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
        tma_load_2d(sW + s * L::kW, &P.w_map, &full[s], (kb0 + i) * 128, nb * 128);
        tma_load_2d(sA + s * L::kA, &P.a_map, &full[s], (kb0 + i) * 128, 0);
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
  } else if (warp <= kIssuers) {
    if (lane == 0) {
      const uint32_t idesc = make_idesc_e4m3(128, T);
      const uint64_t w0 = make_sdesc_sw128(smem_u32(sW), 16, 1024), a0 = make_sdesc_sw128(smem_u32(sA), 16, 1024);
      for (int i = warp - 1; i < n; i += kIssuers) {
        const int s = i % L::kStages, b = i % L::kBufs;
        if (!mbar_wait(&acc_empty[b], ((uint32_t)(i / L::kBufs) & 1u) ^ 1u, wc, kSiteAccEmpty) ||
            !mbar_wait(&full[s], (uint32_t)(i / L::kStages) & 1u, wc, kSiteFull))
          break;
        tc_fence_after();
        const uint64_t wd = desc_advance(w0, s * (L::kW >> 4)), ad = desc_advance(a0, s * (L::kA >> 4));
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma1_f8(tmem + b * T, desc_advance(wd, kk * 2), desc_advance(ad, kk * 2), idesc, kk ? 1u : 0u);
        umma_commit(&acc_full[b]);
      }
      umma_commit(drain);
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try(drain, 0) && global_timer_ns() - t0 < 1000000000ull) {
      }
    }
  } else if (warp >= 4) {
    const uint32_t trow = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(eh * M);
    const float* sw = P.a.w_scale + (long long)nb * P.kblocks + kb0;
    // Each warp keeps a block's factors sa sw, one per activation row of its own, in shared memory;
    // every thread needs all of them.  Lane l fetches row l's one block ahead.
    float* factors = reinterpret_cast<float*>(smem + L::kStages * L::kStage + 256) + (warp - 4) * M;
    const float* sa = P.a.a_scale + (long long)min(eh * M + lane % M, P.a.rows - 1) * P.kblocks + kb0;
    float mine = n > 0 ? __ldg(sa) * __ldg(sw) : 0.f;
    for (int i = 0; i < n; ++i) {
      const int b = i % L::kBufs;
      if (lane < M) factors[lane] = mine;
      __syncwarp();
      const int next = min(i + 1, n - 1);
      mine = __ldg(sa + next) * __ldg(sw + next);
      bool ok = mbar_wait(&acc_full[b], (uint32_t)(i / L::kBufs) & 1u, wc, kSiteAccFull);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (warp == 4 && lane == 0) mbar_arrive(&empty[i % L::kStages]);
      tc_fence_after();
      uint32_t v[M];
      if constexpr (M == 16) tmem_load16(trow + b * T, v);
      else tmem_load32(trow + b * T, v);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[b]);
#pragma unroll
      for (int e = 0; e < M / 2; ++e)
        acc[e] = __ffma2_rn(make_float2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])),
                            *reinterpret_cast<const float2*>(factors + 2 * e), acc[e]);
      __syncwarp();
    }
  }

  const int c = nb * 128 + q * 32 + lane;  // this folding thread's output column
  if (S == 1) {
    if (warp >= 4 && c < P.a.n) {
#pragma unroll
      for (int e = 0; e < M; ++e) {
        const int r = eh * M + e;
        if (r < P.a.rows) P.a.out[(long long)r * P.a.ld_out + c] = __float2bfloat16(e & 1 ? acc[e / 2].y : acc[e / 2].x);
      }
    }
    tc_fence_before();
    __syncthreads();
  } else {
    // Every rank leaves its part [row][column] in its own shared memory (the ring has been read),
    // then adds every S-th row over all ranks.
    float* part = reinterpret_cast<float*>(smem);
    tc_fence_before();
    __syncthreads();
    if (warp >= 4) {
#pragma unroll
      for (int e = 0; e < M; ++e)
        if (eh * M + e < P.a.rows) part[(eh * M + e) * 128 + q * 32 + lane] = e & 1 ? acc[e / 2].y : acc[e / 2].x;
    }
    cluster_sync_all();
    const int c4 = nb * 128 + lane * 4;
    if (warp >= 4 && c4 < P.a.n) {  // a row per warp, four columns per thread (n is a multiple of 8)
      for (int r = rank + (warp - 4) * S; r < P.a.rows; r += S * 4 * L::kFold) {
        const uint32_t at = smem_u32(part + r * 128 + lane * 4);
        float4 v[8], sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = k < S ? ld_cluster_f32x4(map_to_rank(at, k)) : sum;  // all on their way
#pragma unroll
        for (int k = 0; k < 8; ++k) sum.x += v[k].x, sum.y += v[k].y, sum.z += v[k].z, sum.w += v[k].w;
        *reinterpret_cast<uint2*>(P.a.out + (long long)r * P.a.ld_out + c4) =
            make_uint2(pack_bf16x2(sum.x, sum.y), pack_bf16x2(sum.z, sum.w));
      }
    }
    cluster_sync_all();  // no rank leaves while another reads its part
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kTmem);
  }
}

template <typename F>
cudaError_t raise_smem(F* kernel, size_t bytes, int id) {
  static std::atomic<bool> done[16 * 8];  // (device, kernel)
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 16 && done[dev * 8 + id].load(std::memory_order_acquire)) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess && dev < 16) done[dev * 8 + id].store(true, std::memory_order_release);
  return e;
}

bool encode(Params& P, const LinearFp8Args& a, uint32_t a_box, uint32_t w_box) {
  memset(&P, 0, sizeof(P));
  P.a = a;
  P.kblocks = (a.k + 127) / 128;
  const uint64_t ad[2] = {(uint64_t)a.k, (uint64_t)a.rows}, wd[2] = {(uint64_t)a.k, (uint64_t)a.n};
  const uint64_t st[1] = {(uint64_t)a.k};
  const uint32_t ab[2] = {128, a_box}, wb[2] = {128, w_box};
  return encode_tmap_u8(&P.a_map, a.a, 2, ad, st, ab) && encode_tmap_u8(&P.w_map, a.w, 2, wd, st, wb);
}

cudaError_t launch_wide(const LinearFp8Args& a, cudaStream_t s) {
  Params P;
  if (!encode(P, a, 128, Wide::BN / 2)) return cudaErrorInvalidValue;
  P.splits = wide_splits(a.rows, a.n, a.k);
  const uint64_t od[3] = {(uint64_t)a.n, (uint64_t)a.rows, (uint64_t)P.splits};
  if (P.splits > 1) {
    const uint64_t ost[2] = {(uint64_t)a.n * 4, (uint64_t)a.n * a.rows * 4};
    const uint32_t obox[3] = {32, 32, 1};
    if (!encode_tmap_f32(&P.out_map, a.parts, 3, od, ost, obox)) return cudaErrorInvalidValue;
  } else {
    const uint64_t ost[2] = {(uint64_t)a.ld_out * 2, (uint64_t)a.ld_out * a.rows * 2};
    const uint32_t obox[3] = {64, 32, 1};
    if (!encode_tmap_bf16(&P.out_map, a.out, 3, od, ost, obox)) return cudaErrorInvalidValue;
  }
  P.m_tiles = (a.rows + 255) / 256;
  P.items = P.m_tiles * ((a.n + Wide::BN - 1) / Wide::BN) * P.splits;
  auto kernel = P.splits > 1 ? linear_fp8_wide_kernel<true> : linear_fp8_wide_kernel<false>;
  cudaError_t e = raise_smem(kernel, Wide::kBytes, P.splits > 1 ? 4 : 0);
  if (e != cudaSuccess) return e;
  const int most = sm_count() / 2, pairs = P.items < most ? P.items : most;
  {
    LaunchScope scope(kClsLinearFp8Blocks, s);
    e = launch_k(kernel, dim3(2 * pairs), dim3(Wide::kThreads), Wide::kBytes, s, P);
    if (e != cudaSuccess) return e;
  }
  if (P.splits > 1) {
    const long long threads = (long long)a.rows * (a.n / 8);
    LaunchScope scope(kClsLinearFp8Join, s);
    return launch_k(linear_fp8_join_kernel, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, s,
                    (const float*)a.parts, P.splits, a.rows, a.n, a.out, a.ld_out);
  }
  return cudaSuccess;
}

// Clusters of S CTAs, one CTA per SM, that the current device runs at once; it depends on which SMs
// each of its processing clusters has.  Asked once per (device, S).
int clusters_at_once(int dev, int S) {
  static std::atomic<int> known[16 * 9];
  std::atomic<int>* slot = dev < 16 ? &known[dev * 9 + S] : nullptr;
  int n = slot ? slot->load(std::memory_order_relaxed) : 0;
  if (n > 0) return n;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)S);
  cfg.blockDim = dim3(Few<64>::kThreads);
  cfg.dynamicSmemBytes = Few<64>::kBytes;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)S;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (raise_smem(linear_fp8_few_kernel<64>, Few<64>::kBytes, 3) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, linear_fp8_few_kernel<64>, &cfg) != cudaSuccess || n < 1) {
    cudaGetLastError();
    return sm_count() / S / 2;
  }
  if (slot) slot->store(n, std::memory_order_relaxed);
  return n;
}

// Splits of the depth: as many as still run at once, of two blocks at least.  One too many for that
// costs a second wave: 56 x 2288 x 4816 in 18 clusters of 8, where 15 fit, took 15.0 us, in 18 of 6 8.7.
// With the pass that quantises: 1 x 4096 x 2560 5.6 us, 1 x 12288 x 4096 9.2 (5.5 TB/s of weights), 64 x
// 4096 x 4096 8.9, 64 x 12288 x 4096 15.2, within 10 % of the best S at 60 sizes but for depths of 1024
// (up to 1.7 us).
template <int T>
int few_splits(int n, int k) {
  const int blocks = (n + 127) / 128, most = (k + 127) / 128 / 2;
  int S = most < 8 ? most : 8, dev = 0;
  cudaGetDevice(&dev);
  while (S > 1 && blocks > Few<T>::kResident * clusters_at_once(dev, S)) --S;
  return S > 1 ? S : 1;
}

template <int T>
cudaError_t launch_few(const LinearFp8Args& a, cudaStream_t s) {
  Params P;
  if (!encode(P, a, T, 128)) return cudaErrorInvalidValue;
  const cudaError_t e = raise_smem(linear_fp8_few_kernel<T>, Few<T>::kBytes, T == 16 ? 1 : T == 32 ? 2 : 3);
  if (e != cudaSuccess) return e;
  const int S = few_splits<T>(a.n, a.k);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.n + 127) / 128 * S));
  cfg.blockDim = dim3(Few<T>::kThreads);
  cfg.dynamicSmemBytes = Few<T>::kBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)S;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  LaunchScope scope(kClsLinearFp8Blocks, s);
  return cudaLaunchKernelEx(&cfg, linear_fp8_few_kernel<T>, P, S);
}

}  // namespace

cudaError_t launch_quantize_blocks(const bf16* x, long long ld, int rows, int cols, int block_rows, uint8_t* q,
                                   float* scale, cudaStream_t s) {
  const int cb = (cols + 127) / 128;
  LaunchScope scope(kClsQuantBlocks, s);
  if (block_rows == 128)
    return launch_k(quantize_square_blocks_kernel, dim3((unsigned)((rows + 127) / 128), (unsigned)cb), dim3(256), 0, s, x,
                    ld, rows, cols, q, scale);
  int tx = 8;
  while (tx < cb * 8 && tx < 256) tx *= 2;
  const int ty = 256 / tx;
  return launch_k(quantize_row_blocks_kernel, dim3((unsigned)((rows + ty - 1) / ty), (unsigned)((cb * 8 + tx - 1) / tx)),
                  dim3(tx, ty), 0, s, x, ld, rows, cols, q, scale);
}

size_t linear_fp8_parts_bytes(int rows, int n, int k) {
  const int splits = rows > 64 ? wide_splits(rows, n, k) : 1;
  return splits > 1 ? (size_t)splits * rows * n * 4 : 0;
}

cudaError_t launch_linear_fp8(const LinearFp8Args& a, cudaStream_t s) {
  if (a.rows <= 16) return launch_few<16>(a, s);
  if (a.rows <= 32) return launch_few<32>(a, s);
  if (a.rows <= 64) return launch_few<64>(a, s);
  return launch_wide(a, s);
}

}  // namespace dit
