// Rotary positions of a text model: the table of 1-D positions, and the pass that norms
// every query and key head and turns it.
#include <math.h>

#include <atomic>

#include "runtime.h"

namespace dit {

namespace {

// Table of angles p * w_j.  The turn count p * w_j / (2 pi) matters modulo 1 only: with the
// turns per position as a 64-bit fixed-point fraction F_j (2^64 = one turn), the fraction of
// p turns is the low word of p * F_j, an exact reduction in one 64-bit integer product, where
// fp64 angles cost fp64 arithmetic that this GPU has little of.  The nearest quarter turn is
// split off as an integer; 32 bits of the rest, at most 1/8 turn, fix the angle to 4e-10, and Taylor
// series of sine and cosine to y^9 and y^10 are within 2e-9 there (|y| <= pi / 4).
//
// Bound by the table's write and, nearly as much, by the ~40 instructions of a pair.  A thread
// turns two neighbouring pairs (one 16-byte store) of kRows rows: it reads their frequencies, which
// lie in the kernel's parameters and there cost a replay per lane, once.

__device__ __forceinline__ float2 turn(int p, uint64_t freq, float magnitude) {
  // p F mod 2^64 (negative p turns backwards), plus 1/8 turn: the top two bits are the nearest quarter
  const uint64_t u = (uint64_t)(int64_t)p * freq + (1ull << 61);
  const uint32_t quarter = (uint32_t)(u >> 62);
  const int rest = (int)((uint32_t)(u >> 30) ^ 0x80000000u);  // 2^31 = 1/8 turn
  const float x = (float)rest * 0x1p-33f;                      // in half turns: -1/4 .. 1/4
  constexpr double kPi = 3.14159265358979323846, kPi2 = kPi * kPi;
  const float z = x * x;
  // sin(pi x) = x (pi - pi^3 z / 3! + ...), cos(pi x) = 1 - pi^2 z / 2! + ...
  float s = (float)(kPi * kPi2 * kPi2 * kPi2 * kPi2 / 362880.0);
  s = fmaf(s, z, (float)(-kPi * kPi2 * kPi2 * kPi2 / 5040.0));
  s = fmaf(s, z, (float)(kPi * kPi2 * kPi2 / 120.0));
  s = fmaf(s, z, (float)(-kPi * kPi2 / 6.0));
  s = fmaf(s, z, (float)kPi) * x;
  float c = (float)(-kPi2 * kPi2 * kPi2 * kPi2 * kPi2 / 3628800.0);
  c = fmaf(c, z, (float)(kPi2 * kPi2 * kPi2 * kPi2 / 40320.0));
  c = fmaf(c, z, (float)(-kPi2 * kPi2 * kPi2 / 720.0));
  c = fmaf(c, z, (float)(kPi2 * kPi2 / 24.0));
  c = fmaf(c, z, (float)(-kPi2 / 2.0));
  c = fmaf(c, z, 1.0f);
  // turn (c, s) by quarter * 90 degrees
  const float co = (quarter & 1) ? -s : c, si = (quarter & 1) ? c : s;
  const float m = (quarter & 2) ? -magnitude : magnitude;
  return make_float2(co * m, si * m);
}

template <int kRows>
__global__ void __launch_bounds__(256) text_rope_kernel(const __grid_constant__ TextRopeArgs a) {
  grid_dependency_wait();
  allow_dependents();
  const int j = threadIdx.x * 2;  // this thread's first pair
  const int r0 = (blockIdx.x * blockDim.y + threadIdx.y) * kRows;
  if (j >= a.half) return;
  const bool two = j + 1 < a.half;
  const uint64_t f0 = a.freq[j], f1 = a.freq[two ? j + 1 : j];
  int p[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) p[i] = a.pos ? __ldg(a.pos + min(r0 + i, a.n - 1)) : r0 + i;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = r0 + i;
    if (r >= a.n) break;
    const float2 x = turn(p[i], f0, a.magnitude), y = turn(p[i], f1, a.magnitude);
    float* dst = a.table + ((long long)r * a.half + j) * 2;
    if ((a.half & 1) == 0) {  // rows of whole 16-byte pieces
      *reinterpret_cast<float4*>(dst) = make_float4(x.x, x.y, y.x, y.y);
    } else {
      *reinterpret_cast<float2*>(dst) = x;
      if (two) *reinterpret_cast<float2*>(dst + 2) = y;
    }
  }
}

// Norm and rotation: bound by reading and writing the heads.  A lane holds 8 values of a head that turn
// among themselves, so a warp takes 2 heads of 128 or 4 of 64 at once.  Adjacent pairs: 8 neighbours, one
// 16-byte access.  Halves: 4 values and their 4 partners rot_dim / 2 further on, two 8-byte accesses
// (rot_dim / 2 is a multiple of 4); partners in other lanes, fetched by shuffles, took 71 us where this
// takes 49 (10007 rows of 40 heads of 128).  The lanes behind the turned ones hold 8 neighbours each.
__device__ __forceinline__ void unpack4(const uint2& u, float* x) {
  const float2 f = unpack_bf16x2(u.x), g = unpack_bf16x2(u.y);
  x[0] = f.x, x[1] = f.y, x[2] = g.x, x[3] = g.y;
}

// A lane's share of a head: its two groups of 4 values, and the cosines and sines of its four pairs,
// (x_e, x_{e+4}) or (x_{2e}, x_{2e+1}).
template <int D, bool kHalf>
struct Lane {
  static constexpr int kLanes = D / 8, kHeads = 32 / kLanes;  // lanes per head, heads at once
  int l, d0, d1;
  bool turns;
  __device__ __forceinline__ Lane(int lane, int rot_dim) {
    l = lane % kLanes;
    turns = 8 * l < rot_dim;
    d0 = kHalf && turns ? 4 * l : 8 * l;
    d1 = kHalf && turns ? d0 + rot_dim / 2 : d0 + 4;
  }
  __device__ __forceinline__ void load(const bf16* head, uint2 (&u)[2]) const {
    if (kHalf) {
      u[0] = *reinterpret_cast<const uint2*>(head + d0);
      u[1] = *reinterpret_cast<const uint2*>(head + d1);
    } else {
      const uint4 v = *reinterpret_cast<const uint4*>(head + d0);
      u[0] = make_uint2(v.x, v.y);
      u[1] = make_uint2(v.z, v.w);
    }
  }
  __device__ __forceinline__ void store(bf16* head, const uint2 (&u)[2]) const {
    if (kHalf) {
      *reinterpret_cast<uint2*>(head + d0) = u[0];
      *reinterpret_cast<uint2*>(head + d1) = u[1];
    } else {
      *reinterpret_cast<uint4*>(head + d0) = make_uint4(u[0].x, u[0].y, u[1].x, u[1].y);
    }
  }
  // x: the pairs' table entries (cos, sin, cos, sin), y: those of the other two
  __device__ __forceinline__ void apply(uint2 (&u)[2], const bf16* w, float eps, const float4& t0, const float4& t1) const {
    float x[8], y[8];
    unpack4(u[0], x);
    unpack4(u[1], x + 4);
    if (w) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss += x[e] * x[e];
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float rs = rsqrtf(ss * (1.0f / D) + eps);
      float f[8];
      unpack4(__ldg(reinterpret_cast<const uint2*>(w + d0)), f);
      unpack4(__ldg(reinterpret_cast<const uint2*>(w + d1)), f + 4);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= rs * f[e];
    }
    const float c[4] = {t0.x, t0.z, t1.x, t1.z}, s[4] = {t0.y, t0.w, t1.y, t1.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int p = kHalf ? e : 2 * e, q = kHalf ? e + 4 : 2 * e + 1;
      y[p] = turns ? x[p] * c[e] - x[q] * s[e] : x[p];
      y[q] = turns ? x[q] * c[e] + x[p] * s[e] : x[q];
    }
    u[0] = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
    u[1] = make_uint2(pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
  }
};

// Fewer rows: a warp takes kUnroll groups of heads of one row, whose table entries it reads once, and
// the launch is as short as it can be (7 rows: 2.2 us).  Two groups and six blocks per SM hide the chain
// index -> table -> store best (2000 rows of 40 heads of 128: 9.9 us, 4.1 TB/s).
constexpr int kUnroll = 2;

template <int D, bool kHalf>
__global__ void __launch_bounds__(256, 6) qk_norm_rope_kernel(const QKNormRopeArgs a, int chunks) {
  using L = Lane<D, kHalf>;
  grid_dependency_wait();
  allow_dependents();
  const int lane = threadIdx.x & 31;
  const L my(lane, a.rot_dim);
  const long long item = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int row = (int)(item / chunks);
  if (row >= a.rows) return;
  const int head0 = (int)(item - (long long)row * chunks) * (L::kHeads * kUnroll) + lane / L::kLanes;
  const bool indexed = a.rot_dim > 0 && a.table_row;
  const int t = indexed ? __ldg(a.table_row + row) : row;  // checked once the heads' loads are on their way
  const int heads = a.heads_q + a.heads_k;
  uint2 u[kUnroll][2];
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const int h = head0 + i * L::kHeads;
    u[i][0] = u[i][1] = make_uint2(0, 0);
    if (h < heads) my.load(h < a.heads_q ? a.q + row * a.ldq + h * D : a.k + row * a.ldk + (h - a.heads_q) * D, u[i]);
  }
  if (indexed && (t < 0 || t >= a.table_rows)) {
    if (lane == 0) report_bad_entry(a.status, kSiteTextRow);
    return;
  }
  float4 t0 = make_float4(1.f, 0.f, 1.f, 0.f), t1 = t0;
  if (my.turns) {
    const float4* tab = reinterpret_cast<const float4*>(a.table + (long long)t * a.rot_dim + 8 * my.l);
    t0 = __ldg(tab), t1 = __ldg(tab + 1);
  }
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const int h = head0 + i * L::kHeads;
    const bool is_q = h < a.heads_q;
    // groups past the last head have no k_norm to read when there are no key heads
    my.apply(u[i], is_q || h >= heads ? a.q_norm : a.k_norm, a.eps, t0, t1);
    if (h < heads)
      my.store(is_q ? a.q_out + row * a.ldq_out + h * D : a.k_out + row * a.ldk_out + (h - a.heads_q) * D, u[i]);
  }
}

// Many rows: what counts is bytes in flight.  Each warp streams chunks of a row (up to 4 KB of query
// heads or of key heads) through two buffers of its own in shared memory, in and out by bulk copies,
// and works on them in place; the row's index is read two chunks ahead and its table entries one.
// Warps take equal runs of neighbouring chunks.  40000 rows of 40 heads of 128, halves, normed: 132 us
// (6.2 TB/s) against 192 row by row; 10007 rows 37 and 51; 10007 rows of 40 heads of 64, 48 values of
// each turned, 20.3 and 21.2.  24 warps per SM; 16 with a third buffer took 140 us, 32 with 2 KB 152.
constexpr int kStages = 2, kStageBytes = 4096, kStreamWarps = 12;
constexpr size_t kStreamSmem = (size_t)kStreamWarps * kStages * kStageBytes;
enum : uint32_t { kSiteTextStream = 0x611 };

struct Chunks {
  int q, k;        // chunks of a row's query heads and key heads
  int per_q, per_k;  // heads of each
  int total;
};

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
               : "memory");
}

template <int D, bool kHalf>
__global__ void __launch_bounds__(kStreamWarps * 32, 2)
    qk_stream_kernel(const __grid_constant__ QKNormRopeArgs a, const Chunks ch) {
  using L = Lane<D, kHalf>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[kStreamWarps * kStages];
  __shared__ int abort_flag;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t* bars = full + warp * kStages;
  uint8_t* stages = smem + warp * kStages * kStageBytes;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStreamWarps * kStages; ++i) mbar_init(&full[i], 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  grid_dependency_wait();
  allow_dependents();
  const L my(lane, a.rot_dim);
  const WaitCtx wc{a.status, &abort_flag, kWaitLimitNs};
  const int per_row = ch.q + ch.k, warps = gridDim.x * kStreamWarps, w0 = blockIdx.x * kStreamWarps + warp;
  const int first = (int)((long long)ch.total * w0 / warps), end = (int)((long long)ch.total * (w0 + 1) / warps);
  const bool indexed = a.rot_dim > 0 && a.table_row;
  // chunk id: its row, whether of queries, first head and heads
  auto locate = [&](int id, int& row, bool& is_q, int& h0, int& n) {
    row = id / per_row;
    const int c = id - row * per_row;
    is_q = c < ch.q;
    h0 = is_q ? c * ch.per_q : (c - ch.q) * ch.per_k;
    n = is_q ? min(ch.per_q, a.heads_q - h0) : min(ch.per_k, a.heads_k - h0);
  };
  auto fetch = [&](int id, int stage) {  // lane 0
    int row, h0, n;
    bool is_q;
    locate(id, row, is_q, h0, n);
    mbar_arrive_expect_tx(&bars[stage], n * D * 2);
    bulk_load(stages + stage * kStageBytes, (is_q ? a.q + row * a.ldq : a.k + row * a.ldk) + h0 * D, n * D * 2,
              &bars[stage]);
  };
  auto index_of = [&](int id) {
    if (id >= end) return 0;
    const int row = id / per_row;
    return indexed ? __ldg(a.table_row + row) : row;
  };
  auto entries = [&](int t, float4& t0, float4& t1) {
    if (my.turns && t >= 0 && t < a.table_rows) {
      const float4* tab = reinterpret_cast<const float4*>(a.table + (long long)t * a.rot_dim + 8 * my.l);
      t0 = __ldg(tab), t1 = __ldg(tab + 1);
    }
  };
  if (lane == 0)
    for (int s = 0; s < kStages - 1; ++s)
      if (first + s < end) fetch(first + s, s);
  int t = index_of(first), t_next = index_of(first + 1);
  float4 t0 = make_float4(1.f, 0.f, 1.f, 0.f), t1 = t0;
  entries(t, t0, t1);
  bool ok = true;
  int stage = 0;
  uint32_t phase = 0;
  for (int id = first; id < end; ++id) {
    const int t_after = index_of(id + 2);
    float4 n0 = t0, n1 = t1;
    if (id + 1 < end) entries(t_next, n0, n1);
    // the buffer of the chunk before, once its store has read it, takes the chunk kStages - 1 ahead
    if (lane == 0 && id + kStages - 1 < end) {
      asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
      fetch(id + kStages - 1, stage == 0 ? kStages - 1 : stage - 1);
    }
    ok = mbar_wait(&bars[stage], phase, wc, kSiteTextStream);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) break;
    int row, h0, n;
    bool is_q;
    locate(id, row, is_q, h0, n);
    uint8_t* buf = stages + stage * kStageBytes;
    if (indexed && (t < 0 || t >= a.table_rows)) {
      if (lane == 0) report_bad_entry(a.status, kSiteTextRow);
    } else {
      bf16* head = reinterpret_cast<bf16*>(buf) + lane / L::kLanes * D;
      const bf16* w = is_q ? a.q_norm : a.k_norm;
      for (int h = lane / L::kLanes; h - lane / L::kLanes < n; h += 2 * L::kHeads, head += 2 * L::kHeads * D) {
        uint2 u[2][2] = {};
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (h + e * L::kHeads < n) my.load(head + e * L::kHeads * D, u[e]);
#pragma unroll
        for (int e = 0; e < 2; ++e) my.apply(u[e], w, a.eps, t0, t1);
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (h + e * L::kHeads < n) my.store(head + e * L::kHeads * D, u[e]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0)
        bulk_store((is_q ? a.q_out + row * a.ldq_out : a.k_out + row * a.ldk_out) + h0 * D, buf, n * D * 2);
    }
    if (lane == 0) asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    __syncwarp();
    t = t_next;
    t_next = t_after;
    t0 = n0, t1 = n1;
    if (++stage == kStages) {
      stage = 0;
      phase ^= 1u;
    }
  }
  if (lane == 0) {
    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    if (!ok) {  // loads in flight land before the block leaves (bounded)
      const uint64_t since = global_timer_ns();
      while (global_timer_ns() - since < 100000000ull) {
      }
    }
  }
}

template <int D, bool kHalf>
cudaError_t launch_qk(const QKNormRopeArgs& a, cudaStream_t s) {
  LaunchScope scope(kClsQKNormRope, s);
  constexpr int kMost = kStageBytes / (D * 2);  // heads of a chunk
  Chunks ch = {};
  ch.q = (a.heads_q + kMost - 1) / kMost;
  ch.k = (a.heads_k + kMost - 1) / kMost;
  ch.per_q = (a.heads_q + ch.q - 1) / ch.q;
  ch.per_k = ch.k > 0 ? (a.heads_k + ch.k - 1) / ch.k : 0;
  const long long total = (long long)a.rows * (ch.q + ch.k);
  const long long bytes = (long long)a.rows * (a.heads_q + a.heads_k) * D * 2;
  // Streams from 40 MB on, in chunks of 1.5 KB on average (below: 3505 rows of 25 heads of 128 9.9 us
  // row by row, 11.1 streamed; 100000 rows of 8 + 8 heads of 64 98 and 105).
  if (bytes >= 40000000 && bytes / total >= 1536 && total < (1ll << 30)) {
    static std::atomic<bool> raised[16];
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 16 || !raised[dev].load(std::memory_order_acquire)) {
      const cudaError_t e = cudaFuncSetAttribute(qk_stream_kernel<D, kHalf>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 (int)kStreamSmem);
      if (e != cudaSuccess) return e;
      if (dev < 16) raised[dev].store(true, std::memory_order_release);
    }
    ch.total = (int)total;
    return launch_k(qk_stream_kernel<D, kHalf>, dim3((unsigned)(2 * sm_count())), dim3(kStreamWarps * 32), kStreamSmem, s, a,
                    ch);
  }
  const int per_warp = 32 / (D / 8) * kUnroll, chunks = (a.heads_q + a.heads_k + per_warp - 1) / per_warp;
  const long long grid = ((long long)a.rows * chunks + 7) / 8;  // under 2^31: rows x heads <= 2^35
  return launch_k(qk_norm_rope_kernel<D, kHalf>, dim3((unsigned)grid), dim3(256), 0, s, a, chunks);
}

}  // namespace

cudaError_t launch_text_rope(const TextRopeArgs& a, cudaStream_t s) {
  if (a.n == 0) return cudaSuccess;
  int tx = 1;  // threads along a row, two pairs each
  while (tx * 2 < a.half) tx *= 2;
  const int ty = 256 / tx;
  LaunchScope scope(kClsTextRope, s);
  auto run = [&](auto kernel, int rows) {
    return launch_k(kernel, dim3((unsigned)((a.n + rows * ty - 1) / (rows * ty))), dim3(tx, ty), 0, s, a);
  };
  // 16 rows per thread where that leaves four blocks per SM (131072 x 64 pairs: 64 us with one row
  // per thread, 14.1 with 8), else one, for the shortest path through a small table (512 rows: 1.7 us).
  if (a.n / (16 * ty) >= 4 * 152) return run(text_rope_kernel<16>, 16);
  if (a.n / (4 * ty) >= 4 * 152) return run(text_rope_kernel<4>, 4);
  return run(text_rope_kernel<1>, 1);
}

cudaError_t launch_qk_norm_rope(const QKNormRopeArgs& a, cudaStream_t s) {
  if (a.rows == 0) return cudaSuccess;
  if (a.layout) return a.head_dim == 64 ? launch_qk<64, true>(a, s) : launch_qk<128, true>(a, s);
  return a.head_dim == 64 ? launch_qk<64, false>(a, s) : launch_qk<128, false>(a, s);
}

}  // namespace dit
