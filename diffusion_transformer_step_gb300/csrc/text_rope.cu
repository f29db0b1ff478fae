// Rotary positions of a text model: the table of 1-D positions, and the pass that norms
// every query and key head and turns it.
#include <math.h>

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
// among themselves, so a warp takes 2 heads of 128 or 4 of 64 at once, and kUnroll such groups of
// one row, whose cosines and sines it reads once.  Adjacent pairs: 8 neighbours, one 16-byte access.
// Halves: 4 values and their 4 partners rot_dim / 2 further on, two 8-byte accesses (rot_dim / 2 is
// a multiple of 4); partners in other lanes, fetched by shuffles, took 71 us where this takes 49 (heads of 128).
// The lanes behind the turned ones hold 8 neighbours each.
// 10007 rows of 40 heads of 64, 48 values of each turned: 21 us, 4.9 TB/s; two groups and six blocks
// per SM hide the chain index -> table -> store best (one group 25 us, four 24).
constexpr int kUnroll = 2;

__device__ __forceinline__ void unpack4(const uint2& u, float* x) {
  const float2 f = unpack_bf16x2(u.x), g = unpack_bf16x2(u.y);
  x[0] = f.x, x[1] = f.y, x[2] = g.x, x[3] = g.y;
}

template <int D, bool kHalf>
__global__ void __launch_bounds__(256, 6) qk_norm_rope_kernel(const QKNormRopeArgs a, int chunks) {
  constexpr int kLanes = D / 8, kHeads = 32 / kLanes;  // lanes per head, heads at once
  grid_dependency_wait();
  allow_dependents();
  const int lane = threadIdx.x & 31, l = lane % kLanes;
  const long long item = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int row = (int)(item / chunks);
  if (row >= a.rows) return;
  const int head0 = (int)(item - (long long)row * chunks) * (kHeads * kUnroll) + lane / kLanes;
  int t = row;
  if (a.rot_dim > 0 && a.table_row) {
    t = a.table_row[row];
    if (t < 0 || t >= a.table_rows) {
      if (lane == 0) report_bad_entry(a.status, kSiteTextRow);
      return;
    }
  }
  const int heads = a.heads_q + a.heads_k, half = a.rot_dim / 2;
  // where this lane's two groups of 4 values lie, and whether they turn
  const bool turns = 8 * l < a.rot_dim;
  const int d0 = kHalf && turns ? 4 * l : 8 * l, d1 = kHalf && turns ? d0 + half : d0 + 4;
  uint2 u[kUnroll][2];
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const int h = head0 + i * kHeads;
    u[i][0] = u[i][1] = make_uint2(0, 0);
    if (h < heads) {
      const bf16* src = h < a.heads_q ? a.q + row * a.ldq + h * D : a.k + row * a.ldk + (h - a.heads_q) * D;
      if (kHalf) {
        u[i][0] = *reinterpret_cast<const uint2*>(src + d0);
        u[i][1] = *reinterpret_cast<const uint2*>(src + d1);
      } else {
        const uint4 v = *reinterpret_cast<const uint4*>(src + d0);
        u[i][0] = make_uint2(v.x, v.y);
        u[i][1] = make_uint2(v.z, v.w);
      }
    }
  }
  // cosines and sines of the lane's four pairs: (x_e, x_{e+4}), or (x_{2e}, x_{2e+1})
  float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
  if (turns) {
    const float4* tab = reinterpret_cast<const float4*>(a.table + (long long)t * a.rot_dim + 8 * l);
    const float4 x = __ldg(tab), y = __ldg(tab + 1);
    c[0] = x.x, s[0] = x.y, c[1] = x.z, s[1] = x.w, c[2] = y.x, s[2] = y.y, c[3] = y.z, s[3] = y.w;
  }
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const int h = head0 + i * kHeads;
    const bool is_q = h < a.heads_q;
    float x[8];
    unpack4(u[i][0], x);
    unpack4(u[i][1], x + 4);
    if (a.q_norm) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss += x[e] * x[e];
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float rs = rsqrtf(ss * (1.0f / D) + a.eps);
      // groups past the last head have no k_norm to read when there are no key heads
      const bf16* w = is_q || h >= heads ? a.q_norm : a.k_norm;
      float f[8];
      unpack4(__ldg(reinterpret_cast<const uint2*>(w + d0)), f);
      unpack4(__ldg(reinterpret_cast<const uint2*>(w + d1)), f + 4);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= rs * f[e];
    }
    float y[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int p = kHalf ? e : 2 * e, q = kHalf ? e + 4 : 2 * e + 1;
      y[p] = turns ? x[p] * c[e] - x[q] * s[e] : x[p];
      y[q] = turns ? x[q] * c[e] + x[p] * s[e] : x[q];
    }
    if (h < heads) {
      bf16* dst = is_q ? a.q_out + row * a.ldq_out + h * D : a.k_out + row * a.ldk_out + (h - a.heads_q) * D;
      const uint2 lo = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
      const uint2 hi = make_uint2(pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
      if (kHalf) {
        *reinterpret_cast<uint2*>(dst + d0) = lo;
        *reinterpret_cast<uint2*>(dst + d1) = hi;
      } else {
        *reinterpret_cast<uint4*>(dst + d0) = make_uint4(lo.x, lo.y, hi.x, hi.y);
      }
    }
  }
}

template <int D>
cudaError_t launch_qk(const QKNormRopeArgs& a, cudaStream_t s) {
  const int per_warp = 32 / (D / 8) * kUnroll, chunks = (a.heads_q + a.heads_k + per_warp - 1) / per_warp;
  const long long grid = ((long long)a.rows * chunks + 7) / 8;
  if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
  LaunchScope scope(kClsQKNormRope, s);
  if (a.layout) return launch_k(qk_norm_rope_kernel<D, true>, dim3((unsigned)grid), dim3(256), 0, s, a, chunks);
  return launch_k(qk_norm_rope_kernel<D, false>, dim3((unsigned)grid), dim3(256), 0, s, a, chunks);
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
  return a.head_dim == 64 ? launch_qk<64>(a, s) : launch_qk<128>(a, s);
}

}  // namespace dit
