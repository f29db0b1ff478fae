// Rotary positions of a text model: the table of 1-D positions, and the pass that norms
// every query and key head and turns it.
#include "runtime.h"

namespace dit {

namespace {

// Table of angles p * w_j.  The turn count p * w_j / (2 pi) matters modulo 1 only: with the
// turns per position as a 64-bit fixed-point fraction F_j (2^64 = one turn), the fraction of
// p turns is the low word of p * F_j, an exact reduction in one 64-bit integer product, where
// fp64 angles cost fp64 arithmetic that this GPU has little of.  The nearest quarter turn is
// split off as an integer, and the rest, at most 1/8 turn, is exact to 2^-25 relative in fp32.
__global__ void text_rope_kernel(const __grid_constant__ TextRopeArgs a) {
  grid_dependency_wait();
  allow_dependents();
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= (long long)a.n * a.half) return;
  const int row = (int)(i / a.half);
  const int j = (int)(i - (long long)row * a.half);
  const int p = a.pos ? a.pos[row] : row;
  const uint64_t u = (uint64_t)(int64_t)p * a.freq[j];  // p F mod 2^64: negative p turns backwards
  const uint64_t quarter = (u + (1ull << 61)) >> 62;
  const int64_t rest = (int64_t)(u - (quarter << 62));  // [-2^61, 2^61): -1/8 .. 1/8 turn
  float s, c;
  sincospif((float)rest * 0x1p-63f, &s, &c);  // 2^63 = half a turn
  // turn (c, s) by quarter * 90 degrees
  const float co = (quarter & 1) ? -s : c, si = (quarter & 1) ? c : s;
  const float m = (quarter & 2) ? -a.magnitude : a.magnitude;
  reinterpret_cast<float2*>(a.table)[i] = make_float2(co * m, si * m);
}

// One warp per (row, head).  Lane l holds head_dim / 32 adjacent values.
template <int D>
__global__ void qk_norm_rope_kernel(const QKNormRopeArgs a) {
  constexpr int V = D / 32;
  grid_dependency_wait();
  allow_dependents();
  const int heads = a.heads_q + a.heads_k;
  const long long item = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (item >= (long long)a.rows * heads) return;
  const int row = (int)(item / heads);
  const int h = (int)(item - (long long)row * heads);
  const bool is_q = h < a.heads_q;
  const int hh = is_q ? h : h - a.heads_q;
  const bf16* src = is_q ? a.q + row * a.ldq + hh * D : a.k + row * a.ldk + hh * D;
  bf16* dst = is_q ? a.q_out + row * a.ldq_out + hh * D : a.k_out + row * a.ldk_out + hh * D;
  const bf16* w = is_q ? a.q_norm : a.k_norm;
  int t = row;
  if (a.rot_dim > 0 && a.table_row) {
    t = a.table_row[row];
    if (t < 0 || t >= a.table_rows) {
      if (lane == 0) report_bad_entry(a.status, kSiteTextRow);
      return;
    }
  }
  float x[V];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    x[i] = __bfloat162float(src[lane * V + i]);
    ss += x[i] * x[i];
  }
  if (w) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float rs = rsqrtf(ss * (1.0f / D) + a.eps);
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = x[i] * rs * __bfloat162float(w[lane * V + i]);
  }
  const int half = a.rot_dim / 2;
  const float* tab = a.table + (long long)t * a.rot_dim;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int d = lane * V + i;
    if (a.layout == 0) {
      const float other = x[i ^ 1];
      if (d < a.rot_dim) {
        const float c = tab[(d >> 1) * 2], s = tab[(d >> 1) * 2 + 1];
        const float y = (d & 1) ? x[i] * c + other * s : x[i] * c - other * s;
        dst[d] = __float2bfloat16(y);
      } else {
        dst[d] = __float2bfloat16(x[i]);
      }
    } else {
      // the partner's lane: half is a multiple of 4, so slot i of another lane
      const int pd = d < half ? d + half : (d < a.rot_dim ? d - half : d);
      const float other = __shfl_sync(0xffffffffu, x[i], pd / V);
      if (d < a.rot_dim) {
        const int p = d < half ? d : d - half;
        const float c = tab[p * 2], s = tab[p * 2 + 1];
        dst[d] = __float2bfloat16(d < half ? x[i] * c - other * s : x[i] * c + other * s);
      } else {
        dst[d] = __float2bfloat16(x[i]);
      }
    }
  }
}

}  // namespace

cudaError_t launch_text_rope(const TextRopeArgs& a, cudaStream_t s) {
  const long long total = (long long)a.n * a.half;
  if (total == 0) return cudaSuccess;
  LaunchScope scope(kClsTextRope, s);
  return launch_k(text_rope_kernel, dim3((unsigned)((total + 255) / 256)), dim3(256), 0, s, a);
}

cudaError_t launch_qk_norm_rope(const QKNormRopeArgs& a, cudaStream_t s) {
  const long long items = (long long)a.rows * (a.heads_q + a.heads_k);
  if (items == 0) return cudaSuccess;
  const long long grid = (items + 7) / 8;
  if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
  LaunchScope scope(kClsQKNormRope, s);
  if (a.head_dim == 64) return launch_k(qk_norm_rope_kernel<64>, dim3((unsigned)grid), dim3(256), 0, s, a);
  return launch_k(qk_norm_rope_kernel<128>, dim3((unsigned)grid), dim3(256), 0, s, a);
}

}  // namespace dit
