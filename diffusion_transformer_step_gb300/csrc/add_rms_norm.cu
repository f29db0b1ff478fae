// The residual's addition and the RMSNorm behind it, to bf16 and to e4m3 with a scale per 128 values:
//   s = x + res,  y = s / sqrt(mean(s^2) + eps) * (offset + w).
//
// T threads take a row, V chunks of eight values each, which they keep in registers between the sum of squares and the
// outputs: every value is read once and each output written once. With many rows a CTA goes on to further ones, their
// loads ahead of the arithmetic of the row before, and the gains stay in registers; with few it has one chunk
// per thread, for the least time from load to store.
//
// Memory bounds all but the e4m3 output alone: 16384 rows of 4096 with residual 93.5 us to both outputs (6.5 TB/s), 81 to bf16
// (6.6); without residual 48 to bf16 (5.6 TB/s) and 54 to e4m3 alone (3.8), where 158 instructions per eight values do.
// Seven rows of 2560: 2.0 us. With one row per CTA and no loads ahead both outputs, bf16 and e4m3 alone took 96, 82 and 71 us, 16384
// rows of 256 17.1 (now 5.8).
#include <cuda_fp8.h>

#include "runtime.h"

namespace dit {

namespace {

constexpr float kAmaxFloor = 448.0f * 0x1p-118f;  // as in the block quantiser: keeps 448 / max finite

__device__ __forceinline__ void unpack8(const uint4& u, float2 (&f)[4]) {
  f[0] = unpack_bf16x2(u.x), f[1] = unpack_bf16x2(u.y), f[2] = unpack_bf16x2(u.z), f[3] = unpack_bf16x2(u.w);
}

__device__ __forceinline__ uint4 pack8(const float2 (&f)[4]) {
  return make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y), pack_bf16x2(f[2].x, f[2].y),
                    pack_bf16x2(f[3].x, f[3].y));
}

// blockDim = (T, rows of a CTA at once), T a multiple of 32: the sixteen threads of a 128-value block are neighbours in
// one warp. kQ: the e4m3 output.
template <int V>
constexpr int kMost = V == 1 ? 1024 : 512;  // threads of a CTA
template <int V, bool kRes, bool kQ>
__global__ void __launch_bounds__(kMost<V>) add_rms_norm_kernel(const __grid_constant__ AddRmsNormArgs a) {
  __shared__ float red[2][32];
  grid_dependency_wait();
  allow_dependents();
  const int T = blockDim.x, chunks = a.cols / 8, c0 = threadIdx.x, warps = T / 32;
  const long long step = (long long)gridDim.x * blockDim.y;
  const float offset = a.offset;
  uint4 w[V], x[V], r[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    w[i] = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
    if (a.w && c0 + i * T < chunks) w[i] = *reinterpret_cast<const uint4*>(a.w + (c0 + i * T) * 8);
  }
  auto load = [&](long long row) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = c0 + i * T;
      x[i] = make_uint4(0, 0, 0, 0);
      if (kRes) r[i] = x[i];
      if (row < a.rows && c < chunks) {
        x[i] = *reinterpret_cast<const uint4*>(a.x + row * a.ldx + c * 8);
        if (kRes) r[i] = *reinterpret_cast<const uint4*>(a.res + row * a.ld_res + c * 8);
      }
    }
  };
  long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  load(row);
  int turn = 0;
  for (long long first = (long long)blockIdx.x * blockDim.y; first < a.rows; first += step, row += step, turn ^= 1) {
    float2 s[V][4];
    float2 ss2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      unpack8(x[i], s[i]);
      if (kRes) {
        float2 f[4];
        unpack8(r[i], f);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[i][e] = __fadd2_rn(s[i][e], f[e]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) ss2 = __ffma2_rn(s[i][e], s[i][e], ss2);
    }
    if (V < 8) load(row + step);  // eight chunks leave no registers for that
    float ss = ss2.x + ss2.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (warps > 1) {
      // the row's warps: [threadIdx.y * warps, + warps) of the CTA's at most 32
      const int at = threadIdx.y * warps;
      if ((threadIdx.x & 31) == 0) red[turn][at + (threadIdx.x >> 5)] = ss;
      __syncthreads();  // once a row: the next one writes the other half
      const int l = threadIdx.x & 31;
      ss = l < warps ? red[turn][at + l] : 0.f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    }
    const float inv = rsqrtf(ss / (float)a.cols + a.eps);
    const bool ok_row = row < a.rows;
    float most[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = c0 + i * T;
      const bool ok = ok_row && c < chunks;
      if (ok && a.sum) *reinterpret_cast<uint4*>(a.sum + row * a.ld_sum + c * 8) = pack8(s[i]);
      float2 g[4];
      unpack8(w[i], g);
      most[i] = kAmaxFloor;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[i][e] = __fmul2_rn(__fmul2_rn(s[i][e], make_float2(inv, inv)), __fadd2_rn(g[e], make_float2(offset, offset)));
        if (kQ) most[i] = fmaxf(most[i], fmaxf(fabsf(s[i][e].x), fabsf(s[i][e].y)));
      }
      if (ok && a.y) *reinterpret_cast<uint4*>(a.y + row * a.ldy + c * 8) = pack8(s[i]);
    }
    if constexpr (kQ) {
      // The largest magnitude of each of the V blocks that a thread is in, over their sixteen threads (behind the last
      // column x is zero, and with it y). Their divisions are shared out: thread i of the sixteen has block i's.
      const int l = threadIdx.x & 15;
      float mine = 1.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) most[i] = fmaxf(most[i], __shfl_xor_sync(0xffffffffu, most[i], o));
        if (l == i) mine = most[i];
      }
      const float factor = 448.0f / mine;
      if (ok_row && l < V && c0 - l + l * T < chunks)
        a.scale[row * ((a.cols + 127) / 128) + (c0 - l + l * T) / 16] = mine / 448.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = c0 + i * T;
        const float f = __shfl_sync(0xffffffffu, factor, i, 16);
        uint32_t q[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) q[e] = __nv_cvt_float2_to_fp8x2(__fmul2_rn(s[i][e], make_float2(f, f)), __NV_SATFINITE, __NV_E4M3);
        if (ok_row && c < chunks)
          *reinterpret_cast<uint2*>(a.q + row * a.cols + c * 8) = make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
      }
    }
    if (V == 8) load(row + step);
  }
}

template <int V>
cudaError_t launch(const AddRmsNormArgs& a, dim3 grid, dim3 block, cudaStream_t s) {
  auto kernel = a.res ? (a.q ? add_rms_norm_kernel<V, true, true> : add_rms_norm_kernel<V, true, false>)
                      : (a.q ? add_rms_norm_kernel<V, false, true> : add_rms_norm_kernel<V, false, false>);
  return launch_k(kernel, grid, block, 0, s, a);
}

}  // namespace

cudaError_t launch_add_rms_norm(const AddRmsNormArgs& a, cudaStream_t s) {
  const int chunks = a.cols / 8, sms = sm_count();
  const bool few = a.rows <= 2 * sms;
  int V = 1;
  auto threads = [&] { return ((chunks + V - 1) / V + 31) / 32 * 32; };
  while (threads() > (V == 1 ? 1024 : 512)) V *= 2;
  if (!few)
    while (threads() > 32 && V < 4) V *= 2;
  const int T = threads(), R = few || T >= 256 ? 1 : 256 / T;
  long long ctas = ((long long)a.rows + R - 1) / R;
  if (!few) {
    // As many CTAs as are resident, each with several rows; for longer calls up to four times as many, whose ends even out
    // (16384 rows of 4096: 93.5 us so, 104 with the resident ones; 1777 rows of 2576: 10.7 and 8.4)
    const int resident = (V == 1 ? 1024 : 512) / (T * R) > 0 ? (V == 1 ? 1024 : 512) / (T * R) : 1;
    long long most = (long long)sms * resident;
    if (ctas >= 8 * most) most *= V == 1 ? 2 : 4;
    if (ctas > most) ctas = most;
  }
  const dim3 grid((unsigned)ctas), block((unsigned)T, (unsigned)R);
  LaunchScope scope(kClsAddRmsNorm, s);
  return V == 1 ? launch<1>(a, grid, block, s) : V == 2 ? launch<2>(a, grid, block, s)
       : V == 4 ? launch<4>(a, grid, block, s) : launch<8>(a, grid, block, s);
}

}  // namespace dit
