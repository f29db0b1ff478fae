// The residual's addition and the RMSNorm behind it, to bf16 and to e4m3 with a scale per 128 values:
//   s = x + res,  y = s / sqrt(mean(s^2) + eps) * (offset + w).
//
// One CTA per row.  A thread keeps its values in registers between the sum of squares and the output, so
// every value is read once and each output written once; memory bounds it.
#include <cuda_fp8.h>

#include "runtime.h"

namespace dit {

namespace {

constexpr float kAmaxFloor = 448.0f * 0x1p-118f;  // as in the block quantiser: keeps 448 / max finite

__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = unpack_bf16x2(w[i]);
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// A thread holds V chunks of eight values, T threads apart.  T is a multiple of 32, so that the sixteen
// threads of a 128-value block are neighbours in one warp.
template <int V>
__global__ void __launch_bounds__(1024) add_rms_norm_kernel(const AddRmsNormArgs a) {
  grid_dependency_wait();
  allow_dependents();
  const long long row = blockIdx.x;
  const int T = blockDim.x, chunks = a.cols / 8;
  float s[V][8];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = threadIdx.x + i * T;
    uint4 u = make_uint4(0, 0, 0, 0), r = u;
    if (c < chunks) {
      u = *reinterpret_cast<const uint4*>(a.x + row * a.ldx + c * 8);
      if (a.res) r = *reinterpret_cast<const uint4*>(a.res + row * a.ld_res + c * 8);
    }
    unpack8(u, s[i]);
    if (a.res) {
      float f[8];
      unpack8(r, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[i][e] += f[e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(s[i][e], s[i][e], ss);
  }
  __shared__ float red[32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = ss;
  __syncthreads();
  ss = (threadIdx.x & 31) < T / 32 ? red[threadIdx.x & 31] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  const float inv = rsqrtf(ss / (float)a.cols + a.eps);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = threadIdx.x + i * T;
    const bool ok = c < chunks;
    if (ok && a.sum) *reinterpret_cast<uint4*>(a.sum + row * a.ld_sum + c * 8) = pack8(s[i]);
    float y[8], g[8];
    if (ok && a.w) unpack8(*reinterpret_cast<const uint4*>(a.w + c * 8), g);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = ok ? (s[i][e] * inv) * (a.offset + (a.w ? g[e] : 1.0f)) : 0.f;
    if (ok && a.y) *reinterpret_cast<uint4*>(a.y + row * a.ldy + c * 8) = pack8(y);
    if (a.q) {
      float m = kAmaxFloor;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(y[e]));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float f = 448.0f / m;
      uint32_t q[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        q[e] = __nv_cvt_float2_to_fp8x2(make_float2(y[2 * e] * f, y[2 * e + 1] * f), __NV_SATFINITE, __NV_E4M3);
      if (ok) {
        *reinterpret_cast<uint2*>(a.q + row * a.cols + c * 8) = make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
        if (c % 16 == 0) a.scale[row * ((a.cols + 127) / 128) + c / 16] = m / 448.0f;
      }
    }
  }
}

}  // namespace

cudaError_t launch_add_rms_norm(const AddRmsNormArgs& a, cudaStream_t s) {
  const int chunks = a.cols / 8;
  const int V = chunks <= 1024 ? 1 : chunks <= 2048 ? 2 : 4;
  const int T = ((chunks + V - 1) / V + 31) / 32 * 32;
  LaunchScope scope(kClsAddRmsNorm, s);
  auto kernel = V == 1 ? add_rms_norm_kernel<1> : V == 2 ? add_rms_norm_kernel<2> : add_rms_norm_kernel<4>;
  return launch_k(kernel, dim3((unsigned)a.rows), dim3((unsigned)T), 0, s, a);
}

}  // namespace dit
