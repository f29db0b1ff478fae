// Linear layer with bias, activation and residual in its epilogue:
//   out = act(a w^T + bias) + res.
// Tiles of 64 x 64, four by four values per thread, operands through shared memory in fp32.
#include <math.h>

#include "runtime.h"

namespace dit {

namespace {

__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {
    case 1: return z < 0.f ? 0.f : z;
    case 2: return 0.5f * z * erfcf(-0.70710678118654752f * z);
    case 3: return z / (1.0f + expf(-1.5957691216057308f * (z + 0.044715f * z * z * z)));
    case 4: return z / (1.0f + expf(-z));
    default: return z;
  }
}

__global__ void __launch_bounds__(256) linear_act_kernel(const LinearActArgs p) {
  grid_dependency_wait();
  allow_dependents();
  __shared__ float sa[16][68], sw[16][68];
  const int n0 = blockIdx.x * 64, m0 = blockIdx.y * 64;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int lr = threadIdx.x >> 2, lk = (threadIdx.x & 3) * 4;  // the row and depths that this thread loads
  float acc[4][4] = {};
  for (int k0 = 0; k0 < p.k; k0 += 16) {
    uint2 u = make_uint2(0, 0), w = u;
    if (k0 + lk < p.k) {
      if (m0 + lr < p.rows) u = *reinterpret_cast<const uint2*>(p.a + (m0 + lr) * p.lda + k0 + lk);
      if (n0 + lr < p.n) w = *reinterpret_cast<const uint2*>(p.w + (n0 + lr) * p.ldw + k0 + lk);
    }
    const float2 a0 = unpack_bf16x2(u.x), a1 = unpack_bf16x2(u.y), w0 = unpack_bf16x2(w.x), w1 = unpack_bf16x2(w.y);
    sa[lk][lr] = a0.x, sa[lk + 1][lr] = a0.y, sa[lk + 2][lr] = a1.x, sa[lk + 3][lr] = a1.y;
    sw[lk][lr] = w0.x, sw[lk + 1][lr] = w0.y, sw[lk + 2][lr] = w1.x, sw[lk + 3][lr] = w1.y;
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < 16; ++kk)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[kk][ty * 4 + i], sw[kk][tx * 4 + j], acc[i][j]);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int r = m0 + ty * 4 + i, c = n0 + tx * 4 + j;
      if (r >= p.rows || c >= p.n) continue;
      float z = activate(acc[i][j] + (p.bias ? __bfloat162float(p.bias[c]) : 0.f), p.act);
      if (p.res) z += __bfloat162float(p.res[r * p.ld_res + c]);
      if (p.out_f32) reinterpret_cast<float*>(p.out)[r * p.ld_out + c] = z;
      else reinterpret_cast<bf16*>(p.out)[r * p.ld_out + c] = __float2bfloat16(z);
    }
}

}  // namespace

size_t linear_act_parts_bytes(int, int, int) { return 0; }

cudaError_t launch_linear_act(const LinearActArgs& a, cudaStream_t s) {
  LaunchScope scope(kClsLinearAct, s);
  return launch_k(linear_act_kernel, dim3((unsigned)((a.n + 63) / 64), (unsigned)((a.rows + 63) / 64)), dim3(256), 0, s, a);
}

}  // namespace dit
