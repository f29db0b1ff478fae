// e4m3 operands with one fp32 scale per block of 128: quantisation and the product.
#include <cuda_fp8.h>

#include "runtime.h"

namespace dit {

namespace {

constexpr float kAmaxFloor = 448.0f * 0x1p-118f;  // keeps 448 / max finite

// One CTA of 128 threads per block of block_rows x 128 values: thread t takes column t.
__global__ void quantize_blocks_kernel(const bf16* x, long long ld, int rows, int cols, int block_rows, uint8_t* q,
                                       float* scale) {
  grid_dependency_wait();
  allow_dependents();
  const int cb = blockIdx.x, rb = blockIdx.y + blockIdx.z * 65535;
  const int r0 = rb * block_rows;
  if (r0 >= rows) return;
  const int c = cb * 128 + threadIdx.x, r1 = min(rows, r0 + block_rows);
  float amax = 0.f;
  if (c < cols)
    for (int r = r0; r < r1; ++r) amax = fmaxf(amax, fabsf(__bfloat162float(x[r * ld + c])));
  __shared__ float red[4];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
  __syncthreads();
  amax = fmaxf(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])), kAmaxFloor);
  const float inv = 448.0f / amax;
  if (c < cols)
    for (int r = r0; r < r1; ++r)
      q[(long long)r * cols + c] =
          (uint8_t)__nv_cvt_float_to_fp8(__bfloat162float(x[r * ld + c]) * inv, __NV_SATFINITE, __NV_E4M3);
  if (threadIdx.x == 0) scale[(long long)rb * gridDim.x + cb] = amax / 448.0f;
}

__device__ __forceinline__ float e4m3(uint8_t b) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(b, __NV_E4M3)));
}

// 16 x 16 outputs per CTA, one per thread, the operands of 32 depths staged as fp32.
__global__ void linear_fp8_simple_kernel(const LinearFp8Args p) {
  __shared__ float sa[16][33], sw[16][33];
  grid_dependency_wait();
  allow_dependents();
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int r0 = blockIdx.y * 16, c0 = blockIdx.x * 16;
  const int kb_n = (p.k + 127) / 128;
  float acc = 0.f;
  for (int k0 = 0; k0 < p.k; k0 += 128) {
    float part = 0.f;
    for (int k1 = k0; k1 < min(p.k, k0 + 128); k1 += 32) {
      for (int e = threadIdx.x; e < 512; e += 256) {
        const int r = e >> 5, kk = e & 31;
        sa[r][kk] = (r0 + r < p.rows && k1 + kk < p.k) ? e4m3(p.a[(long long)(r0 + r) * p.k + k1 + kk]) : 0.f;
        sw[r][kk] = (c0 + r < p.n && k1 + kk < p.k) ? e4m3(p.w[(long long)(c0 + r) * p.k + k1 + kk]) : 0.f;
      }
      __syncthreads();
#pragma unroll
      for (int kk = 0; kk < 32; ++kk) part += sa[ty][kk] * sw[tx][kk];
      __syncthreads();
    }
    if (r0 + ty < p.rows && c0 + tx < p.n)
      acc += part * (p.a_scale[(long long)(r0 + ty) * kb_n + k0 / 128] *
                     p.w_scale[(long long)((c0 + tx) / 128) * kb_n + k0 / 128]);
  }
  if (r0 + ty < p.rows && c0 + tx < p.n)
    p.out[(long long)(r0 + ty) * p.ld_out + c0 + tx] = __float2bfloat16(acc);
}

}  // namespace

cudaError_t launch_quantize_blocks(const bf16* x, long long ld, int rows, int cols, int block_rows, uint8_t* q,
                                   float* scale, cudaStream_t s) {
  const int rb = (rows + block_rows - 1) / block_rows;
  const dim3 grid((unsigned)((cols + 127) / 128), (unsigned)(rb < 65535 ? rb : 65535), (unsigned)((rb + 65534) / 65535));
  LaunchScope scope(kClsQuantBlocks, s);
  return launch_k(quantize_blocks_kernel, grid, dim3(128), 0, s, x, ld, rows, cols, block_rows, q, scale);
}

size_t linear_fp8_parts_bytes(int, int, int) { return 0; }

cudaError_t launch_linear_fp8(const LinearFp8Args& a, cudaStream_t s) {
  const dim3 grid((unsigned)((a.n + 15) / 16), (unsigned)((a.rows + 15) / 16));
  if (grid.y > 65535) return cudaErrorInvalidValue;
  LaunchScope scope(kClsLinearFp8Blocks, s);
  return launch_k(linear_fp8_simple_kernel, grid, dim3(256), 0, s, a);
}

}  // namespace dit
