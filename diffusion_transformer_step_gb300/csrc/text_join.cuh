// Output rows from the parts that runs of keys left in the workspace.
#pragma once

#include "common.cuh"

namespace dit {

// A sum of probabilities times 2^by, by <= 0, in two steps: where references follow the products of probability and value scale,
// `by` holds the logarithm of the scales' ratio as well, down to -162, and 2^by alone is below fp32's range.
__device__ __forceinline__ float rescaled(float l, float by) {
  const float half = ex2_approx(0.5f * by);
  return l * half * half;
}

// One output row from its n parts, in order: part i has (max, sum) at ml[at(i)] and the unnormalised
// row at o[at(i) D].  One warp; the parts' rows are fetched eight at a time, since what a join costs
// is the latency of its loads. kScaled: references that hold scales.
template <int D, bool kScaled, typename At>
__device__ __forceinline__ void join_row(const float2* ml, const float* o, At at, int n, int lane, bf16* out) {
  constexpr int V = D / 32;
  float m = -INFINITY;
  for (int s = lane; s < n; s += 32) m = fmaxf(m, ml[at(s)].x);
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
  const float ref = m == -INFINITY ? 0.f : m;
  float l = 0.f, sum[V];
#pragma unroll
  for (int e = 0; e < V; ++e) sum[e] = 0.f;
  for (int s0 = 0; s0 < n; s0 += 32) {
    float2 x = make_float2(0.f, 0.f);
    if (s0 + lane < n) x = ml[at(s0 + lane)];
    // a part that held no key the row sees adds nothing, whatever its row holds
    const float f = x.y == 0.f ? -1.f : ex2_approx(x.x - ref);
    l += f < 0.f ? 0.f : kScaled ? rescaled(x.y, x.x - ref) : f * x.y;
    for (int i = 0; i < 32 && s0 + i < n; i += 8) {
      float v[8][V];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float* p = o + at(min(s0 + i + u, n - 1)) * D + lane * V;
#pragma unroll
        for (int e = 0; e < V; e += 2) {
          const float2 t = *reinterpret_cast<const float2*>(p + e);
          v[u][e] = t.x;
          v[u][e + 1] = t.y;
        }
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float w = __shfl_sync(0xffffffffu, f, i + u);
#pragma unroll
        for (int e = 0; e < V; ++e) sum[e] += w < 0.f ? 0.f : w * v[u][e];
      }
    }
  }
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
  const float inv = l == 0.f ? 0.f : 1.0f / l;
#pragma unroll
  for (int e = 0; e < V; e += 2)
    *reinterpret_cast<uint32_t*>(out + lane * V + e) = pack_bf16x2(sum[e] * inv, sum[e + 1] * inv);
}

// The same of parts `step` rows from one another.
template <int D, bool kScaled = false>
__device__ __forceinline__ void join_row(const float2* ml, const float* o, int step, int n, int lane, bf16* out) {
  join_row<D, kScaled>(ml, o, [=](int i) { return (long long)i * step; }, n, lane, out);
}

}  // namespace dit
