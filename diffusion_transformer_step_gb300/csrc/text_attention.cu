// Attention with grouped heads over packed or padded sequences, causal or not.
#include "runtime.h"

namespace dit {

namespace {

struct Span {
  int q0, nq, k0, nk;
  bool ok;
};

// Rows of sequence s, checked against the buffers: the host cannot see these arrays.
__device__ __forceinline__ Span load_span(const TextAttnArgs& a, int s) {
  Span r;
  r.q0 = a.q_off[s];
  r.k0 = a.k_off[s];
  const long long nq = a.q_len ? (long long)a.q_len[s] : (long long)a.q_off[s + 1] - r.q0;
  const long long nk = a.k_len ? (long long)a.k_len[s] : (long long)a.k_off[s + 1] - r.k0;
  r.ok = r.q0 >= 0 && nq >= 0 && nq <= a.max_q && r.q0 + nq <= a.rows_q && r.k0 >= 0 && nk >= 0 && nk <= a.max_k &&
         r.k0 + nk <= a.rows_k;
  r.nq = r.ok ? (int)nq : 0;
  r.nk = r.ok ? (int)nk : 0;
  return r;
}

// One warp per (query row of a sequence, query head): the running maximum and sum of the
// softmax over one pass of the keys, each lane holding head_dim / 32 values.
template <int D>
__global__ void text_attention_simple_kernel(const TextAttnArgs a) {
  constexpr int V = D / 32;
  grid_dependency_wait();
  allow_dependents();
  const int lane = threadIdx.x & 31;
  const int i = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int h = blockIdx.y, s = blockIdx.z;
  const Span sp = load_span(a, s);
  if (!sp.ok) {
    if (threadIdx.x == 0) report_bad_entry(a.status, kSiteTextLengths);
    return;
  }
  if (i >= sp.nq) return;
  const int hk = h / (a.heads_q / a.heads_k);
  const bf16* qp = a.q + (long long)(sp.q0 + i) * a.ldq + h * D + lane * V;
  float q[V], o[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    q[e] = __bfloat162float(qp[e]) * a.scale;
    o[e] = 0.f;
  }
  const int end = a.causal ? min(sp.nk, i + sp.nk - sp.nq + 1) : sp.nk;
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < end; ++j) {
    const bf16* kp = a.k + (long long)(sp.k0 + j) * a.ldk + hk * D + lane * V;
    const bf16* vp = a.v + (long long)(sp.k0 + j) * a.ldv + hk * D + lane * V;
    float x = 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e) x += q[e] * __bfloat162float(kp[e]);
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
    const float mn = fmaxf(m, x);
    const float al = __expf(m - mn), p = __expf(x - mn);
    m = mn;
    l = l * al + p;
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] = o[e] * al + p * __bfloat162float(vp[e]);
  }
  bf16* op = a.out + (long long)(sp.q0 + i) * a.ldo + h * D + lane * V;
  const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < V; ++e) op[e] = __float2bfloat16(o[e] * inv);
}

}  // namespace

size_t text_attention_parts_bytes(const TextAttnArgs&) { return 0; }

cudaError_t launch_text_attention(const TextAttnArgs& a, cudaStream_t s) {
  const dim3 grid((unsigned)((a.max_q + 7) / 8), (unsigned)a.heads_q, (unsigned)a.seqs);
  LaunchScope scope(kClsTextAttention, s);
  if (a.head_dim == 64) return launch_k(text_attention_simple_kernel<64>, grid, dim3(256), 0, s, a);
  return launch_k(text_attention_simple_kernel<128>, grid, dim3(256), 0, s, a);
}

}  // namespace dit
