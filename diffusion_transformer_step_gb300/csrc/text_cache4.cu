// A paged cache of keys and values in 4 bits: writing, reading back, and the attention over it.
//
// 32 neighbouring values of a token's head share a bf16 scale = max / 7; a code is rint(x / scale) + 8, 1 to
// 15.  A head of a page holds its tokens' key codes, key scales, value codes and value scales.  The words
// of a row are ordered for the attention's matrix fragments: a lane of four finds its eight values of every group of
// 32 keys side by side, a lane of eight its four of every group of 32 values.
#include <math.h>

#include "runtime.h"

namespace dit {

namespace {

// ---- writing and reading ------------------------------------------------------------------------

struct Run {
  int first, n, start;  // rows of the buffers, how many, the first one's place in the sequence
  bool ok;
};

// The rows of sequence s that a call moves.  Appended rows end at k_len, read ones start at 0.
__device__ __forceinline__ Run load_run(const Cache4MoveArgs& a, int s) {
  Run r;
  r.first = a.off[s];
  const long long n = a.len ? (long long)a.len[s] : (long long)a.off[s + 1] - r.first;
  const long long end = a.k_len ? (long long)a.k_len[s] : n;
  r.ok = r.first >= 0 && n >= 0 && n <= a.max_len && r.first + n <= a.rows && end >= n &&
         end <= (long long)a.c.max_pages << a.c.page_shift;
  r.n = r.ok ? (int)n : 0;
  r.start = r.ok ? (int)(end - n) : 0;
  return r;
}

// Eight values of one head and token per thread: a word of key codes, or two half-words of value codes.
// grid (tokens x heads x chunks of eight of keys, then of values; sequences).
template <int D, bool kAppend>
__global__ void __launch_bounds__(256) cache4_move_kernel(const Cache4MoveArgs a) {
  constexpr int C = D / 8, G = D / 32;
  grid_dependency_wait();
  allow_dependents();
  const Run run = load_run(a, blockIdx.y);
  if (!run.ok) {
    if (blockIdx.x == 0 && threadIdx.x == 0) report_bad_entry(a.status, kSiteCache4Lengths);
    return;
  }
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const int chunk = (int)(i % C), head = (int)(i / C % a.c.heads);
  const bool value = (i / C / a.c.heads) & 1;
  const long long t = i / C / a.c.heads / 2;
  if (t >= run.n) return;  // the four threads of a group leave together
  const int pos = run.start + (int)t, slot = pos & ((1 << a.c.page_shift) - 1);
  const int page = a.table[(long long)blockIdx.y * a.c.max_pages + (pos >> a.c.page_shift)];
  if (page < 0 || page >= a.c.pages) {
    if (chunk == 0 && head == 0 && !value) report_bad_entry(a.status, kSiteCache4Page);
    return;
  }
  uint8_t* slab = a.cache + ((long long)page * a.c.heads + head) * a.c.slab() + (value ? a.c.slab() / 2 : 0);
  uint8_t* row = slab + slot * (D / 2);
  bf16* scale_at = reinterpret_cast<bf16*>(slab + a.c.code_bytes()) + slot * G + chunk / 4;
  const int j = chunk / 4, q = chunk & 3;  // group of 32, eight of it
  uint32_t* key_at = reinterpret_cast<uint32_t*>(row) + q * G + j;
  uint16_t* value_at = reinterpret_cast<uint16_t*>(row) + 2 * q * G + j;  // and G further on
  const long long col = (long long)head * D + chunk * 8;
  if constexpr (kAppend) {
    const uint4 u = *reinterpret_cast<const uint4*>(value ? a.v_in + (run.first + t) * a.ldv + col
                                                          : a.k_in + (run.first + t) * a.ldk + col);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    uint32_t top = 0;  // magnitudes of bf16 compare as integers, NaN above infinity
#pragma unroll
    for (int e = 0; e < 4; ++e) top = max(top, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
    const uint32_t four = 0xfu << (threadIdx.x & 28);
    top = max(top, __shfl_xor_sync(four, top, 1));
    top = max(top, __shfl_xor_sync(four, top, 2));
    const bool bad = top >= 0x7f80u;
    const bf16 sc = __float2bfloat16(fmaxf(__uint_as_float(top << 16), 7.0f * 0x1p-118f) / 7.0f);
    const float inv = bad ? 0.f : 1.0f / __bfloat162float(sc);
    uint32_t code = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = unpack_bf16x2(w[e]);
      code |= (uint32_t)(max(-7, min(7, __float2int_rn(f.x * inv))) + 8) << (8 * e);
      code |= (uint32_t)(max(-7, min(7, __float2int_rn(f.y * inv))) + 8) << (8 * e + 4);
    }
    if (bad) code = 0x88888888u;
    if (value) {
      value_at[0] = (uint16_t)code;
      value_at[G] = (uint16_t)(code >> 16);
    } else {
      *key_at = code;
    }
    if (q == 0) *reinterpret_cast<uint16_t*>(scale_at) = bad ? 0x7fffu : __bfloat16_as_ushort(sc);
  } else {
    const uint32_t code = value ? value_at[0] | ((uint32_t)value_at[G] << 16) : *key_at;
    const float sc = __bfloat162float(*scale_at);
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = pack_bf16x2((float)((int)((code >> (8 * e)) & 15u) - 8) * sc, (float)((int)((code >> (8 * e + 4)) & 15u) - 8) * sc);
    *reinterpret_cast<uint4*>(value ? a.v_out + (run.first + t) * a.ldv + col : a.k_out + (run.first + t) * a.ldk + col) =
        make_uint4(w[0], w[1], w[2], w[3]);
  }
}

template <bool kAppend>
cudaError_t launch_move(const Cache4MoveArgs& a, int cls, cudaStream_t s) {
  const long long threads = (long long)a.max_len * 2 * a.c.heads * (a.c.head_dim / 8), blocks = (threads + 255) / 256;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  LaunchScope scope(cls, s);
  auto kernel = a.c.head_dim == 64 ? cache4_move_kernel<64, kAppend> : cache4_move_kernel<128, kAppend>;
  return launch_k(kernel, dim3((unsigned)blocks, (unsigned)a.seqs), dim3(256), 0, s, a);
}

// ---- attention ----------------------------------------------------------------------------------

// One warp per query token and head: a lane holds D / 32 values of the query and of the output.
template <int D>
__global__ void __launch_bounds__(128) cache4_attention_kernel(const Cache4AttnArgs a) {
  constexpr int V = D / 32, G = D / 32;
  grid_dependency_wait();
  allow_dependents();
  const int s = blockIdx.y, lane = threadIdx.x & 31;
  const int q0 = a.q_off[s];
  const long long nq = a.q_len ? (long long)a.q_len[s] : (long long)a.q_off[s + 1] - q0;
  const int nk = a.k_len[s];
  if (q0 < 0 || nq < 0 || nq > a.max_q || q0 + nq > a.rows_q || nk < 0 || nk > a.max_k) {
    if (blockIdx.x == 0 && threadIdx.x == 0) report_bad_entry(a.status, kSiteCache4Lengths);
    return;
  }
  const long long item = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int token = (int)(item / a.heads_q), head = (int)(item % a.heads_q), hk = head / (a.heads_q / a.c.heads);
  if (token >= nq) return;
  float q[V], o[V] = {}, m = -INFINITY, l = 0.f;
  for (int e = 0; e < V; ++e)
    q[e] = __bfloat162float(a.q[(long long)(q0 + token) * a.ldq + head * D + lane * V + e]);
  const int seen = a.causal ? min(nk, token + nk - (int)nq + 1) : nk;
  for (int pos = 0; pos < seen; ++pos) {
    const int page = a.table[(long long)s * a.c.max_pages + (pos >> a.c.page_shift)], slot = pos & ((1 << a.c.page_shift) - 1);
    if (page < 0 || page >= a.c.pages) {
      if (lane == 0) report_bad_entry(a.status, kSiteCache4Page);
      continue;
    }
    const uint8_t* slab = a.cache + ((long long)page * a.c.heads + hk) * a.c.slab();
    float kv[2][V];
    for (int h = 0; h < 2; ++h) {
      const uint8_t* at = slab + h * (a.c.slab() / 2);
      for (int e = 0; e < V; ++e) {
        const int i = lane * V + e, j = i / 32, u = i % 32;
        const int byte = h == 0 ? ((u / 8) * G + j) * 4 + (u % 8) / 2 : ((u / 4) * G + j) * 2 + (u % 4) / 2;
        const int code = (at[slot * (D / 2) + byte] >> ((u & 1) * 4)) & 15;
        kv[h][e] = (float)(code - 8) * __bfloat162float(reinterpret_cast<const bf16*>(at + a.c.code_bytes())[slot * G + j]);
      }
    }
    float x = 0.f;
    for (int e = 0; e < V; ++e) x = fmaf(q[e], kv[0][e], x);
    for (int w = 16; w > 0; w >>= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
    x *= a.scale;
    const float mn = fmaxf(m, x), ref = mn == -INFINITY ? 0.f : mn, f = expf(m - ref), p = expf(x - ref);
    m = mn;
    l = l * f + p;
    for (int e = 0; e < V; ++e) o[e] = o[e] * f + p * kv[1][e];
  }
  const float inv = l == 0.f ? 0.f : 1.0f / l;
  for (int e = 0; e < V; ++e)
    a.out[(long long)(q0 + token) * a.ldo + head * D + lane * V + e] = __float2bfloat16(l == 0.f ? 0.f : o[e] * inv);
}

}  // namespace

cudaError_t launch_cache4_append(const Cache4MoveArgs& a, cudaStream_t s) {
  return launch_move<true>(a, kClsCache4Append, s);
}

cudaError_t launch_cache4_read(const Cache4MoveArgs& a, cudaStream_t s) {
  return launch_move<false>(a, kClsCache4Read, s);
}

size_t cache4_attention_parts_bytes(const Cache4AttnArgs&) { return 0; }

cudaError_t launch_cache4_attention(const Cache4AttnArgs& a, cudaStream_t s) {
  const long long blocks = ((long long)a.max_q * a.heads_q + 3) / 4;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  LaunchScope scope(kClsCache4Attention, s);
  auto kernel = a.c.head_dim == 64 ? cache4_attention_kernel<64> : cache4_attention_kernel<128>;
  return launch_k(kernel, dim3((unsigned)blocks, (unsigned)a.seqs), dim3(128), 0, s, a);
}

}  // namespace dit
