// A paged cache of keys and values in 4 bits: writing, reading back, and the attention over it.
//
// 32 neighbouring values of a token's head share a bf16 scale = max / 7; a code is rint(x / scale) + 8, 1 to
// 15.  A head of a page holds its tokens' key codes, key scales, value codes and value scales.  The words
// of a row are ordered for the attention's matrix fragments: a lane of four finds its eight values of every group of
// 32 keys side by side, a lane of eight its four of every group of 32 values.
#include <math.h>
#include <string.h>

#include <atomic>
#include <type_traits>

#include "cta_pair.cuh"
#include "runtime.h"
#include "text_join.cuh"

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

// Four threads take a token's head of keys or values: thread t the values 32 j + 8 t onwards, eight of every group j, which
// lie side by side in the cache (a word each of the keys' codes, two half-words of the values') and in whole sectors of
// the rows. A CTA has `tokens` tokens (a power of two), and where those do not fill it several heads side by side; each
// thread goes through U of them with its loads ahead of its stores. The table is read once per token.
// Memory bounds it: 512 new tokens of 16 sequences in and 700 to 8192 of each out (429 MB) take 73.7 us for both calls, 5.8
// TB/s (reading alone 6.7); with eight values a thread, and so many small CTAs, 214. Appending alone, 3.6 TB/s, is as much
// arithmetic as traffic: 8192 tokens of 8 heads 11.9 us, with all divisions in all four threads, conversions and clamps
// 14.3. A decoding step's append and read of eight short sequences: 5.9 us, two launches.
template <int D, bool kAppend, int U>
__global__ void __launch_bounds__(256) cache4_move_kernel(const Cache4MoveArgs a, int tokens, int side, int parts) {
  constexpr int G = D / 32;
  grid_dependency_wait();
  allow_dependents();
  const Run run = load_run(a, blockIdx.y);
  if (!run.ok) {
    if (blockIdx.x == 0 && threadIdx.x == 0) report_bad_entry(a.status, kSiteCache4Lengths);
    return;
  }
  const int block = blockIdx.x / parts, first = (blockIdx.x - block * parts) * side * U;  // of the heads, keys then values
  const int t = threadIdx.x & 3, i = block * tokens + (int)(threadIdx.x >> 2) % tokens, lane = (threadIdx.x >> 2) / tokens;
  if (i >= run.n) return;  // a token's four threads leave together
  const int pos = run.start + i, slot = pos & ((1 << a.c.page_shift) - 1);
  const int page = a.table[(long long)blockIdx.y * a.c.max_pages + (pos >> a.c.page_shift)];
  if (page < 0 || page >= a.c.pages) {
    if (first + lane == 0 && t == 0) report_bad_entry(a.status, kSiteCache4Page);
    return;
  }
  const int heads = a.c.heads, slab = a.c.slab(), scales = a.c.code_bytes() + slot * (G * 2);
  uint8_t* const pages = a.cache + (long long)page * heads * slab;
  const long long row = run.first + i;
  const uint32_t four = 0xfu << (threadIdx.x & 28);
  auto place = [&](int u, bool& value, int& head) {
    const int h = first + u * side + lane;
    value = h >= heads;
    head = value ? h - heads : h;
    return h < 2 * heads;
  };
  if constexpr (kAppend) {
    uint4 in[U][G];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      bool value;
      int head;
      if (!place(u, value, head)) continue;
      const bf16* src = (value ? a.v_in + row * a.ldv : a.k_in + row * a.ldk) + head * D + t * 8;
#pragma unroll
      for (int j = 0; j < G; ++j) in[u][j] = *reinterpret_cast<const uint4*>(src + 32 * j);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      bool value;
      int head;
      if (!place(u, value, head)) continue;  // the same for a token's four threads
      uint32_t top[G], code[G], sc[G];  // magnitudes of bf16 compare as integers, NaN above infinity
#pragma unroll
      for (int j = 0; j < G; ++j) {
        const uint32_t w[4] = {in[u][j].x, in[u][j].y, in[u][j].z, in[u][j].w};
        top[j] = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) top[j] = max(top[j], max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
        top[j] = max(top[j], __shfl_xor_sync(four, top[j], 1));
        top[j] = max(top[j], __shfl_xor_sync(four, top[j], 2));
      }
      // each thread divides for one group (two of four do it for the same one where there are two)
      uint32_t most = top[G - 1];
#pragma unroll
      for (int j = 0; j < G - 1; ++j)
        if ((t & (G - 1)) == j) most = top[j];
      const bf16 scale = __float2bfloat16(fmaxf(__uint_as_float(most << 16), 7.0f * 0x1p-118f) / 7.0f);
      const float own = 1.0f / __bfloat162float(scale);
#pragma unroll
      for (int j = 0; j < G; ++j) {
        const uint32_t w[4] = {in[u][j].x, in[u][j].y, in[u][j].z, in[u][j].w};
        const bool bad = top[j] >= 0x7f80u;
        const float inv = __shfl_sync(four, own, j, 4);
        sc[j] = __shfl_sync(four, (uint32_t)__bfloat16_as_ushort(scale), j, 4);
        // Added to 2^23 + 2^22 + 8 a product is rounded to an integer, ties to even, and its code left in the lowest four bits;
        // no product reaches 7.5, since the scale is within 2^-8 of max / 7.
        code[j] = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = unpack_bf16x2(w[e]);
          code[j] |= (__float_as_uint(__fadd_rn(__fmul_rn(f.x, inv), 12582920.0f)) & 15u) << (8 * e);
          code[j] |= (__float_as_uint(__fadd_rn(__fmul_rn(f.y, inv), 12582920.0f)) & 15u) << (8 * e + 4);
        }
        if (bad) code[j] = 0x88888888u, sc[j] = 0x7fffu;
      }
      uint32_t out[G];
#pragma unroll
      for (int j = 0; j < G / 2; ++j) {  // keys: the groups' words; values: the groups' low half-words, then the high ones
        out[j] = value ? __byte_perm(code[2 * j], code[2 * j + 1], 0x5410) : code[j];
        out[G / 2 + j] = value ? __byte_perm(code[2 * j], code[2 * j + 1], 0x7632) : code[G / 2 + j];
      }
      uint8_t* half = pages + (long long)head * slab + (value ? slab / 2 : 0);
      uint32_t* dst = reinterpret_cast<uint32_t*>(half + slot * (D / 2)) + t * G;
      uint32_t* sdst = reinterpret_cast<uint32_t*>(half + scales);
      if constexpr (G == 4) {
        *reinterpret_cast<uint4*>(dst) = make_uint4(out[0], out[1], out[2], out[3]);
        if (t == 0) *reinterpret_cast<uint2*>(sdst) = make_uint2(sc[0] | sc[1] << 16, sc[2] | sc[3] << 16);
      } else {
        *reinterpret_cast<uint2*>(dst) = make_uint2(out[0], out[1]);
        if (t == 0) *sdst = sc[0] | sc[1] << 16;
      }
    }
  } else {
    uint32_t in[U][G], sc[U][G / 2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      bool value;
      int head;
      if (!place(u, value, head)) continue;
      const uint8_t* half = pages + (long long)head * slab + (value ? slab / 2 : 0);
      const uint8_t *src = half + slot * (D / 2) + t * (G * 4), *ssrc = half + scales;
      if constexpr (G == 4) {
        const uint4 w = *reinterpret_cast<const uint4*>(src);
        const uint2 s2 = *reinterpret_cast<const uint2*>(ssrc);
        in[u][0] = w.x, in[u][1] = w.y, in[u][2] = w.z, in[u][3] = w.w, sc[u][0] = s2.x, sc[u][1] = s2.y;
      } else {
        const uint2 w = *reinterpret_cast<const uint2*>(src);
        in[u][0] = w.x, in[u][1] = w.y, sc[u][0] = *reinterpret_cast<const uint32_t*>(ssrc);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      bool value;
      int head;
      if (!place(u, value, head)) continue;
      bf16* dst = (value ? a.v_out + row * a.ldv : a.k_out + row * a.ldk) + head * D + t * 8;
#pragma unroll
      for (int j = 0; j < G; ++j) {
        const uint32_t code = value ? __byte_perm(in[u][j / 2], in[u][G / 2 + j / 2], j & 1 ? 0x7632 : 0x5410) : in[u][j];
        const uint32_t s2 = sc[u][j / 2];
        const float scale = __uint_as_float(j & 1 ? s2 & 0xffff0000u : s2 << 16);
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          w[e] = pack_bf16x2((float)((int)((code >> (8 * e)) & 15u) - 8) * scale,
                             (float)((int)((code >> (8 * e + 4)) & 15u) - 8) * scale);
        *reinterpret_cast<uint4*>(dst + 32 * j) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
}

template <bool kAppend>
cudaError_t launch_move(const Cache4MoveArgs& a, int cls, cudaStream_t s) {
  constexpr int U = kAppend ? 2 : 4;
  int tokens = 1;
  while (tokens < 64 && tokens < a.max_len) tokens *= 2;
  const int side = 64 / tokens, parts = (2 * a.c.heads + side * U - 1) / (side * U);
  const long long blocks = (((long long)a.max_len + tokens - 1) / tokens) * parts;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  LaunchScope scope(cls, s);
  auto kernel = a.c.head_dim == 64 ? cache4_move_kernel<64, kAppend, U> : cache4_move_kernel<128, kAppend, U>;
  return launch_k(kernel, dim3((unsigned)blocks, (unsigned)a.seqs), dim3(256), 0, s, a, tokens, side, parts);
}

// ---- attention ----------------------------------------------------------------------------------

// One CTA takes a run of keys of one sequence and key head for up to 8 NT query rows (tokens x heads of the
// group): warp 4 brings stages of 128 tokens in by bulk copies, page by page, and warps 0 to 3 take 32 tokens of a
// stage each through mma.sync with a running maximum and sum of their own, which add up at the end in order. Runs of
// several CTAs are joined in shared memory where they are a cluster, by a second kernel otherwise. The runs are cut by the
// bounds that the host knows, or, for longer calls, evenly by the lengths on the device (kEven): then a CTA has pieces of
// several sequences and heads, one after another.
//
// The tokens are the rows of both products, the few queries their columns: S^T = K Q^T and O^T = V^T P^T. What bounds
// this kernel is issue: 311 instructions per 16 tokens (8 rows, 128 dims), 144 of them on the integer pipe, which takes half a warp
// per cycle, to spread 4-bit codes over 16-bit operands, and 21 MMAs (17 in even shares, see kAdds), with three warps per scheduler to choose from (a fourth,
// with two CTAs of seven and a sender, gains its scheduler 5 %; from L2 the same calls take 2 % less). So a code is left where one AND leaves it. As the bits of an fp16 number, a code c in the lowest four
// bits is the subnormal c 2^-24, in the next four c 2^-20: both exact operands, five operations per eight codes of the keys
// and six of the values. (As bf16 128 + c, with an OR and more shifts, and an exact subtraction of 136 for the values: 458
// instructions per 16 tokens instead of 355, 64 tokens over 8192 each 172 us instead of 140, all else equal.)
//
// Keys: the queries become fp16 times a power of two per row (largest magnitude in [2^13, 2^14)), exact down to 2^-26 of the
// row's largest; those that meet the higher codes are divided by 16. The 8 that every code is too large is taken off
// by -8 sum(q) per group: scales times those sums is one more small product (they go in as three bf16 parts, 24 bits), and
// the accumulators of the groups are added to it, times the key's scale, in fp32.
// Values: the scales, one per token and 32 values, belong to the index that the product sums over, so they go into the
// probabilities. f = p s is rounded to fp16 (2^-11): the reference that a row's exponents are taken from is that of its largest
// p s, 2^6 below it, so that f stays under 2^15, and what is rounded coarser (subnormal) is below 2^-20 of the row's
// largest weight, within 2^-31 of it. The 8 is taken off at the end: -8 sum(f) of the rounded f, by one more product with ones, or
// by additions (kAdds): four products of the 21 that a tile takes, or sixteen additions and half of the registers (64 x 8192 tokens
// 124.4 -> 121.6 us, 12 rows 104.9 -> 102; eight short sequences 8.8 -> 9.5, for their code has to come first).
// The unit that sums a step's sixteen products lines them up by the exponents of their operands, and a subnormal has that of
// 2^-14: of each product what lies below 2^-24 2^-14 of the largest other operand is cut off, 2^-14 of that operand per code
// (measured: one step of random codes is within 2^-20.5 of the sum of magnitudes, eight steps 2^-24.4).
constexpr int kKeys = 128, kStages = 3, kAhead = 2;
// Whether the warps that compute send for the stages themselves, in turns, or a fifth warp does. A scheduler's 16384
// registers hold four warps of 128, three of 168 or two of 255: with sixteen rows of 128-wide heads two CTAs of four warps
// that do not spill are faster than two of five that do (12 rows over 32 x 8192 tokens 117 us, 142); the others have
// room for the fifth (8 rows over 64 x 8192: 121 us, 126 with three CTAs of four warps of 168, 137 with four of 128; 15 rows of
// 64-wide heads 17.3, 20.0).
template <int D, int NT>
constexpr bool kOwn = D == 128 && NT == 2;
template <int D, int NT>
constexpr int kThreads = kOwn<D, NT> ? 128 : 160;

enum : uint32_t { kSiteCache4Full = 0x811, kSiteCache4Empty };

struct Plan {
  int rows, tile, tiles, walk;  // query rows per key head, of a CTA, tiles, tiles side by side
  int chunk, splits;            // keys per CTA, CTAs per sequence, head and tile
  bool cluster;                 // the splits are a cluster
  int even;                     // CTAs that share all blocks of keys out evenly, or 0
};

// Even shares: the parts that the last piece of a CTA's share, the first of its sequence and head, is joined from.
struct Cut {
  int head, q0, nq, parts;  // parts 0: there is none
};

struct Params {
  Cache4AttnArgs a;
  int group, rows, tiles, walk, chunk, splits, cluster, even;
  float scale_log2;
  float2* ml;
  float* o;
  Cut* cuts;
};

// CTAs per SM, of `rows` query rows (8 or 16) each. For eight rows 128 registers and three CTAs of five warps; for sixteen three
// warps of 168 registers (64-wide heads) or two of 255 fit a scheduler, which is two CTAs of five or four. The plan cuts the keys
// for as many CTAs as run at once, so it takes this number from here, and the kernel's launch bounds do too. (Cut for three CTAs of sixteen rows
// of 64-wide heads, a third of the shares began in a second round: 12 rows over 32 x 8192 tokens 82 us instead of 62, 15 over 4
// sequences of up to 32768 44 instead of 32; where runs are cut by bounds 17 tokens of 4 heads over 20000 21 instead of 15.)
__host__ __device__ constexpr int ctas_per_sm(int rows) { return rows == 8 ? 3 : 2; }

// What a piece of an even share costs besides its keys, in blocks of them: more of the 64-wide ones, which are shorter,
// and more again where two CTAs per SM instead of three hide it. Microseconds with 2, 3, 4, 6 and 8, 4 or 12 query rows
// per key head, lengths drawn from a tenth of the longest on:
//   rows x width   64 of up to 4096 keys     200 of up to 3000     48 of up to 32768     9 of up to 5001
//    8 x 128       47.5 45.9 46.4 48.5 49.5  101  97  99 101 104   195 193 194 197 199   17.2 16.7 16.8 19.1 22.1
//   16 x 128       75.0 71.8 70.2 70.9 73.6  170 161 155 159 162   306 302 303 304 307   23.4 23.4 23.3 23.4 23.5
//    8 x 64        31.8 30.5 30.6 31.2 32.4   70  65  65  66  67   121 119 119 120 122   13.3 12.6 12.6 14.2 15.5
//   16 x 64        52.0 50.6 47.5 45.2 46.6  117 110 105 101 102   186 181 180 177 179   15.3 15.2 15.3 15.2 15.2
// Calls of equal lengths take the same within 4 % with 2 to 4.
__host__ __device__ constexpr int piece_cost(int head_dim, int rows) {
  return head_dim == 128 ? 3 : rows == 8 ? 4 : 6;
}

Plan make_plan(const Cache4AttnArgs& a) {
  Plan p;
  const long long G = a.heads_q / a.c.heads, rows = (long long)a.max_q * G, heads = (long long)a.seqs * a.c.heads;
  p.rows = (int)(rows < (1ll << 30) ? rows : (1ll << 30));
  p.tile = rows <= 8 ? 8 : 16;
  p.tiles = (p.rows + p.tile - 1) / p.tile;
  // Runs that give every SM as many CTAs as it holds where the keys allow it, of 128 keys at least: one more waits for a second
  // round (one token over 32768 keys 25.3 us in six per SM, 19.0 in three). Up to 512 keys one run, without the second
  // kernel (16 tokens over up to 300 keys 9.0 us in two runs, 6.5 in one; over 1000 9.7 in one, 7.1 in eight), and runs of
  // at most 4096, so that ragged lengths even out (1024 cost 13 % more at 64 x 8192: a run takes ~3 us besides its keys).
  const long long items = heads * p.tiles < (1ll << 30) ? heads * p.tiles : (1ll << 30);
  const int slots = ctas_per_sm(p.tile) * kSMs;
  long long chunk = (long long)a.max_k * items / slots;
  if (chunk > 4096) chunk = 4096;
  if (chunk < kKeys) chunk = kKeys;
  if (a.max_k <= 512) chunk = a.max_k;
  // no more than 2^17 rows of parts (68 MB): splits <= 2^16 / rows + 1, one split past 2^16 rows
  const long long all = heads <= (1 << 16) ? heads * p.rows : (1 << 17);
  const long long least = all <= (1 << 16) ? ((a.max_k * all) >> 16) + 1 : a.max_k;
  if (chunk < least) chunk = least;
  if (chunk > a.max_k) chunk = a.max_k;
  if (chunk < 1) chunk = 1;
  p.chunk = (int)((chunk + kKeys - 1) / kKeys * kKeys);
  p.splits = (a.max_k + p.chunk - 1) / p.chunk;
  if (p.splits < 1) p.splits = 1;
  // A cluster joins its runs without a second kernel: one token over 1000 keys 7.1 -> 5.9 us, over 4000 in eight runs instead
  // of 32 9.4 -> 8.0 (over 8000 in eight it would be 11.3 instead of 10.8). Only while all of them run at once: clusters
  // wait for places side by side and for their longest run (8 x 4096 tokens 16.0 -> 21 us, 48 ragged ones 187 -> 325).
  if (p.splits > 8 && a.max_k <= 4096 && items * 8 <= 2 * kSMs) {
    p.chunk = ((a.max_k + 7) / 8 + kKeys - 1) / kKeys * kKeys;
    p.splits = (a.max_k + p.chunk - 1) / p.chunk;
  }
  p.cluster = p.splits > 1 && p.splits <= 8 && items * p.splits <= 2 * kSMs;
  // Longer calls of few rows share all keys out evenly over the CTAs that run at once, from 512 keys each on and for sequences
  // that may be longer than 2048 (48 tokens over up to 32768 keys 186 -> 151 us, 32 over up to 8192 57.9 -> 40.8, 64 over 8192
  // each 127.8 -> 120; 8 over 4096 each, 574 keys per CTA, 16.4 and 15.9; many short sequences are better off with a CTA each,
  // whose starts overlap: 200 of up to 2000 70.8 and 75.4, 1000 of up to 400 129 and 148).
  const long long blocks = heads * ((a.max_k + kKeys - 1) / kKeys + 1 + piece_cost(a.c.head_dim, p.tile));
  p.even = p.tiles == 1 && !p.cluster && a.seqs <= 1024 && a.max_k > 2048 && a.max_k * heads >= 512 * slots && blocks < (1 << 30)
               ? slots : 0;
  const long long most = (1ll << 30) / (heads * p.splits);
  p.walk = p.tiles < most ? p.tiles : (int)(most < 1 ? 1 : most);
  return p;
}

struct Parts {
  size_t ml, o, cuts, total;
};
Parts parts_of(const Plan& p, const Cache4AttnArgs& a) {
  const size_t n = p.even ? (size_t)2 * p.even * p.rows
                          : p.splits > 1 && !p.cluster ? (size_t)a.seqs * a.c.heads * p.splits * p.rows : 0;
  Parts l;
  l.ml = 0;
  l.o = (n * 8 + 255) & ~size_t(255);
  l.cuts = l.o + n * (size_t)a.c.head_dim * 4;
  l.total = l.cuts + (size_t)p.even * sizeof(Cut);
  return l;
}

struct Span {
  int q0, nq, nk;
  bool ok;
};
__device__ __forceinline__ Span load_span(const Cache4AttnArgs& a, int s) {
  Span r;
  r.q0 = a.q_off[s];
  const long long nq = a.q_len ? (long long)a.q_len[s] : (long long)a.q_off[s + 1] - r.q0;
  r.nk = a.k_len[s];
  r.ok = r.q0 >= 0 && nq >= 0 && nq <= a.max_q && r.q0 + nq <= a.rows_q && r.nk >= 0 && r.nk <= a.max_k;
  r.nq = r.ok ? (int)nq : 0;
  return r;
}

// Keys that the query rows [base, base + rows) of a sequence see: those of the last one.
__device__ __forceinline__ int keys_seen(const Cache4AttnArgs& a, const Span& sp, int G, int base, int rows) {
  if (!a.causal) return sp.nk;
  return min(sp.nk, max(0, (base + rows - 1) / G + sp.nk - sp.nq + 1));
}

// ---- even shares: all blocks of 128 keys of all sequences and key heads in a row, as much of them to each CTA ---------

// Of a head of sequence s: its blocks and what comes on top, or zero. Queries without keys have one.
template <int kCost>
__device__ __forceinline__ int cost_of(const Cache4AttnArgs& a, int s) {
  if (s >= a.seqs) return 0;
  const Span sp = load_span(a, s);
  return sp.nq == 0 ? 0 : max(1, (sp.nk + kKeys - 1) / kKeys) + kCost;
}

struct Share {
  int per;     // what a CTA has of it
  int before;  // of a head of the sequences before `seq`
  int seq, n;  // a sequence and its own
};

// The share's size, and the sequence that holds the first block of the CTA's (a.seqs: there is none). One warp, all lanes the
// same; the lengths of 128 sequences are fetched at once.
template <int kCost>
__device__ __forceinline__ Share find_share(const Cache4AttnArgs& a, int ctas, int cta, int lane) {
  int all = 0, n[4];
  for (int s0 = 0; s0 < a.seqs; s0 += 128) {
#pragma unroll
    for (int i = 0; i < 4; ++i) n[i] = cost_of<kCost>(a, s0 + 32 * i + lane);
    all += n[0] + n[1] + n[2] + n[3];
  }
  all = __reduce_add_sync(0xffffffffu, all);
  Share r;
  // at least what comes on top and one block, so that a share which begins with a head has some of its keys (shares of seven or
  // ten blocks at least: 9 tokens over up to 5001 of 128-wide heads 16.7 us -> 19.4 and 22.5, of 64-wide ones 12.6 -> 13.9, 15.7)
  r.per = max(kCost + 1, (int)((unsigned)(all * a.c.heads + ctas - 1) / (unsigned)ctas));
  r.before = 0;
  r.seq = a.seqs, r.n = 0;
  for (int s0 = 0; s0 < a.seqs; s0 += 128) {
    if (a.seqs > 128) {
#pragma unroll
      for (int i = 0; i < 4; ++i) n[i] = cost_of<kCost>(a, s0 + 32 * i + lane);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      int upto = n[i];
#pragma unroll
      for (int w = 1; w < 32; w <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, upto, w);
        if (lane >= w) upto += t;
      }
      const uint32_t hit = __ballot_sync(0xffffffffu, (unsigned)((r.before + upto) * a.c.heads) > (unsigned)(cta * r.per));
      if (hit) {
        const int l = __ffs(hit) - 1;
        r.seq = s0 + 32 * i + l;
        r.n = __shfl_sync(0xffffffffu, n[i], l);
        r.before += __shfl_sync(0xffffffffu, upto - n[i], l);
        return r;
      }
      r.before += __shfl_sync(0xffffffffu, upto, 31);
    }
  }
  return r;
}

// What a CTA does at a time: of a sequence and key head the keys from block `block` on.
struct Piece {
  int seq, head, q0, nq, nk;
  int block, keys;           // keys < 0: nothing is left
  int whole;                 // these are all keys
  int n, left, per;          // even shares: blocks of the sequence, what is left of the share at its first block, a share
  long long row;             // of the parts
  __device__ __forceinline__ void of(const Cache4AttnArgs& a, int s) {
    const Span sp = load_span(a, s);
    seq = s, q0 = sp.q0, nq = sp.nq, nk = sp.nk;
  }
  __device__ __forceinline__ void cut(const Params& P) {
    const int count = min(n - block, left);
    keys = count > 0 ? count * kKeys : -1;
    whole = count == n;
    row = (long long)(2 * blockIdx.x + (block + count == n ? 0 : 1)) * P.rows;
  }
  template <int kCost>
  __device__ __forceinline__ void next(const Params& P) {
    left -= keys / kKeys + kCost;
    block = 0;
    if (left > 0 && ++head == P.a.c.heads) {
      head = 0;
      int cost;
      do cost = cost_of<kCost>(P.a, ++seq);
      while (cost == 0 && seq < P.a.seqs);
      n = cost == 0 ? 0 : cost - kCost;
      if (n > 0) of(P.a, seq);
    }
    cut(P);
  }
};

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// The same from an accumulator of zeros.
__device__ __forceinline__ void mma_f16_new(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]), "f"(0.f));
}
__device__ __forceinline__ void mma_bf16_new(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]), "f"(0.f));
}

__device__ __forceinline__ float2 ld_cluster(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Both halves of an fp16 pair added in fp32.
template <int N>
__device__ __forceinline__ void add_f16x2(float (&s)[N], uint32_t v) {
  asm("{\n\t.reg .f16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tadd.rn.f32.f16 %0, lo, %0;\n\tadd.rn.f32.f16 %1, hi, %1;\n\t}"
      : "+f"(s[0]), "+f"(s[1])
      : "r"(v));
}

__device__ __forceinline__ float lg2_approx(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// bf16 pairs, both halves' larger ones (a NaN loses).
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

template <int D>
struct Stage {  // 128 tokens of one head: pages of up to 64 tokens as they lie in the cache, larger ones' parts
  static constexpr int G = D / 32;
  static constexpr uint32_t kBytes = kKeys * D * 9 / 8;
};

// Where a lane finds what it reads of a warp's first tile of 16 tokens in a stage: bytes from the stage's start.
struct Places {
  int key_codes, key_scales, value_codes, value_scales;
};

template <int N>  // N words at once, N = 1, 2 or 4
__device__ __forceinline__ void lds(uint32_t (&w)[N], const uint8_t* at) {
  if constexpr (N == 4) {
    const uint4 u = *reinterpret_cast<const uint4*>(at);
    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
  } else if constexpr (N == 2) {
    const uint2 u = *reinterpret_cast<const uint2*>(at);
    w[0] = u.x, w[1] = u.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(at);
  }
}

template <int N>  // scales of bf16 pairs
__device__ __forceinline__ void scales(float (&s)[2 * N], const uint32_t (&w)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    s[2 * i] = __uint_as_float(w[i] << 16);
    s[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// What a warp keeps of its query rows: columns 8 n + c0 + {0, 1} of the scores and the output, c0 = 2 (lane % 4).
template <int D, int NT, bool kLong>
struct Rows {
  static constexpr int G = D / 32;
  static constexpr bool kAdds = kLong || NT == 2;  // how sums of f are taken
  static constexpr int kF = kAdds ? 2 : 4;
  uint32_t q[NT][2 * G][2];  // the queries as the scores' column operand
  uint32_t eight[NT][2];     // -8 sums of their groups, in three bf16 parts
  float scale[NT][2];        // from sums of products to exponents of two
  int limit[NT][2];          // keys that the columns see
  float o[NT][2 * G][4], f[NT][G][kF];  // sums of c f, times 2^-24 (the codes' odd places: 2^-20), and of f
  float m[NT][2], l[NT][2];            // what exponents are taken from, sums of probabilities
};

constexpr float kRoom = 6.0f;  // a row's largest weight lies 2^6 above its reference when that is set, 2^15 at most

// A warp's 32 tokens of a stage, from token t0 of the sequence on. kMasked: some column does not see some of them. kSmall: the
// two tiles are pages of 16 tokens each, not neighbours in one.
template <int D, int NT, bool kMasked, bool kSmall, bool kLong>
__device__ __forceinline__ void attend(Rows<D, NT, kLong>& R, const uint8_t* stage, const Places& at, int t0, uint32_t here, int last,
                                       int lane) {
  constexpr int G = Stage<D>::G;
  constexpr int kCodesOn = kSmall ? 16 * D * 9 / 8 : 16 * D / 2, kScalesOn = kSmall ? 16 * D * 9 / 8 : 16 * G * 2;
  const int r0 = lane >> 2, odd = lane & 2 ? -(D / 2) : D / 2;
  // whether column e of n sees this lane's token r0 + 8 h of tile i
  auto sees = [&](int i, int n, int h, int e) {
    return ((here >> i) & 1u) && t0 + i * 16 + r0 + 8 * h < min(R.limit[n][e], last);
  };
  float x[2][NT][4];           // scores, then probabilities, of two tiles of 16 tokens
  uint32_t vs[2][2][G / 2];    // scales of the values of the tokens r0 and r0 + 8
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint8_t *codes = stage + at.key_codes + i * kCodesOn, *sc = stage + at.key_scales + i * kScalesOn;
    lds<G / 2>(vs[i][0], stage + at.value_scales + i * kScalesOn);
    lds<G / 2>(vs[i][1], stage + at.value_scales + i * kScalesOn + 8 * (G * 2));
    uint32_t lo[G], hi[G], wlo[G / 2], whi[G / 2];  // codes and scales of the tokens r0 and r0 + 8
    lds<G>(lo, codes);
    lds<G>(hi, codes + 8 * (D / 2));
    lds<G / 2>(wlo, sc);
    lds<G / 2>(whi, sc + 8 * (G * 2));
    {
      const bool odd = G == 4 && (lane & 1);
      const uint32_t u = wlo[odd ? G / 2 - 1 : 0], w = whi[odd ? G / 2 - 1 : 0], A[4] = {u, w, u, w};
#pragma unroll
      for (int n = 0; n < NT; ++n) mma_bf16_new(x[i][n], A, R.eight[n]);
    }
    float slo[G], shi[G];
    scales<G / 2>(slo, wlo);
    scales<G / 2>(shi, whi);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      float acc[NT][4];
      const uint32_t A[4] = {lo[g] & 0x000f000fu, hi[g] & 0x000f000fu, lo[g] & 0x00f000f0u, hi[g] & 0x00f000f0u};
      const uint32_t l8 = lo[g] >> 8, h8 = hi[g] >> 8;
      const uint32_t B[4] = {l8 & 0x000f000fu, h8 & 0x000f000fu, l8 & 0x00f000f0u, h8 & 0x00f000f0u};
#pragma unroll
      for (int n = 0; n < NT; ++n) mma_f16_new(acc[n], A, R.q[n][2 * g]);
#pragma unroll
      for (int n = 0; n < NT; ++n) mma_f16(acc[n], B, R.q[n][2 * g + 1]);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        x[i][n][0] = fmaf(slo[g], acc[n][0], x[i][n][0]);
        x[i][n][1] = fmaf(slo[g], acc[n][1], x[i][n][1]);
        x[i][n][2] = fmaf(shi[g], acc[n][2], x[i][n][2]);
        x[i][n][3] = fmaf(shi[g], acc[n][3], x[i][n][3]);
      }
    }
  }
  if constexpr (kMasked) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (!sees(i, n, e >> 1, e & 1)) x[i][n][e] = -INFINITY;
  }
  // References move rarely: only where a weight could pass 2^8 times what it was when the reference was set. The check
  // takes the largest score and the largest scale of the lane's four tokens together, which errs on that side.
  auto largest = [](const uint32_t (&w)[G / 2]) {
    uint32_t u = w[0];
    if constexpr (G == 4) u = max2(w[0], w[1]);
    return u;
  };
  auto exponent = [](uint32_t u) {
    const float s = fmaxf(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    return fmaxf(lg2_approx(s), -64.0f);
  };
  const float most = exponent(max2(max2(largest(vs[0][0]), largest(vs[0][1])), max2(largest(vs[1][0]), largest(vs[1][1]))));
  bool move = false;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float top = fmaxf(fmaxf(x[0][n][e], x[0][n][e + 2]), fmaxf(x[1][n][e], x[1][n][e + 2]));
      move = move || fmaf(top, R.scale[n][e], most) > R.m[n][e] + (kRoom + 8.0f);  // also from minus infinity
    }
  if (__any_sync(0xffffffffu, move)) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float alpha[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) top = fmaxf(top, fmaf(x[i][n][e + 2 * h], R.scale[n][e], exponent(largest(vs[i][h]))));
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
        const float mn = fmaxf(R.m[n][e], top - kRoom);
        const float by = R.m[n][e] - (mn == -INFINITY ? 0.f : mn);
        alpha[e] = ex2_approx(by);
        R.m[n][e] = mn;
        R.l[n][e] = rescaled(R.l[n][e], by);
      }
#pragma unroll
      for (int g = 0; g < G; ++g) {
        R.f[n][g][0] *= alpha[0];
        R.f[n][g][1] *= alpha[1];
        if constexpr (!R.kAdds) R.f[n][g][2] = R.f[n][g][3] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 2 * G; ++i) {
        R.o[n][i][0] *= alpha[0];
        R.o[n][i][1] *= alpha[1];
        R.o[n][i][2] *= alpha[0];
        R.o[n][i][3] *= alpha[1];
      }
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float ref = R.m[n][e] == -INFINITY ? 0.f : R.m[n][e];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x[i][n][e] = ex2_approx(fmaf(x[i][n][e], R.scale[n][e], -ref));
        x[i][n][e + 2] = ex2_approx(fmaf(x[i][n][e + 2], R.scale[n][e], -ref));
        R.l[n][e] += x[i][n][e] + x[i][n][e + 2];
      }
    }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    // codes of the tokens c0, c0 + 1, c0 + 8 and c0 + 9: this lane's columns of V^T. Half of the lanes fetch the odd ones
    // first, so that the four rows of a load lie in other banks (half as many conflicts), and pick them the other way round.
    const uint8_t* row = stage + at.value_codes + i * kCodesOn;
    uint32_t w0[G / 2], w1[G / 2], w2[G / 2], w3[G / 2];
    lds<G / 2>(w0, row);
    lds<G / 2>(w1, row + odd);
    lds<G / 2>(w2, row + 8 * (D / 2));
    lds<G / 2>(w3, row + 8 * (D / 2) + odd);
    float slo[G], shi[G];
    scales<G / 2>(slo, vs[i][0]);
    scales<G / 2>(shi, vs[i][1]);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      uint32_t b[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float f[4] = {x[i][n][0] * slo[g], x[i][n][1] * slo[g], x[i][n][2] * shi[g], x[i][n][3] * shi[g]};
        if constexpr (kMasked) {  // a probability of zero does not silence a scale that is not finite
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!sees(i, n, e >> 1, e & 1)) f[e] = 0.f;
        }
        const uint32_t lo = pack_f16x2(f[0], f[1]), hi = pack_f16x2(f[2], f[3]);
        if constexpr (R.kAdds) {
          add_f16x2(R.f[n][g], lo);
          add_f16x2(R.f[n][g], hi);
        }
        b[n][0] = transpose8x8(lo);
        b[n][1] = transpose8x8(hi);
        if constexpr (!R.kAdds) {
          const uint32_t one[4] = {0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u};
          mma_f16(R.f[n][g], one, b[n]);  // rows 8 to 15 are the same again
        }
      }
      // the codes' low bytes of the group's half-words, then the high ones
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t pick = (lane & 2 ? 0x0044u : 0x0440u) + (uint32_t)(2 * (g & 1) + h) * 0x0101u;
        const uint32_t near = __byte_perm(w0[g / 2], w1[g / 2], pick), far = __byte_perm(w2[g / 2], w3[g / 2], pick);
        const uint32_t A[4] = {near & 0x000f000fu, near & 0x00f000f0u, far & 0x000f000fu, far & 0x00f000f0u};
#pragma unroll
        for (int n = 0; n < NT; ++n) mma_f16(R.o[n][2 * g + h], A, b[n]);
      }
    }
  }
}

// Brings a run's stages of 128 tokens in. Pages of up to 64 tokens come whole, lane i the i-th of a stage; of larger ones lane
// `part` brings a part (codes or scales, of the keys or the values). Copies this large matter: a page of 16 tokens in
// four of them kept the copy unit busy for as long as the arithmetic.
template <int D>
struct Sender {
  static constexpr int G = D / 32;
  const uint8_t* heads;  // this head of page 0
  const int32_t* table;
  uint8_t* smem;
  uint64_t *full, *empty;
  uint32_t* live;
  const WaitCtx* wc;
  long long page_bytes;
  int pages, shift, first, last, blocks, used, lane, width, slab, part, t0, each, src0, dst0, sent;
  bool whole;

  Sender() = default;
  __device__ __forceinline__ Sender(const Params& P, const WaitCtx& w, uint8_t* smem_, uint64_t* full_, uint64_t* empty_,
                                    uint32_t* live_, int seq, int hk, int first_, int last_, int blocks_, int used_, int lane_)
      : smem(smem_), full(full_), empty(empty_), live(live_), wc(&w), first(first_), last(last_), blocks(blocks_), used(used_),
        lane(lane_) {
    const Cache4& c = P.a.c;
    pages = c.pages, shift = c.page_shift, slab = c.slab(), sent = -1;
    const int ps = 1 << shift;
    width = min(ps, kKeys), whole = ps <= 64;
    part = whole ? 0 : lane, t0 = whole ? lane * ps : lane < 4 ? 0 : kKeys;
    each = part & 1 ? G * 2 : D / 2;  // bytes of a token in a part
    src0 = (part & 2 ? slab / 2 : 0) + (part & 1 ? c.code_bytes() : 0);
    dst0 = whole ? lane * slab : (part & 2 ? (int)Stage<D>::kBytes / 2 : 0) + (part & 1 ? kKeys * D / 2 : 0);
    heads = P.a.cache + (long long)hk * slab, page_bytes = (long long)c.heads * slab;
    table = P.a.table + (long long)seq * c.max_pages;
  }
  __device__ __forceinline__ int page_of(int j) const {
    const int t = first + j * kKeys + t0;
    return j < blocks && t0 < kKeys && t < last ? table[t >> shift] : -2;
  }
  // Block j, whose page of this lane is `page`, once its stage is free; false if that wait gave up.
  __device__ __forceinline__ bool send(int j, int page) {
    const int n = used + j, st = n % kStages, t = first + j * kKeys;
    const bool wanted = t0 < kKeys && t + t0 < last, ok = wanted && (uint32_t)page < (uint32_t)pages;
    uint32_t all = 0xffu, total = Stage<D>::kBytes, bytes = whole ? slab : kKeys * each;
    if (t + kKeys > last || __any_sync(0xffffffffu, wanted && !ok)) {  // not all of the stage
      if (wanted && !ok && part == 0) report_bad_entry(wc->status, kSiteCache4Page);
      const int tiles = ok ? (min(width, last - t - t0) + 15) / 16 : 0;  // of 16 tokens
      bytes = whole ? slab : tiles * 16 * each;
      all = __reduce_or_sync(0xffffffffu, part == 0 && ok ? ((1u << tiles) - 1u) << (t0 / 16) : 0u);
      total = __reduce_add_sync(0xffffffffu, ok ? bytes : 0u);
    }
    if (!__all_sync(0xffffffffu, mbar_wait_sleep(&empty[st], ((uint32_t)(n / kStages) & 1u) ^ 1u, *wc, kSiteCache4Empty))) return false;
    if (lane == 0) {
      live[st] = all;
      mbar_arrive_expect_tx(&full[st], total);
    }
    __syncwarp();
    if (ok)
      bulk_load(smem + st * Stage<D>::kBytes + dst0,
                heads + page * page_bytes + src0 + (whole ? 0 : ((t + t0) & ((1 << shift) - 1)) * each), bytes, &full[st]);
    sent = n;
    return true;
  }
  // After a wait that gave up: nothing leaves before this warp's copies on their way have landed (bounded).
  __device__ __forceinline__ void land() const {
    if (*wc->abort_flag && lane == 0 && sent >= 0) {
      const uint64_t t = global_timer_ns();
      for (int n = max(0, sent - kStages + 1); n <= sent; ++n)
        while (!mbar_try(&full[n % kStages], (uint32_t)(n / kStages) & 1u) && global_timer_ns() - t < 200000000ull) {
        }
    }
    __syncwarp();
  }
};

template <int D, int NT, bool kSmall, bool kEven>
__global__ void __launch_bounds__(kThreads<D, NT>, ctas_per_sm(8 * NT)) cache4_attention_kernel(const __grid_constant__ Params P) {
  using L = Stage<D>;
  constexpr int G = L::G, R = 8 * NT, V = D / 32, kCost = piece_cost(D, R);
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[kStages], empty[kStages];
  __shared__ uint32_t live[kStages];  // the tiles of 16 tokens that a stage holds
  __shared__ float2 ml[4][R], sums[R];
  __shared__ int abort_flag;
  __shared__ Piece piece;
  const Cache4AttnArgs& a = P.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, group = P.group;
  // the splits of a cluster side by side, or the tiles of the same keys
  const int side = !kEven && P.cluster ? P.splits : P.walk, at = blockIdx.x / side, in = blockIdx.x - at * side;
  const int over = at / (!kEven && P.cluster ? P.walk : P.splits), under = at - over * (!kEven && P.cluster ? P.walk : P.splits);
  const int split = !kEven && P.cluster ? in : under, tile0 = !kEven && P.cluster ? under : in;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 4);
    }
    abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  grid_dependency_wait();
  allow_dependents();
  Span sp;
  int hk = over % a.c.heads, seq = over / a.c.heads, first = split * P.chunk, keys = P.chunk;
  if constexpr (kEven) {
    if (warp == 0) {
      const int c = blockIdx.x;
      if (c == 0)
        for (int i = lane; i < a.seqs; i += 32)
          if (!load_span(a, i).ok) report_bad_entry(a.status, kSiteCache4Lengths);
      const Share h = find_share<kCost>(a, P.even, c, lane);
      if (lane == 0) {
        P.cuts[c].parts = 0;
        piece.keys = -1;
        piece.per = h.per;
        if (h.seq < a.seqs) {
          const int in = c * h.per - h.before * a.c.heads;
          piece.of(a, h.seq);
          piece.head = in / h.n, piece.n = h.n - kCost;
          const int at_cost = in % h.n - kCost;  // a share that begins in what comes on top begins with the first block
          piece.block = max(0, at_cost), piece.left = h.per + min(0, at_cost);
          piece.cut(P);
        }
      }
    }
    __syncthreads();
  } else {
    sp = load_span(a, seq);
    if (!sp.ok) {
      if (split == 0 && hk == 0 && tile0 == 0 && threadIdx.x == 0) report_bad_entry(a.status, kSiteCache4Lengths);
      return;
    }
  }
  const WaitCtx wc{a.status, &abort_flag, kWaitLimitNs};
  const int r0 = lane >> 2, c0 = (lane & 3) * 2;  // fragment row, and first of two columns
  int used = 0;  // stages filled (or emptied) so far

  for (int tile = kEven ? 0 : tile0; kEven || tile < P.tiles; tile += kEven ? 0 : P.walk) {
    if constexpr (kEven) {
      if (piece.keys < 0) break;
      seq = piece.seq, hk = piece.head, first = piece.block * kKeys, keys = piece.keys;
      sp = Span{piece.q0, piece.nq, piece.nk, true};
    }
    const int base = tile * R, rows = min(R, sp.nq * group - base);  // this tile's query rows
    if (rows <= 0) break;
    const int last = min(keys_seen(a, sp, group, base, rows), first + keys);
    if (!kEven && first >= last && split > 0 && !P.cluster) continue;
    const int blocks = first < last ? (last - first + kKeys - 1) / kKeys : 0;

    [[maybe_unused]] typename std::conditional<kOwn<D, NT>, Sender<D>, int>::type sender;
    [[maybe_unused]] int page = 0;
    if constexpr (kOwn<D, NT>) {
      sender = Sender<D>(P, wc, smem, full, empty, live, seq, hk, first, last, blocks, used, lane);
      if (warp < kAhead && warp < blocks) sender.send(warp, sender.page_of(warp));
      page = sender.page_of(warp + kAhead);  // of this warp's next turn: the blocks warp + kAhead, + 4, + 8, ...
    } else if (warp == 4) {
      Sender<D> only(P, wc, smem, full, empty, live, seq, hk, first, last, blocks, used, lane);
      page = only.page_of(0);
      for (int j = 0; j < blocks; ++j) {
        const int next = only.page_of(j + 1);
        if (!only.send(j, page)) break;
        page = next;
      }
      only.land();
    }

    Rows<D, NT, kEven> Q;
    if (warp < 4) {
      int open = last;  // keys below it are seen by all rows
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int r = base + n * 8 + r0, token = r / group;
        const bool ok = n * 8 + r0 < rows;
        const uint16_t* src = reinterpret_cast<const uint16_t*>(a.q) + (long long)(sp.q0 + (ok ? token : 0)) * a.ldq +
                              (hk * group + (ok ? r - token * group : 0)) * D + (lane & 3) * 8;
        uint32_t w[G][4], top = 0;
#pragma unroll
        for (int j = 0; j < G; ++j) {
          const uint4 u = ok ? *reinterpret_cast<const uint4*>(src + 32 * j) : make_uint4(0u, 0u, 0u, 0u);
          w[j][0] = u.x, w[j][1] = u.y, w[j][2] = u.z, w[j][3] = u.w;
#pragma unroll
          for (int e = 0; e < 4; ++e) top = max(top, max(w[j][e] & 0x7fffu, (w[j][e] >> 16) & 0x7fffu));
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^up takes the row's largest magnitude to [2^13, 2^14): its biased exponent to 140
        const int up = top == 0 ? 0 : min(140 - (int)max(top >> 7, 1u), 126);
        const float factor = __uint_as_float((uint32_t)(127 + up) << 23);
        float part[4 * 3];  // three bf16 parts of -8 sum(q) 2^-24, part p of group j at [p G + j]
#pragma unroll
        for (int i = 0; i < 12; ++i) part[i] = 0.f;
#pragma unroll
        for (int j = 0; j < G; ++j) {
          // values i and i + 4 side by side, as the keys' codes are; those of the higher codes divided by 16
          float v[8], sum = 0.f;
          uint32_t h[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = unpack_bf16x2(w[j][e]);
            v[2 * e] = f.x * factor;
            v[2 * e + 1] = f.y * factor;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float d = e & 1 ? 0.0625f : 1.0f;
            h[e] = pack_f16x2(v[e] * d, v[e + 4] * d);
            sum += v[e] + v[e + 4];
          }
          Q.q[n][2 * j][0] = h[0];
          Q.q[n][2 * j][1] = h[1];
          Q.q[n][2 * j + 1][0] = h[2];
          Q.q[n][2 * j + 1][1] = h[3];
          sum += __shfl_xor_sync(0xffffffffu, sum, 1);
          sum += __shfl_xor_sync(0xffffffffu, sum, 2);
          sum *= -8.0f * 0x1p-24f;
#pragma unroll
          for (int p = 0; p < 3; ++p) {
            const float f = __bfloat162float(__float2bfloat16(sum));
            part[p * G + j] = f;
            sum -= f;
          }
        }
        // rows 2 t, 2 t + 1 and 2 t + 8, 2 t + 9 of the column operand
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float lo = 0.f, hi = 0.f;
#pragma unroll
          for (int i = 0; i < 12; i += 2)
            if (i == c0 + 8 * h) lo = part[i], hi = part[i + 1];
          Q.eight[n][h] = pack_bf16x2(lo, hi);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int i = n * 8 + c0 + e;
          // never zero, whose product with the minus infinity of a key that is not seen would be NaN; what it adds to a factor below
          // fp32's smallest number is at most 2^-21 of an exponent
          Q.scale[n][e] = fmaxf(ldexpf(P.scale_log2, 24 - __shfl_sync(0xffffffffu, up, (c0 + e) * 4)), 0x1p-149f);
          Q.limit[n][e] = i < rows && a.causal ? min(sp.nk, (base + i) / group + sp.nk - sp.nq + 1) : sp.nk;
          open = min(open, Q.limit[n][e]);
          Q.m[n][e] = -INFINITY;
          Q.l[n][e] = 0.f;
#pragma unroll
          for (int g = 0; g < G; ++g)
#pragma unroll
            for (int i = e; i < Q.kF; i += 2) Q.f[n][g][i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 2 * G; ++i) Q.o[n][i][0] = Q.o[n][i][1] = Q.o[n][i][2] = Q.o[n][i][3] = 0.f;
      }
      open = min(open, __shfl_xor_sync(0xffffffffu, open, 1));
      open = min(open, __shfl_xor_sync(0xffffffffu, open, 2));

      Places at;
      {
        const int held_shift = min(a.c.page_shift, 7), held = 1 << held_shift;  // tokens of a page that a stage holds
        const int page = ((warp * 32) >> held_shift) * (held * (D * 9 / 8)), in = (warp * 32) & (held - 1);
        at.key_codes = page + (in + r0) * (D / 2) + (lane & 3) * (G * 4);
        at.key_scales = page + held * (D / 2) + (in + r0) * (G * 2);
        at.value_codes = page + held * (D * 9 / 16) + (in + c0 + (lane & 2 ? 1 : 0)) * (D / 2) + r0 * (G * 2);
        at.value_scales = at.key_scales + held * (D * 9 / 16);
      }
      int st = used % kStages, from = first + warp * 32;
      uint32_t phase = (uint32_t)(used / kStages) & 1u;
      const uint8_t* stage = smem + st * L::kBytes;
#pragma unroll 1
      for (int j = 0; j < blocks; ++j) {
        if constexpr (kOwn<D, NT>) {
          if ((j & 3) == warp && j + kAhead < blocks) {
            sender.send(j + kAhead, page);
            page = sender.page_of(j + kAhead + 4);
          }
        }
        bool ok = mbar_wait(&full[st], phase, wc, kSiteCache4Full);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t here = (live[st] >> (2 * warp)) & 3u;
        if (here == 3u && from + 32 <= open) attend<D, NT, false, kSmall, kEven>(Q, stage, at, from, here, last, lane);
        else if (here) attend<D, NT, true, kSmall, kEven>(Q, stage, at, from, here, last, lane);
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
        from += kKeys;
        stage += L::kBytes;
        if (++st == kStages) {
          st = 0;
          phase ^= 1u;
          stage = smem;
        }
      }
      // From sums of codes to values: 8 sums of f off, the codes' powers of two undone.
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int w = 4; w < 32; w <<= 1) Q.l[n][e] += __shfl_xor_sync(0xffffffffu, Q.l[n][e], w);
#pragma unroll
          for (int g = 0; g < G; ++g) {
            float f = Q.f[n][g][e];
#pragma unroll
            for (int w = 4; w < 32 && Q.kAdds; w <<= 1) f += __shfl_xor_sync(0xffffffffu, f, w);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              Q.o[n][2 * g + h][e] = fmaf(Q.o[n][2 * g + h][e], 0x1p24f, -8.0f * f);
              Q.o[n][2 * g + h][e + 2] = fmaf(Q.o[n][2 * g + h][e + 2], 0x1p20f, -8.0f * f);
            }
          }
        }
    }
    if constexpr (kOwn<D, NT>) sender.land();
    used += blocks;

    // The four warps' rows through shared memory: all stages have been read.
    __syncthreads();
    // even shares: read again, since the loop has no registers for them
    const int at0 = kEven ? 0 : base, many = kEven ? min(R, piece.nq * group) : rows;
    const int head = kEven ? piece.head : hk, q0 = kEven ? piece.q0 : sp.q0;
    // this CTA has all the keys of its rows; the first row of its parts
    const bool whole = kEven ? piece.whole : !P.cluster && sp.nk <= P.chunk;
    const long long row0 = kEven ? piece.row : ((long long)over * P.splits + split) * P.rows;
    float* parts = reinterpret_cast<float*>(smem);  // [warp][row][dim]
    float* mine = parts + 4 * R * D;                 // a cluster's: this run's rows
    if (warp < 4) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = n * 8 + c0 + e;
          if (r0 == 0) ml[warp][r] = make_float2(Q.m[n][e], Q.l[n][e]);
          if (r < many) {
#pragma unroll
            for (int i = 0; i < 2 * G; ++i)
              *reinterpret_cast<float2*>(parts + (warp * R + r) * D + (i >> 1) * 32 + 4 * r0 + 2 * (i & 1)) =
                  make_float2(Q.o[n][i][e], Q.o[n][i][e + 2]);
          }
        }
    }
    __syncthreads();
    if (warp < 4 && !abort_flag) {
      for (int r = warp; r < many; r += 4) {
        float mr = -INFINITY, lr = 0.f, out[V];
#pragma unroll
        for (int w = 0; w < 4; ++w) mr = fmaxf(mr, ml[w][r].x);
        const float ref = mr == -INFINITY ? 0.f : mr;
#pragma unroll
        for (int e = 0; e < V; ++e) out[e] = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float2 y = ml[w][r];
          if (y.y == 0.f) continue;  // no key that the row sees
          const float by = (y.x == -INFINITY ? 0.f : y.x) - ref, f = ex2_approx(by);
          lr += rescaled(y.y, by);
#pragma unroll
          for (int e = 0; e < V; ++e) out[e] += f * parts[(w * R + r) * D + lane * V + e];
        }
        if (whole) {
          const int token = (at0 + r) / group, g = at0 + r - token * group;
          const float inv = lr == 0.f ? 0.f : 1.0f / lr;
          bf16* dst = a.out + (long long)(q0 + token) * a.ldo + (head * group + g) * D + lane * V;
#pragma unroll
          for (int e = 0; e < V; e += 2)
            *reinterpret_cast<uint32_t*>(dst + e) = lr == 0.f ? 0u : pack_bf16x2(out[e] * inv, out[e + 1] * inv);
        } else if (!kEven && P.cluster) {
          if (lane == 0) sums[r] = make_float2(mr, lr);
#pragma unroll
          for (int e = 0; e < V; e += 2) *reinterpret_cast<float2*>(mine + r * D + lane * V + e) = make_float2(out[e], out[e + 1]);
        } else {
          const long long to = row0 + at0 + r;
          if (lane == 0) P.ml[to] = make_float2(mr, lr);
#pragma unroll
          for (int e = 0; e < V; e += 2)
            *reinterpret_cast<float2*>(P.o + to * D + lane * V + e) = make_float2(out[e], out[e + 1]);
        }
      }
    }
    if (!kEven && P.cluster) {
      // Every rank adds every splits-th row up over all runs, in order, one row per warp.
      cluster_sync_all();
      for (int r = split + warp * P.splits; warp < 4 && r < many; r += 4 * P.splits) {
        float2 y[8];
        float mr = -INFINITY, lr = 0.f, out[V];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          y[k] = make_float2(-INFINITY, 0.f);
          if (k < P.splits) y[k] = ld_cluster(map_to_rank(smem_u32(&sums[r]), k));
          mr = fmaxf(mr, y[k].x);
        }
        const float ref = mr == -INFINITY ? 0.f : mr;
        float v[8][V];
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
          for (int e = 0; e < V; e += 2) {
            const float2 t = k < P.splits ? ld_cluster(map_to_rank(smem_u32(mine + r * D + lane * V + e), k)) : make_float2(0.f, 0.f);
            v[k][e] = t.x;
            v[k][e + 1] = t.y;
          }
#pragma unroll
        for (int e = 0; e < V; ++e) out[e] = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (y[k].y == 0.f) continue;  // no key that the row sees
          const float by = (y[k].x == -INFINITY ? 0.f : y[k].x) - ref, f = ex2_approx(by);
          lr += rescaled(y[k].y, by);
#pragma unroll
          for (int e = 0; e < V; ++e) out[e] += f * v[k][e];
        }
        const int token = (at0 + r) / group, g = at0 + r - token * group;
        const float inv = lr == 0.f ? 0.f : 1.0f / lr;
        bf16* dst = a.out + (long long)(q0 + token) * a.ldo + (head * group + g) * D + lane * V;
        if (!abort_flag) {
#pragma unroll
          for (int e = 0; e < V; e += 2)
            *reinterpret_cast<uint32_t*>(dst + e) = lr == 0.f ? 0u : pack_bf16x2(out[e] * inv, out[e + 1] * inv);
        }
      }
      __syncwarp();
      cluster_sync_all();  // no rank goes on while another reads its rows
    }
    if (kEven || P.walk < P.tiles) fence_proxy_async_smem();  // before the next tile's copies
    if (kEven && threadIdx.x == 0) {
      const int done = piece.keys / kKeys;
      if (piece.block == 0 && done < piece.n && !abort_flag)
        P.cuts[blockIdx.x] = Cut{piece.head, piece.q0, piece.nq, 1 + (piece.n - done + piece.per - 1) / piece.per};
      piece.template next<kCost>(P);
    }
    __syncthreads();
    if ((kEven || !P.cluster) && abort_flag) return;
  }
}

// Adds up the runs of the sequences that took several, in order: one warp per row, grid (sequence and key head, or the share
// where they begin, four rows).
template <int D>
__global__ void __launch_bounds__(128) cache4_join_kernel(const __grid_constant__ Params P) {
  grid_dependency_wait();
  allow_dependents();
  const Cache4AttnArgs& a = P.a;
  const int G = P.group, lane = threadIdx.x & 31;
  if (P.even) {
    const Cut cut = P.cuts[blockIdx.x];
    const int r = blockIdx.y * 4 + (threadIdx.x >> 5), token = r / G, first = blockIdx.x, end = first + cut.parts - 1;
    if (cut.parts == 0 || r >= cut.nq * G) return;
    // the last part is the first piece of its CTA, the others the last ones of theirs
    join_row<D, true>(P.ml + r, P.o + (long long)r * D,
                [&](int i) { return (long long)(2 * (first + i) + (first + i < end ? 1 : 0)) * P.rows; }, cut.parts, lane,
                a.out + (long long)(cut.q0 + token) * a.ldo + (cut.head * G + r - token * G) * D);
    return;
  }
  const int hk = blockIdx.x % a.c.heads, seq = blockIdx.x / a.c.heads;
  const Span sp = load_span(a, seq);
  if (!sp.ok) return;
  if (sp.nk <= P.chunk) return;
  const int tile = P.rows <= 8 ? 8 : 16;
  for (int r = blockIdx.y * 4 + (threadIdx.x >> 5); r < sp.nq * G; r += gridDim.y * 4) {
    const int base = r / tile * tile;
    const int seen = keys_seen(a, sp, G, base, min(tile, sp.nq * G - base)), runs = (seen + P.chunk - 1) / P.chunk;
    const long long at = (long long)blockIdx.x * P.splits * P.rows + r;
    const int token = r / G;
    join_row<D, true>(P.ml + at, P.o + at * D, P.rows, max(1, runs), lane,
                a.out + (long long)(sp.q0 + token) * a.ldo + (hk * G + r - token * G) * D);
  }
}

template <int D, int NT, bool kSmall, bool kEven>
cudaError_t launch_attention_as(const Cache4AttnArgs& a, const Plan& p, cudaStream_t s) {
  static std::atomic<bool> raised[16];  // per device
  Params P;
  memset(&P, 0, sizeof(P));
  const Parts l = parts_of(p, a);
  uint8_t* ws = reinterpret_cast<uint8_t*>(a.parts);
  P.a = a;
  P.group = a.heads_q / a.c.heads;
  P.rows = p.rows;
  P.tiles = p.tiles;
  P.walk = p.walk;
  P.chunk = p.chunk;
  P.splits = p.splits;
  P.cluster = p.cluster;
  P.even = p.even;
  P.scale_log2 = (float)(1.4426950408889634 * (double)a.scale);
  P.ml = reinterpret_cast<float2*>(ws + l.ml);
  P.o = reinterpret_cast<float*>(ws + l.o);
  P.cuts = reinterpret_cast<Cut*>(ws + l.cuts);
  constexpr size_t smem = kStages * Stage<D>::kBytes;
  static_assert(smem >= 5 * 8 * NT * D * 4, "the parts reuse the stages");
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 16 || !raised[dev].load(std::memory_order_acquire)) {
    const cudaError_t e =
        cudaFuncSetAttribute(cache4_attention_kernel<D, NT, kSmall, kEven>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    if (dev < 16) raised[dev].store(true, std::memory_order_release);
  }
  const long long heads = (long long)a.seqs * a.c.heads;
  {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.even ? (unsigned)p.even : (unsigned)(heads * p.splits * p.walk));
    cfg.blockDim = dim3(kThreads<D, NT>);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (pdl_enabled()) {
      attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (p.cluster) {
      attr[n].id = cudaLaunchAttributeClusterDimension;
      attr[n].val.clusterDim.x = (unsigned)p.splits;
      attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
      ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    LaunchScope scope(kClsCache4Attention, s);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, cache4_attention_kernel<D, NT, kSmall, kEven>, P);
    if (e != cudaSuccess) return e;
  }
  if (p.even || (p.splits > 1 && !p.cluster)) {
    const int fours = (p.rows + 3) / 4;
    LaunchScope scope(kClsCache4Join, s);
    return launch_k(cache4_join_kernel<D>, dim3(p.even ? (unsigned)p.even : (unsigned)heads, (unsigned)(fours < 65535 ? fours : 65535)), dim3(128), 0, s, P);
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_cache4_append(const Cache4MoveArgs& a, cudaStream_t s) {
  return launch_move<true>(a, kClsCache4Append, s);
}

cudaError_t launch_cache4_read(const Cache4MoveArgs& a, cudaStream_t s) {
  return launch_move<false>(a, kClsCache4Read, s);
}

size_t cache4_attention_parts_bytes(const Cache4AttnArgs& a) {
  if (a.seqs == 0 || a.rows_q == 0 || a.max_q == 0) return 0;
  return parts_of(make_plan(a), a).total;
}

cudaError_t launch_cache4_attention(const Cache4AttnArgs& a, cudaStream_t s) {
  const Plan p = make_plan(a);
  const bool small = a.c.page_shift == 4, eight = p.tile == 8;
  auto of = [&](auto d, auto small_page) {
    constexpr int D = decltype(d)::value;
    constexpr bool kSmall = decltype(small_page)::value;
    if (p.even) return eight ? launch_attention_as<D, 1, kSmall, true>(a, p, s) : launch_attention_as<D, 2, kSmall, true>(a, p, s);
    return eight ? launch_attention_as<D, 1, kSmall, false>(a, p, s) : launch_attention_as<D, 2, kSmall, false>(a, p, s);
  };
  using D64 = std::integral_constant<int, 64>;
  using D128 = std::integral_constant<int, 128>;
  if (a.c.head_dim == 64) return small ? of(D64{}, std::true_type{}) : of(D64{}, std::false_type{});
  return small ? of(D128{}, std::true_type{}) : of(D128{}, std::false_type{});
}

}  // namespace dit
