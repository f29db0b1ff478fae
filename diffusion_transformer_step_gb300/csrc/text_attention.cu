// Attention with grouped heads over packed or padded sequences, causal or not: whole prompts,
// their last parts over a cache, single new tokens.
//
// The query heads that share a key head are rows of one tile: row r of a 128-row tile is query
// token r / G and head r % G of the group (G = heads_q / heads_k), so a key tile is read once for
// the whole group and a short sequence still fills its tile.  TQ = 128 / G tokens per tile; a work
// item is two tiles (2 TQ tokens) of one key head.  Up to 16 rows per key head in all (single new
// tokens), and small calls, take text_attention_few_kernel, further down.
//
// text_attention_kernel, one persistent CTA per SM, 352 threads, runs the two-tile pipeline of the
// joint attention: warp 0 loads (Q through a 4-D tensor map whose box is G heads x TQ tokens), warp
// 1 issues S_t = Q_t K^T and O_t += P_t V on tcgen05 with P read from Tensor Memory, warps 2-5 and
// 6-9 run one tile's softmax each, one thread per row, with the lazy running maximum, and warp 10
// finds the work items, one ahead.  What is different here:
//   - Masks.  Row r sees the keys below its own limit (causal: token + 1 + nk - nq), compared per
//     thread, only in the key blocks that a warp's rows do not see whole.  A tile runs only as
//     many key blocks as its last token sees.  A row that sees nothing keeps m = -inf, l = 0 and
//     writes zeros.
//   - Keys past the sequence's end are other sequences' or unwritten memory.  Their scores are
//     replaced, not added to; their V rows, which a zero probability would not silence if they
//     hold NaN, are zeroed in shared memory before the last block's MMA.
//   - V rows that a causal row must not see but its tile needs can hold NaN as well.  Rows that come out
//     not finite are noted down; when its CTA is through with its items, or with room for notes, each
//     softmax warp looks at the (under 256) keys behind its rows' limits that the tile took in, and
//     where one of them is to blame works the rows out again, sixteen at a time (repair_rows).  One NaN
//     near the end of 8192 tokens costs 2.1 ms so; one row at a time, within the item while the other
//     roles waited, it cost 123 ms and from some 130 thousand tokens on more than a wait may take.
//   - Work order.  Items come longest first over all sequences (index within the sequence,
//     descending) from a counter, so the last ones are short.  For up to 64 sequences warp 10 finds
//     an item itself: with n_s items in sequence s, C(v) = sum max(0, n_s - v) items have an index
//     >= v, and a search over v takes a few warp sums.  For more, a one-CTA kernel lists the
//     items first.
//   - Items overlap.  The next item's Q and K load when the last scores of one are complete, its scores
//     run while the softmax warps write out, whole-token rows by TMA store.
//   - Key splits.  Where items x key heads leave SMs idle, the keys are cut into equal runs of
//     blocks whose unnormalised outputs, maxima and sums go to the workspace, and
//     text_attention_join_kernel adds them up in split order.
//
// Bound, as the joint attention, by the softmax and MMAs of a key block taking turns: 1.57 us per
// 256 rows x 128 keys x 128 dims.  Causal, 32 query heads on 8 of 128: one sequence of 8192 tokens 376 us in
// a burst of twenty (1460 TFLOP/s of visible pairs), 394 call after call for a second, at the clocks that
// power leaves (1395 TFLOP/s); eleven of 17 to 1500 tokens 114 and 115 us (936 TFLOP/s): there an
// item's ends (first block without its neighbour's overlap 1 us, last PV 0.8 us, output 1.5 us) stand
// against five blocks.  One sequence of 512: 13.6 us, 64 items of up to four blocks on 64 SMs.
//
// Probabilities are rounded to bf16 for the product with V, here and in the few-row kernel: an MMA takes A
// and B of one 16-bit type and V is bf16, and a second product with what the rounding leaves would make three
// products per key block of two.  It costs 0.0020 to 0.0023 relative error against 64 bits, where fp32 probabilities
// and the output's own rounding give 0.0015 to 0.0017.  Sums and statistics are of the unrounded ones, in fp32.
//
// Measured and left: an issuing thread per tile (8192 tokens 378 -> 504 us: the tiles' MMAs interleave and
// both wait longer); for heads of 64, P beside S in Tensor Memory and the next QK ahead of the PV (8192
// tokens of 32 heads on 8 304 -> 326); one tile per item for 512 tokens (13.3 -> 13.1).
#include <math.h>

#include <atomic>

#include "runtime.h"
#include "tc_attention.cuh"
#include "text_join.cuh"

namespace dit {

namespace {

constexpr int kThreads = 352;
constexpr int kKeys = 128;                     // keys per block
constexpr uint32_t kHalfBytes = 128 * 64 * 2;  // 64 dims of a 128-row tile
constexpr uint32_t kTmemCols = 512;
constexpr float kPsumLimit = 4096.0f;  // row sum of P that sends a key block down the slow path
constexpr int kInlineSeqs = 64;        // up to here one warp finds its item itself
constexpr int kLevels = 1024;          // tile-index levels of the listing kernel

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

struct Plan {
  int group, tq, tp;   // heads per key head, tokens per tile and per pair
  int tiles, levels;   // bounds of the pairs over all sequences, and of one sequence's
  int splits;
  bool list;
};

Plan make_plan(const TextAttnArgs& a) {
  Plan p;
  p.group = a.heads_q / a.heads_k;
  p.tq = 128 / p.group;
  p.tp = 2 * p.tq;
  p.levels = (a.max_q + p.tp - 1) / p.tp;
  const long long packed = (long long)a.rows_q / p.tp + a.seqs, padded = (long long)a.seqs * p.levels;
  p.tiles = (int)(packed < padded ? packed : padded);
  p.list = a.seqs > kInlineSeqs;
  // Splits only fill SMs that would stay idle, and leave each part four key blocks: a part costs
  // a fixed ~3 us (launch, first loads, join) against ~1.3 us per block.  300 tokens of 3 heads over
  // 3366 keys of one: 49.8 us whole, 20.6 in six parts.
  const long long items = (long long)p.tiles * a.heads_k;
  const int blocks = (a.max_k + kKeys - 1) / kKeys;
  p.splits = 1;
  if (items > 0 && items < kSMs) {
    int s = (int)(kSMs / items);
    if (s > blocks / 4) s = blocks / 4;
    if (s > 32) s = 32;
    p.splits = s < 1 ? 1 : s;
  }
  return p;
}

// Workspace: the tile list, then per tile its first output row and token count, then the splits'
// (max, sum) and unnormalised outputs, 256 rows per (tile, key head, split).
struct Parts {
  size_t list, desc, ml, o, total;
};
inline size_t up256(size_t x) { return (x + 255) & ~size_t(255); }
Parts parts_layout(const Plan& p, int heads_k, int head_dim) {
  Parts l;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t r = at;
    at = up256(at + bytes);
    return r;
  };
  const size_t items = p.splits > 1 ? (size_t)p.tiles * heads_k * p.splits : 0;
  l.list = take(p.list ? (size_t)p.tiles * 8 : 0);
  l.desc = take(p.splits > 1 ? (size_t)p.tiles * 8 : 0);
  l.ml = take(items * 256 * 8);
  l.o = take(items * 256 * (size_t)head_dim * 4);
  l.total = at;
  return l;
}

struct alignas(64) TextAttnParams {
  CUtensorMap q_map, k_map, v_map, o_map;  // o_map: one softmax warp's rows, where they are whole tokens
  TextAttnArgs a;
  int group, tq, levels, tiles, splits, items;
  float scale_log2;
  const int2* list;
  int2* desc;
  float2* ml;
  float* o;
};

enum : uint32_t {
  kSiteQ = 0x511, kSiteFree, kSiteReady, kSitePFull, kSiteSFull, kSiteODone, kSiteFixed, kSiteFix, kSiteItem, kSiteItemFree
};

__device__ __forceinline__ void tma_store_4d(const CUtensorMap* m, const void* src, int x, int y, int z, int w) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void mbar_inval(uint64_t* bar) {
  asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// Every store of this thread has been read out of shared memory.
__device__ __forceinline__ void tma_store_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

// Records (work item, rows) of rows that came out not finite: how many a softmax warp can hold, and with
// how many of them its CTA takes no further items for now (two may be on their way when warp 10 looks).
constexpr int kOddMost = 24, kOddFull = kOddMost - 3;
constexpr int kBars = 17;  // mbarriers
enum : int { kRepair = 1, kAgain = 2 };  // after a pass over work items: rows to repair; more items

template <int D>
struct Smem {
  static constexpr uint32_t kTile = (D / 64) * kHalfBytes;  // a 128-row tile of Q, K or V
  static constexpr uint32_t kQ = 0, kK = 2 * kTile, kV = 4 * kTile;
  static constexpr uint32_t kOut = 6 * kTile;            // 32 rows x 64 dims of output per softmax warp
  static constexpr uint32_t kBar = kOut + 8 * 4096;
  static constexpr uint32_t kOdd = kBar + 288;           // kOddMost records of each softmax warp
  static constexpr size_t kBytes = 1024 + kOdd + 8 * kOddMost * sizeof(uint2);
};

// One work item of a CTA, as warp 10 found it.
struct Item {
  int q0, nq, k0, nk, tok0;  // the sequence's rows, and the pair's first token
  int n0, n1, b0;            // key blocks of each tile, and the first of them (of this split)
  int hk, split, rank;       // key head, key split, place of the pair in the work order
  int stop;                  // no more items
};

// The t-th pair of tiles, longest first (whole warp; span and tile index broadcast).
__device__ __forceinline__ bool find_tile(const TextAttnArgs& a, int tp, int levels, int tiles, int t, int lane,
                                          bool report, Span& sp, int& index) {
  Span s[2];
  int n[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int id = lane + 32 * i;
    s[i] = Span{0, 0, 0, 0, true};
    if (id < a.seqs) s[i] = load_span(a, id);
    n[i] = (s[i].nq + tp - 1) / tp;
    if (!s[i].ok && report) report_bad_entry(a.status, kSiteTextLengths);
  }
  auto count = [&](int v) { return __reduce_add_sync(0xffffffffu, max(0, n[0] - v) + max(0, n[1] - v)); };
  const int all = count(0);
  // more tiles than the buffers' rows allow: query rows of several sequences overlap
  if (all > tiles && report && lane == 0) report_bad_entry(a.status, kSiteTextLengths);
  if (all <= t) return false;
  int lo = 0, hi = levels;  // count(lo) > t >= count(hi)
  while (hi - lo > 1) {
    const int v = (lo + hi) >> 1;
    if (count(v) > t) lo = v;
    else hi = v;
  }
  index = lo;
  int r = t - count(lo + 1);  // the r-th sequence with more than `lo` tiles
  const uint32_t b0 = __ballot_sync(0xffffffffu, n[0] > lo), b1 = __ballot_sync(0xffffffffu, n[1] > lo);
  const int second = r >= __popc(b0);
  const uint32_t b = second ? b1 : b0;
  if (second) r -= __popc(b0);
  const bool me = ((b >> lane) & 1u) && __popc(b & ((1u << lane) - 1u)) == r;
  const int src = __ffs(__ballot_sync(0xffffffffu, me)) - 1;
  sp.q0 = __shfl_sync(0xffffffffu, second ? s[1].q0 : s[0].q0, src);
  sp.nq = __shfl_sync(0xffffffffu, second ? s[1].nq : s[0].nq, src);
  sp.k0 = __shfl_sync(0xffffffffu, second ? s[1].k0 : s[0].k0, src);
  sp.nk = __shfl_sync(0xffffffffu, second ? s[1].nk : s[0].nk, src);
  return true;
}

// Lists the pairs of tiles (sequence, index), longest first up to kLevels steps: a histogram of
// the tiles' levels, its running sum from the top, then every tile to the next place of its
// level.  Unused places get sequence -1.
__global__ void __launch_bounds__(1024) text_attention_list_kernel(const TextAttnArgs a, int tp, int levels, int tiles,
                                                                   int2* list) {
  __shared__ int at[kLevels];
  __shared__ int total, warp_sum[32];
  grid_dependency_wait();
  allow_dependents();
  const int t = threadIdx.x;
  at[t] = 0;
  __syncthreads();
  const int shift = levels <= kLevels ? 0 : 32 - __clz((levels - 1) / kLevels);
  for (int s = t; s < a.seqs; s += 1024) {
    const Span sp = load_span(a, s);
    if (!sp.ok) report_bad_entry(a.status, kSiteTextLengths);
    const int n = (sp.nq + tp - 1) / tp;
    for (int i = 0; i < n; ++i) atomicAdd(&at[i >> shift], 1);
  }
  __syncthreads();
  // thread t: the tiles of the levels above level kLevels - 1 - t
  const int mine = at[kLevels - 1 - t];
  int sum = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, sum, o);
    if ((t & 31) >= o) sum += v;
  }
  if ((t & 31) == 31) warp_sum[t >> 5] = sum;
  __syncthreads();
  for (int w = 0; w < (t >> 5); ++w) sum += warp_sum[w];
  at[kLevels - 1 - t] = sum - mine;
  if (t == kLevels - 1) total = sum;
  __syncthreads();
  if (t == 0 && total > tiles) report_bad_entry(a.status, kSiteTextLengths);
  for (int s = t; s < a.seqs; s += 1024) {
    const int n = (load_span(a, s).nq + tp - 1) / tp;
    for (int i = 0; i < n; ++i) {
      const int p = atomicAdd(&at[i >> shift], 1);
      if (p < tiles) list[p] = make_int2(s, i);
    }
  }
  for (int p = total + t; p < tiles; p += 1024) list[p] = make_int2(-1, 0);
}

// ---- tensor-core work ------------------------------------------------------------------

template <int D>
struct Descs {
  uint64_t q[2][D / 16], k[2][D / 16], v[2][8];
};

template <int D>
__device__ __forceinline__ void make_descs(uint8_t* smem, Descs<D>& d) {
  using L = Smem<D>;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      const uint32_t off = (kk >> 2) * kHalfBytes + (kk & 3) * 32;
      d.q[t][kk] = make_sdesc_sw128(smem_u32(smem + L::kQ + t * L::kTile) + off, 16, 1024);
      d.k[t][kk] = make_sdesc_sw128(smem_u32(smem + L::kK + t * L::kTile) + off, 16, 1024);
    }
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)
      d.v[t][kk] = make_sdesc_sw128(smem_u32(smem + L::kV + t * L::kTile) + kk * 2048, kHalfBytes, 1024);
  }
}

template <int ST>
__device__ __forceinline__ void issue_qk(const Descs<128>& d, uint32_t tmem, int t, uint32_t idesc, uint64_t* bar) {
  umma8_ss(tmem + (uint32_t)(t * 256), d.q[t], d.k[ST], idesc);
  umma_commit(bar);
}
template <int ST>
__device__ __forceinline__ void issue_qk(const Descs<64>& d, uint32_t tmem, int t, uint32_t idesc, uint64_t* bar) {
  umma4_ss(tmem + (uint32_t)(t * 256), d.q[t], d.k[ST], idesc);
  umma_commit(bar);
}

struct Bars {
  uint64_t *q_full, *ready, *slot_free, *s_full, *p_full, *o_done, *fixed, *drain, *item_full, *item_free;
};

// How often a role has waited on each of two barriers: the parity of its next wait.
struct Turns {
  uint32_t n[2] = {0, 0};
  __device__ __forceinline__ uint32_t next(int i) { return (i ? n[1]++ : n[0]++) & 1u; }
};

// Key block j of the issuer (ring stage ST = j & 1), n[t] blocks for tile t:
//   O0 += P0 V_j, S0 = Q0 K_{j+1}^T, O1 += P1 V_j, S1 = Q1 K_{j+1}^T.
template <int D, int ST>
__device__ __forceinline__ bool mma_block(const Descs<D>& d, uint32_t tmem, int j, int n0, int n1, bool fix,
                                          uint32_t idesc_qk, uint32_t idesc_pv, const Bars& bar, const WaitCtx& wc,
                                          Turns& t_ready, Turns& t_p, uint32_t& t_fixed) {
  if (!mbar_wait(&bar.ready[ST], t_ready.next(ST), wc, kSiteReady)) return false;
  if (fix && j + 1 == max(n0, n1) && !mbar_wait(bar.fixed, t_fixed++ & 1u, wc, kSiteFixed)) return false;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int n = t ? n1 : n0;
    if (j < n) {
      if (!mbar_wait(&bar.p_full[t], t_p.next(t), wc, kSitePFull)) return false;
      tc_fence_after();
      umma8_ts(tmem + (uint32_t)(t * 256 + 128), tmem + (uint32_t)(t * 256), d.v[ST], idesc_pv, j > 0 ? 1u : 0u);
      if (j + 1 < n) issue_qk<ST ^ 1>(d, tmem, t, idesc_qk, &bar.s_full[t]);
      else umma_commit(&bar.o_done[t]);
    }
  }
  return true;
}

// ---- rows that met a value they do not see ------------------------------------------------

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// D += A B, 16 x 8 x 16, bf16 in, fp32 out.
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A head of V: whether a value of it is infinite or NaN, and whether all are NaN.
template <int D>
__device__ __forceinline__ void scan_values(const bf16* v, bool& bad, bool& all_nan) {
  bad = false;
  all_nan = true;
#pragma unroll 4
  for (int i = 0; i < D / 8; ++i) {
    const uint4 u = *reinterpret_cast<const uint4*>(v + i * 8);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t lo = w[e] & 0x7fffu, hi = (w[e] >> 16) & 0x7fffu;
      bad |= lo >= 0x7f80u || hi >= 0x7f80u;
      all_nan &= lo > 0x7f80u && hi > 0x7f80u;
    }
  }
}

// Of the rows (one per lane, those in `rows`) whose sums came out not finite, those that may owe it to a
// key they do not see: lane's row sees the keys below `seen`, its tile took in those of [first, end).  Rows
// whose last visible key is NaN throughout are so by right.
template <int D>
__device__ __noinline__ uint32_t spoiled_rows(const bf16* vp, long long ldv, uint32_t rows, int seen, int first, int end,
                                              int lane) {
  const bool mine = (rows >> lane) & 1u;
  const int lo = __reduce_min_sync(0xffffffffu, mine ? max(seen, first) : end);
  int last = -1;  // the last key with a bad value
  for (int top = end; top > lo && last < 0; top -= 32) {
    const int j = top - 1 - lane;
    bool bad = false, all_nan;
    if (j >= lo) scan_values<D>(vp + j * ldv, bad, all_nan);
    const uint32_t b = __ballot_sync(0xffffffffu, bad);
    if (b) last = top - __ffs(b);
  }
  bool redo = mine && seen <= last;
  if (redo && seen > first) {
    bool bad, all_nan;
    scan_values<D>(vp + (seen - 1) * ldv, bad, all_nan);
    redo = !all_nan;
  }
  return __ballot_sync(0xffffffffu, redo);
}

// Up to 16 rows of a key head by one warp, apart from the tiles.  Lane r < 16 brings row r: its query, the
// keys it sees (0: no row) and where it goes: the normalised output row, or a part's unnormalised one and
// its (max, sum).  16 keys a step through mma.sync, V by way of `stage` (16 x D bf16 of this warp's shared
// memory); in the last steps, where some rows see fewer keys than others, P V is done by plain FMAs, in which
// a key that a row does not see is left out and not multiplied by zero.  m in log2 units.
// Bound by the latency of a step's loads.
template <int D, bool kParts>
__device__ __noinline__ void attend_rows(const TextAttnArgs& a, const bf16* qp, const bf16* kp, const bf16* vp, int limit,
                                         float c, int lane, void* dst, float2* ml, uint8_t* stage) {
  const int r0 = lane >> 2, c0 = (lane & 3) * 2;  // fragments: rows r0 and r0 + 8, columns c0 + {0, 1}
  const int most = __reduce_max_sync(0xffffffffu, limit);
  const int least = __reduce_min_sync(0xffffffffu, limit > 0 ? limit : most);
  uint32_t q[D / 16][4];
  int lim[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    lim[i] = __shfl_sync(0xffffffffu, limit, r0 + 8 * i);
    const bf16* src = reinterpret_cast<const bf16*>(
                          __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(qp), r0 + 8 * i)) + c0;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      q[k][i] = lim[i] > 0 ? *reinterpret_cast<const uint32_t*>(src + k * 16) : 0u;
      q[k][i + 2] = lim[i] > 0 ? *reinterpret_cast<const uint32_t*>(src + k * 16 + 8) : 0u;
    }
  }
  float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int d = 0; d < D / 8; ++d) o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.f;
  for (int j = 0; j < most; j += 16) {
    // V rows in 16-byte pieces (swizzled), on their way while the scores are worked out
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      const int piece = i * 32 + lane, row = piece / (D / 8), col = piece % (D / 8);
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(stage + row * D * 2 + ((col ^ (row & 7)) << 4))),
                   "l"(vp + min(j + row, most - 1) * a.ldv + col * 8)
                   : "memory");
    }
    float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    uint32_t kb[2][D / 8];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const bf16* key = kp + min(j + n * 8 + r0, most - 1) * a.ldk + c0;
#pragma unroll
      for (int k = 0; k < D / 8; ++k) kb[n][k] = *reinterpret_cast<const uint32_t*>(key + k * 8);
    }
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int k = 0; k < D / 16; ++k) mma_bf16(s[n], q[k], kb[n][2 * k], kb[n][2 * k + 1]);
    float p[2][4], alpha[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float mx = -INFINITY;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        p[i][e] = j + (e >> 1) * 8 + c0 + (e & 1) < lim[i] ? s[e >> 1][2 * i + (e & 1)] * c : -INFINITY;
        mx = fmaxf(mx, p[i][e]);
      }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float mn = fmaxf(m[i], mx), ref = mn == -INFINITY ? 0.f : mn;
      alpha[i] = m[i] == mn ? 1.f : ex2_approx(m[i] - ref);
      m[i] = mn;
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) sum += p[i][e] = ex2_approx(p[i][e] - ref);
      l[i] = l[i] * alpha[i] + sum;
    }
    if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
      for (int d = 0; d < D / 8; ++d) o[d][0] *= alpha[0], o[d][1] *= alpha[0], o[d][2] *= alpha[1], o[d][3] *= alpha[1];
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
    if (j + 16 <= least) {
      // rounded to bf16 as in the tiles
      const uint32_t pf[4] = {pack_bf16x2(p[0][0], p[0][1]), pack_bf16x2(p[1][0], p[1][1]), pack_bf16x2(p[0][2], p[0][3]),
                              pack_bf16x2(p[1][2], p[1][3])};
      const int vk = lane & 15, vc = lane >> 4;
#pragma unroll
      for (int d = 0; d < D / 16; ++d) {
        uint32_t b[4];
        ldmatrix4_trans(b, smem_u32(stage + vk * D * 2 + (((d * 2 + vc) ^ (vk & 7)) << 4)));
        mma_bf16(o[2 * d], pf, b[0], b[1]);
        mma_bf16(o[2 * d + 1], pf, b[2], b[3]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll 1
        for (int t = 0; t < 4; ++t) {  // a key of the step, whose probabilities lane t of the four holds
          const int row = (e >> 1) * 8 + t * 2 + (e & 1);
          const float p0 = __shfl_sync(0xffffffffu, p[0][e], (lane & 28) + t);
          const float p1 = __shfl_sync(0xffffffffu, p[1][e], (lane & 28) + t);
          const bool see0 = j + row < lim[0], see1 = j + row < lim[1];
#pragma unroll
          for (int d = 0; d < D / 8; ++d) {
            const uint8_t* v = stage + row * D * 2 + ((d ^ (row & 7)) << 4) + c0 * 2;
            const float2 x = unpack_bf16x2(*reinterpret_cast<const uint32_t*>(v));
            if (see0) o[d][0] = fmaf(p0, x.x, o[d][0]), o[d][1] = fmaf(p0, x.y, o[d][1]);
            if (see1) o[d][2] = fmaf(p1, x.x, o[d][2]), o[d][3] = fmaf(p1, x.y, o[d][3]);
          }
        }
    }
    __syncwarp();  // V has been read
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    const unsigned long long to = __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(dst), r0 + 8 * i);
    const unsigned long long at = __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(ml), r0 + 8 * i);
    if (lim[i] <= 0) continue;
    const float inv = l[i] == 0.f ? 0.f : 1.0f / l[i];
#pragma unroll
    for (int d = 0; d < D / 8; ++d) {
      if (kParts)
        *reinterpret_cast<float2*>(reinterpret_cast<float*>(to) + d * 8 + c0) = make_float2(o[d][2 * i], o[d][2 * i + 1]);
      else
        *reinterpret_cast<uint32_t*>(reinterpret_cast<bf16*>(to) + d * 8 + c0) =
            l[i] == 0.f ? 0u : pack_bf16x2(o[d][2 * i] * inv, o[d][2 * i + 1] * inv);
    }
    if (kParts && (lane & 3) == 0) *reinterpret_cast<float2*>(at) = make_float2(m[i], l[i]);
  }
}

// Work item `id`: its place, and where its sequence has tiles, its rows and key blocks (whole warp).
template <bool kSplit>
__device__ __forceinline__ bool locate_item(const TextAttnParams& P, int id, int lane, bool report, Item& it) {
  const TextAttnArgs& a = P.a;
  const int TP = 2 * P.tq;
  int index = 0, rank = id / a.heads_k, split = 0;
  const int hk = id - rank * a.heads_k;
  if (kSplit) {
    split = rank % P.splits;
    rank /= P.splits;
  }
  Span sp{0, -1, 0, 0, true};
  bool found;
  if (P.list) {
    const int2 e = P.list[rank];
    found = e.x >= 0;
    if (found) sp = load_span(a, e.x);
    index = e.y;
  } else {
    found = find_tile(a, TP, P.levels, P.tiles, rank, lane, report, sp, index);
  }
  it = Item{sp.q0, sp.nq, sp.k0, sp.nk, index * TP, 0, 0, 0, hk, split, rank, 0};
  if (found) {
    // key blocks of each tile, and this split's run [b0, b0 + n) of them
    const int shift = it.nk - it.nq;
    auto blocks = [&](int first) {
      if (first >= it.nq) return 0;
      const int last = min(first + P.tq, it.nq) - 1;
      const int end = a.causal ? min(it.nk, last + shift + 1) : it.nk;
      return end > 0 ? (end + kKeys - 1) / kKeys : 0;
    };
    it.n0 = blocks(it.tok0);
    it.n1 = blocks(it.tok0 + P.tq);
    if (kSplit) {
      const int nb = max(it.n0, it.n1);
      it.b0 = (int)((long long)nb * split / P.splits);
      const int b1 = (int)((long long)nb * (split + 1) / P.splits);
      it.n0 = max(0, min(it.n0, b1) - it.b0);
      it.n1 = max(0, min(it.n1, b1) - it.b0);
    }
  }
  return found;
}

// The rows of a softmax warp (bits of `rows`) that came out not finite in work item `id`, worked out again
// where a value behind their keys may be why.
template <int D, bool kSplit>
__device__ __forceinline__ void repair_rows(const TextAttnParams& P, int id, uint32_t rows, int warp, int lane,
                                            uint8_t* stage) {
  const TextAttnArgs& a = P.a;
  Item it;
  locate_item<kSplit>(P, id, lane, false, it);
  const int G = P.group, tile = (warp - 2) >> 2, row = (warp & 3) * 32 + lane, token = row / G;
  const int begin = it.b0 * kKeys, end = min(it.nk, begin + (tile ? it.n1 : it.n0) * kKeys);
  const int seen = a.causal ? min(it.nk, it.tok0 + tile * P.tq + token + it.nk - it.nq + 1) : it.nk;
  rows &= __ballot_sync(0xffffffffu, seen < end);
  if (!rows) return;
  const bf16* vp = a.v + (long long)it.k0 * a.ldv + it.hk * D;
  rows = spoiled_rows<D>(vp, a.ldv, rows, seen, begin, end, lane);
  const long long part = (((long long)it.rank * a.heads_k + it.hk) * P.splits + it.split) * 256;
  while (rows) {
    const uint32_t src = lane < 16 ? __fns(rows, 0, lane + 1) : 32u;  // lane r < 16 takes the r-th of them
    const bool have = src < 32u;
    const int r = (warp & 3) * 32 + (have ? (int)src : 0), r_token = r / G, r_col = (it.hk * G + r - r_token * G) * D;
    const int r_seen = __shfl_sync(0xffffffffu, seen, src & 31u);
    const long long q_row = it.q0 + it.tok0 + tile * P.tq + r_token, prow = part + tile * P.tq * G + r;
    void* dst = kSplit ? (void*)(P.o + prow * D) : (void*)(a.out + q_row * a.ldo + r_col);
    attend_rows<D, kSplit>(a, a.q + q_row * a.ldq + r_col, a.k + (long long)(it.k0 + begin) * a.ldk + it.hk * D,
                           vp + begin * a.ldv, have ? r_seen - begin : 0, P.scale_log2, lane, dst, P.ml + prow, stage);
    for (int i = 0; i < 16 && rows; ++i) rows &= rows - 1;
  }
}

// The kernel's shared memory behind the tiles.
template <int D>
struct Shared {
  uint8_t* smem;
  uint64_t* bars;
  Bars bar;
  uint32_t* tmem_slot;
  volatile int* abort_flag;
  Item* items;           // two: the current one and the next
  int* after;            // what follows the pass: kRepair, kAgain
  volatile int* odd_n;   // each softmax warp's records, and how many there are
  uint2* odd;
  static_assert(Smem<D>::kBar + (kBars + 1) * 8 + 2 * sizeof(Item) + 9 * sizeof(int) <= Smem<D>::kOdd, "room for all of it");
  static_assert(Smem<D>::kBytes <= 227 * 1024, "what a CTA may have");
  __device__ __forceinline__ explicit Shared(uint8_t* base)
      : smem(base),
        bars(reinterpret_cast<uint64_t*>(base + Smem<D>::kBar)),
        bar{bars + 0, bars + 1, bars + 3, bars + 5, bars + 7, bars + 9, bars + 11, bars + 12, bars + 13, bars + 15},
        tmem_slot(reinterpret_cast<uint32_t*>(bars + kBars)),
        abort_flag(reinterpret_cast<volatile int*>(tmem_slot + 1)),
        items(reinterpret_cast<Item*>(bars + kBars + 1)),
        after(reinterpret_cast<int*>(items + 2)),
        odd_n(after + 1),
        odd(reinterpret_cast<uint2*>(base + Smem<D>::kOdd)) {}
};

template <int D>
__device__ __forceinline__ void init_pass(const Shared<D>& sh) {
  const Bars& bar = sh.bar;
  mbar_init(bar.q_full, 1);
  for (int i = 0; i < 2; ++i) {
    mbar_init(&bar.ready[i], 1);
    mbar_init(&bar.slot_free[i], 1);
    mbar_init(&bar.s_full[i], 1);
    mbar_init(&bar.p_full[i], 4);
    mbar_init(&bar.o_done[i], 1);
    mbar_init(&bar.item_full[i], 1);
    mbar_init(&bar.item_free[i], 10);  // the loader, the issuer and eight softmax warps
  }
  mbar_init(bar.fixed, 1);
  mbar_init(bar.drain, 1);
  *sh.after = 0;
  for (int i = 0; i < 8; ++i) sh.odd_n[i] = 0;
  fence_mbar_init();
}

// A CTA's work items, until there are none left or a softmax warp's records are full: each warp's role.
template <int D, bool kSplit>
__device__ __forceinline__ void run_items(const TextAttnParams& P, const Shared<D>& sh, uint32_t tmem, bool first_pass) {
  using L = Smem<D>;
  uint8_t* const smem = sh.smem;
  const Bars& bar = sh.bar;
  Item* const items = sh.items;
  const TextAttnArgs& a = P.a;
  int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("" : "+r"(warp), "+r"(lane));  // not carried from pass to pass either (see the kernel)
  const int G = P.group, TQ = P.tq;
  const WaitCtx wc{a.status, sh.abort_flag, kWaitLimitNs};
  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    // Ring slot j & 1 carries V_j and K_{j+1}; slot j >= 1 is loaded once the scores of block
    // j - 1 of the longer tile are complete, which ends every read of V_{j-2} and K_{j-1}.  The next
    // item's Q and K_0 follow when the last scores are complete (every QK is done), its V_0 and K_1
    // when the last O of both tiles is: while the softmax warps finish one item, the next one's loads
    // and scores are under way.
    Turns t_free, t_o, t_ready;
    uint32_t live = 0;             // items with key blocks so far
    int pn = 0, pn0 = 0, pn1 = 0;  // the last such item's blocks
    bool ok = true;
    for (uint32_t k = 0; ok; ++k) {
      ok = mbar_wait_sleep(&bar.item_full[k & 1], (k >> 1) & 1u, wc, kSiteItem);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const Item it = items[k & 1];
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.item_free[k & 1]);
      if (it.stop) break;
      const int nmax = max(it.n0, it.n1);
      if (nmax == 0) continue;
      const int krow = it.k0 + it.b0 * kKeys;
      if (lane == 0) {
        int issued = 0;
        if (live > 0) ok = mbar_wait_sleep(&bar.slot_free[pn & 1], t_free.next(pn & 1), wc, kSiteFree);
        if (ok) {
          const uint32_t qbytes = (uint32_t)(G * TQ) * 128u * (D / 64);
          mbar_arrive_expect_tx(bar.q_full, (uint32_t)((it.n0 > 0) + (it.n1 > 0)) * qbytes + L::kTile);
          for (int t = 0; t < 2; ++t)
            if ((t ? it.n1 : it.n0) > 0)
              for (int h = 0; h < D / 64; ++h)
                tma_load_4d(smem + L::kQ + t * L::kTile + h * kHalfBytes, &P.q_map, bar.q_full, h * 64, 0, it.hk,
                            it.q0 + it.tok0 + t * TQ);
          for (int h = 0; h < D / 64; ++h)
            tma_load_3d(smem + L::kK + h * kHalfBytes, &P.k_map, bar.q_full, h * 64, it.hk, krow);
          ++live;
          if (pn0 > 0) ok = mbar_wait_sleep(&bar.o_done[0], t_o.next(0), wc, kSiteODone);
          if (ok && pn1 > 0) ok = mbar_wait_sleep(&bar.o_done[1], t_o.next(1), wc, kSiteODone);
        }
        for (int j = 0; j < nmax && ok; ++j) {
          const int b = j & 1;
          if (j >= 1 && !mbar_wait_sleep(&bar.slot_free[b], t_free.next(b), wc, kSiteFree)) {
            ok = false;
            break;
          }
          const bool more = j + 1 < nmax;
          mbar_arrive_expect_tx(&bar.ready[b], more ? 2 * L::kTile : L::kTile);
          for (int h = 0; h < D / 64; ++h)
            tma_load_3d(smem + L::kV + b * L::kTile + h * kHalfBytes, &P.v_map, &bar.ready[b], h * 64, it.hk,
                        krow + j * kKeys);
          if (more)
            for (int h = 0; h < D / 64; ++h)
              tma_load_3d(smem + L::kK + (b ^ 1) * L::kTile + h * kHalfBytes, &P.k_map, &bar.ready[b], h * 64, it.hk,
                          krow + (j + 1) * kKeys);
          issued = j + 1;
        }
        if (!ok) {
          // Unwinding: let copies in flight land (bounded) before the block exits.
          const uint64_t t0 = global_timer_ns();
          while (live > 0 && !mbar_try(bar.q_full, (live - 1) & 1u) && global_timer_ns() - t0 < 100000000ull) {
          }
          for (int j = (issued > 2 ? issued - 2 : 0); j < issued; ++j)
            while (!mbar_try(&bar.ready[j & 1], (t_ready.n[j & 1] + (uint32_t)(j >> 1)) & 1u) &&
                   global_timer_ns() - t0 < 200000000ull) {
            }
        }
      }
      __syncwarp();
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      pn = nmax;
      pn0 = it.n0;
      pn1 = it.n1;
      t_ready.n[0] += (uint32_t)(nmax + 1) >> 1;  // uses of each ring slot so far
      t_ready.n[1] += (uint32_t)nmax >> 1;
      if ((it.b0 + nmax) * kKeys > it.nk) {
        // rows of the last block's V past the sequence's keys must read as zeros
        const int j = nmax - 1, b = j & 1;
        ok = mbar_wait_sleep(&bar.ready[b], (t_ready.n[b] - 1u) & 1u, wc, kSiteFix);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const int valid = it.nk - (it.b0 + j) * kKeys;  // 1 .. 127: rows are 128 contiguous bytes each
        for (int h = 0; h < D / 64; ++h) {
          uint4* v = reinterpret_cast<uint4*>(smem + L::kV + b * L::kTile + h * kHalfBytes);
          for (int i = valid * 8 + lane; i < kKeys * 8; i += 32) v[i] = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar.fixed);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // An item's QK may overwrite S while the softmax warps still write out the one before: P over
    // it has been read by MMAs issued earlier.  Its first PV waits for its first P, which those
    // warps store after they have read O.
    if (lane == 0) {
      const uint32_t idesc_qk = make_idesc_bf16(128, kKeys, false);
      const uint32_t idesc_pv = make_idesc_bf16(128, D, true);
      Descs<D> d;
      make_descs<D>(smem, d);
      Turns t_ready, t_p;
      uint32_t t_fixed = 0, live = 0;
      bool ok = true;
      for (uint32_t k = 0; ok; ++k) {
        ok = mbar_wait(&bar.item_full[k & 1], (k >> 1) & 1u, wc, kSiteItem);
        if (!ok) break;
        const Item& it = items[k & 1];
        const int n0 = it.n0, n1 = it.n1, nmax = max(n0, n1);
        const bool stop = it.stop, fix = (it.b0 + nmax) * kKeys > it.nk;
        mbar_arrive(&bar.item_free[k & 1]);
        if (stop) break;
        if (nmax == 0) continue;
        ok = mbar_wait(bar.q_full, live++ & 1u, wc, kSiteQ);
        if (ok) {
          tc_fence_after();
          if (n0 > 0) issue_qk<0>(d, tmem, 0, idesc_qk, &bar.s_full[0]);
          if (n1 > 0) issue_qk<0>(d, tmem, 1, idesc_qk, &bar.s_full[1]);
        }
        for (int j = 0; j < nmax && ok; j += 2) {
          ok = mma_block<D, 0>(d, tmem, j, n0, n1, fix, idesc_qk, idesc_pv, bar, wc, t_ready, t_p, t_fixed);
          if (ok && j + 1 < nmax)
            ok = mma_block<D, 1>(d, tmem, j + 1, n0, n1, fix, idesc_qk, idesc_pv, bar, wc, t_ready, t_p, t_fixed);
        }
      }
      umma_commit(bar.drain);
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try(bar.drain, 0) && global_timer_ns() - t0 < 1000000000ull) {
      }
    }
  } else if (warp == 10) {
    // ------------------------------------------------------------ work items
    // One item ahead of the others: the counter's and the lengths' latency is nobody's wait.
    uint32_t out = 0;  // items handed on
    bool ok = true;
    for (int k = 0; ok; ++k) {
      // the first item by place, the others as they come, longest first
      int id = (int)blockIdx.x;
      bool full = false;  // of records: the CTA repairs rows before it goes on
      if (!first_pass || k > 0) {
        full = __any_sync(0xffffffffu, lane < 8 && sh.odd_n[lane] >= kOddFull);
        if (lane == 0 && !full) id = (int)(gridDim.x + atomicAdd(&a.status->next_item, 1u));
        id = __shfl_sync(0xffffffffu, id, 0);
      }
      const bool stop = full || (uint32_t)id >= (uint32_t)P.items;  // a counter that was not zero wraps to no item
      Item it{0, -1, 0, 0, 0, 0, 0, 0, 0, 0, 0, 1};
      if (!stop) {
        const bool found = locate_item<kSplit>(P, id, lane, first_pass && k == 0 && blockIdx.x == 0, it);
        if (kSplit && it.hk == 0 && it.split == 0 && lane == 0)
          P.desc[it.rank] = found ? make_int2(it.q0 + it.tok0, min(2 * TQ, it.nq - it.tok0)) : make_int2(0, 0);
        if (!found) continue;
      }
      if (full && lane == 0) atomicOr(sh.after, kAgain);
      ok = mbar_wait_sleep(&bar.item_free[out & 1], ((out >> 1) & 1u) ^ 1u, wc, kSiteItemFree);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (lane == 0) {
        items[out & 1] = it;
        mbar_arrive(&bar.item_full[out & 1]);
      }
      __syncwarp();
      ++out;
      if (stop) break;
    }
  } else {
    // ------------------------------------------------------------ softmax / output
    const int tile = (warp - 2) >> 2;  // warps 2-5 -> tile 0, warps 6-9 -> tile 1
    const int qq = warp & 3;           // TMEM lane quarter of this warp
    const int row = qq * 32 + lane;
    const uint32_t tS = tmem + (uint32_t)(tile * 256) + ((uint32_t)(qq * 32) << 16);
    const uint32_t tO = tS + 128;
    const float c = P.scale_log2;
    const int token = row / G, g = row - token * G;
    uint8_t* staged = smem + L::kOut + (warp - 2) * 4096;
    uint32_t t_s = 0, t_o = 0;
    bool ok = true;
    for (uint32_t k = 0; ok; ++k) {
      ok = mbar_wait(&bar.item_full[k & 1], (k >> 1) & 1u, wc, kSiteItem);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      // The slot stays this warp's until the end of the item: its fields are read again after the key
      // loop, whose registers are full.
      const volatile Item& it = items[k & 1];
      if (it.stop) break;
      const int n = tile ? it.n1 : it.n0;
      const bool releaser = tile == (it.n1 >= it.n0 ? 1 : 0) && qq == 2 && lane == 0;
      const int qi = it.tok0 + tile * TQ + token;
      const bool active = token < TQ && qi < it.nq;
      // keys this row sees, counted from this split's first block (causal: token i sees keys
      // j <= i + nk - nq); rows that are not stored need no mask
      const int limit =
          (!active ? 0x3fffffff : (a.causal ? min(it.nk, qi + it.nk - it.nq + 1) : it.nk)) - it.b0 * kKeys;
      float m_run = active ? -INFINITY : 0.f, l_run = 0.f;
      for (int j = 0; j < n; ++j) {
        ok = mbar_wait(&bar.s_full[tile], t_s++ & 1u, wc, kSiteSFull);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (releaser) mbar_arrive(&bar.slot_free[(j + 1) & 1]);
        tc_fence_after();
        const int kv_valid = limit - j * kKeys;
        const bool whole = __all_sync(0xffffffffu, kv_valid >= kKeys);
        // Fast path against the running maximum; the slow path finds the block's maximum first.  A
        // row that has none yet (its first block) starts from the maximum over 32 keys: any
        // reference does as long as the row sum of P stays within bounds.
        uint32_t pk[64];
        float psum = 0.f, unused = -INFINITY, alpha = 1.0f;
        if (__any_sync(0xffffffffu, m_run == -INFINITY)) {
          uint32_t r[32];
          tmem_load32(tS, r);
          float mx = -INFINITY;
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (whole || i < kv_valid) mx = fmaxf(mx, __uint_as_float(r[i]));
          if (m_run == -INFINITY) m_run = mx * c;
        }
        const float m_ref = m_run == -INFINITY ? 0.f : m_run;
        if (whole) softmax_row<false, false>(tS, kv_valid, c, -m_ref, unused, psum, pk);
        else softmax_row<true, false>(tS, kv_valid, c, -m_ref, unused, psum, pk);
        const bool slow = active && (psum > kPsumLimit || m_run == -INFINITY);
        if (__any_sync(0xffffffffu, slow)) {
          float mx = -INFINITY;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t r[32];
            tmem_load32(tS + q * 32, r);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (whole || q * 32 + i < kv_valid) mx = fmaxf(mx, __uint_as_float(r[i]));
          }
          const float m_cand = fmaxf(m_run, mx * c);
          bool resc = false;
          if (active && m_cand > m_run) {
            alpha = ex2_approx(m_run - m_cand);
            m_run = m_cand;
            resc = true;
          }
          if (j > 0 && __any_sync(0xffffffffu, resc)) {
#pragma unroll 1
            for (int cc = 0; cc < D / 32; ++cc) {
              uint32_t r[32];
              tmem_load32(tO + cc * 32, r);
#pragma unroll
              for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
              tmem_store32(tO + cc * 32, r);
            }
          }
          const float mneg = m_run == -INFINITY ? 0.f : -m_run;
          if (whole) softmax_row<false, false>(tS, kv_valid, c, mneg, unused, psum, pk);
          else softmax_row<true, false>(tS, kv_valid, c, mneg, unused, psum, pk);
        }
        l_run = l_run * alpha + psum;
        tmem_store32(tS, *reinterpret_cast<const uint32_t(*)[32]>(&pk[0]));
        tmem_store32(tS + 32, *reinterpret_cast<const uint32_t(*)[32]>(&pk[32]));
        tmem_store_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.p_full[tile]);
      }
      if (ok && n > 0) {
        ok = mbar_wait_sleep(&bar.o_done[tile], t_o++ & 1u, wc, kSiteODone);
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
      }
      if (ok) {
        const bool none = n == 0 || l_run == 0.f;  // no key seen: zeros
        const float inv_l = none ? 0.f : 1.0f / l_run;
        const int q0 = it.q0, hk = it.hk, tok0 = it.tok0;
        const int prow = (tile * TQ + token) * G + g;
        const long long out_at = active ? (long long)(q0 + qi) * a.ldo + (hk * G + g) * D : -1;  // this row's output
        const long long part = ((long long)it.rank * a.heads_k + hk) * P.splits + it.split;
        // this warp's first row: a tile's rows r < TQ G are consecutive in the part
        float* po = kSplit ? P.o + (part * 256 + tile * TQ * G + qq * 32) * D : nullptr;
        const uint32_t rows_in = __ballot_sync(0xffffffffu, active);
        // 64 dims at a time through the warp's staging rows (16-byte pieces swizzled): a warp that holds
        // whole tokens of the sequence hands them to a TMA store and goes on (1.1 us a tile less than
        // stores of 128-byte pieces of four rows each, as the others do it).  A split's fp32 rows leave
        // 32 dims at a time.
        const bool whole_rows = !kSplit && 32 % G == 0 && __all_sync(0xffffffffu, active);
        if (lane == 0) tma_store_wait_read();  // the item before has left the staging rows
        __syncwarp();
        float zero = 0.f;
#pragma unroll 1
        for (int h = 0; h < D / 64; ++h) {
#pragma unroll 1
          for (int cc = 0; cc < 2; ++cc) {
            uint32_t r[32];
            if (n > 0) tmem_load32(tO + h * 64 + cc * 32, r);
            float f[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              f[i] = none ? 0.f : __uint_as_float(r[i]);
              zero = fmaf(f[i], 0.f, zero);  // NaN once a value is not finite
            }
            if (kSplit) {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                *reinterpret_cast<float4*>(staged + lane * 128 + ((i ^ (lane & 7)) << 4)) =
                    make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
              __syncwarp();
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const int r = i * 4 + (lane >> 3);
                if ((rows_in >> r) & 1u)
                  *reinterpret_cast<float4*>(po + r * D + h * 64 + cc * 32 + (lane & 7) * 4) =
                      *reinterpret_cast<const float4*>(staged + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
              }
              __syncwarp();
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                *reinterpret_cast<uint4*>(staged + lane * 128 + (((cc * 4 + i) ^ (lane & 7)) << 4)) =
                    make_uint4(pack_bf16x2(f[8 * i] * inv_l, f[8 * i + 1] * inv_l),
                               pack_bf16x2(f[8 * i + 2] * inv_l, f[8 * i + 3] * inv_l),
                               pack_bf16x2(f[8 * i + 4] * inv_l, f[8 * i + 5] * inv_l),
                               pack_bf16x2(f[8 * i + 6] * inv_l, f[8 * i + 7] * inv_l));
            }
          }
          if (whole_rows) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_4d(&P.o_map, staged, h * 64, 0, hk, q0 + tok0 + tile * TQ + qq * (32 / G));
              if (h + 1 < D / 64) tma_store_wait_read();  // the staging rows are written again
            }
            __syncwarp();
          } else if (!kSplit) {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int r = i * 4 + (lane >> 3);
              const long long at = __shfl_sync(0xffffffffu, out_at, r);
              if (at >= 0)
                *reinterpret_cast<uint4*>(a.out + at + h * 64 + (lane & 7) * 8) =
                    *reinterpret_cast<const uint4*>(staged + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
            }
            __syncwarp();
          }
        }
        if (active && kSplit) P.ml[part * 256 + prow] = none ? make_float2(-INFINITY, 0.f) : make_float2(m_run, l_run);
        // Rows that are not finite: whether a value that they do not see is to blame (causal calls only: the
        // others' tiles hold nothing else) is looked into once the CTA has no item left that waits for this warp.
        const uint32_t rows = __ballot_sync(0xffffffffu, zero != 0.f && active);
        if (rows && a.causal && lane == 0) {
          const int at = sh.odd_n[warp - 2];
          const int id = (it.rank * P.splits + it.split) * a.heads_k + hk;
          sh.odd[(warp - 2) * kOddMost + at] = make_uint2((uint32_t)id, rows);
          sh.odd_n[warp - 2] = at + 1;
          atomicOr(sh.after, kRepair);
        }
      }
      tc_fence_before();  // O has been read before the next item's first P is announced
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.item_free[k & 1]);
    }
    if (lane == 0) tma_store_wait_read();
  }

}

// The rows that came out not finite, each softmax warp its own; nothing is in flight and no role waits.
template <int D, bool kSplit>
__device__ __noinline__ void repair_all(const TextAttnParams& P, uint8_t* smem) {
  const Shared<D> sh(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp < 2 || warp >= 10) return;
  const int records = sh.odd_n[warp - 2];
  if (records == 0) return;
  if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // rows may be written again
  __syncwarp();
  const uint2* mine = sh.odd + (warp - 2) * kOddMost;
  for (int i = 0; i < records; ++i)
    repair_rows<D, kSplit>(P, (int)mine[i].x, mine[i].y, warp, lane, smem + Smem<D>::kOut + (warp - 2) * 4096);
}

template <int D, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1) text_attention_kernel(const __grid_constant__ TextAttnParams P) {
  using L = Smem<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const TextAttnArgs& a = P.a;
  uint32_t tmem;
  {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Shared<D> sh(smem);
    if (threadIdx.x == 32) {
      *sh.abort_flag = 0;
      init_pass(sh);
    }
    if (warp == 2 && lane == 0) {
      tma_prefetch_desc(&P.q_map);
      tma_prefetch_desc(&P.k_map);
      tma_prefetch_desc(&P.v_map);
    }
    __syncwarp();
    if (warp == 1) {
      tmem_alloc(sh.tmem_slot, kTmemCols);
      tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    tmem = *sh.tmem_slot;
  }
  grid_dependency_wait();  // lengths, Q, K, V and the output belong to earlier kernels of the stream
  allow_dependents();

  for (bool first_pass = true;; first_pass = false) {
    // A pass finds its addresses anew: carried from pass to pass they cost the key loop registers (8192 tokens
    // 378 -> 397 us).
    asm volatile("" : "+l"(smem), "+r"(tmem));
    const Shared<D> sh(smem);
    run_items<D, kSplit>(P, sh, tmem, first_pass);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // Nothing is in flight and no role waits: the rows that came out not finite, each warp its own.
    const int after = *(volatile int*)sh.after;
    if (after == 0 || *sh.abort_flag) break;
    repair_all<D, kSplit>(P, sh.smem);
    if (!(after & kAgain)) break;
    __syncthreads();
    if (threadIdx.x == 32) {
      for (int i = 0; i < kBars; ++i) mbar_inval(sh.bars + i);
      init_pass(sh);
    }
    __syncthreads();
  }

  if ((threadIdx.x >> 5) == 1) tmem_dealloc(tmem, kTmemCols);
  // the last CTA leaves the counters as it found them, for the next call on this workspace
  if (threadIdx.x == 0 && atomicAdd(&a.status->items_done, 1u) == gridDim.x - 1) {
    a.status->next_item = 0;
    a.status->items_done = 0;
  }
}

// Adds the splits of every row of a pair of tiles up, in split order: one warp per row, grid (pair
// and key head, eight rows).
template <int D>
__global__ void __launch_bounds__(256) text_attention_join_kernel(const __grid_constant__ TextAttnParams P) {
  grid_dependency_wait();
  allow_dependents();
  const int r = blockIdx.y * 8 + (threadIdx.x >> 5);
  const int hk = blockIdx.x % P.a.heads_k, G = P.group;
  const int2 d = P.desc[blockIdx.x / P.a.heads_k];
  // A call that gave up on a wait may leave rows of the list as they were: whatever they hold, stay in
  // the output.
  if (d.x < 0 || d.y < 0 || d.y > 2 * P.tq || d.x > P.a.rows_q - d.y || r >= d.y * G) return;
  const long long at = (long long)blockIdx.x * P.splits * 256 + r;
  const int token = r / G;
  join_row<D>(P.ml + at, P.o + at * D, 256, P.splits, threadIdx.x & 31,
              P.a.out + (long long)(d.x + token) * P.a.ldo + (hk * G + r - token * G) * D);
}

std::atomic<bool> g_attr_set[64];  // (device, split, head_dim): the shared-memory attribute is raised

template <int D>
cudaError_t launch(const TextAttnArgs& a, const Plan& p, cudaStream_t s) {
  TextAttnParams P;
  memset(&P, 0, sizeof(P));
  const uint64_t G = p.group, Hk = a.heads_k;
  // rows_k == 0: the maps are never used; they only have to be valid
  const bf16* k = a.rows_k > 0 ? a.k : a.q;
  const bf16* v = a.rows_k > 0 ? a.v : a.q;
  const uint64_t qd[4] = {D, G, Hk, (uint64_t)a.rows_q}, qs[3] = {D * 2, G * D * 2, (uint64_t)a.ldq * 2};
  const uint32_t qb[4] = {64, (uint32_t)G, 1, (uint32_t)p.tq};
  const uint64_t rk = a.rows_k > 0 ? a.rows_k : 1;
  const uint64_t kd[3] = {D, Hk, rk}, ks[2] = {D * 2, (uint64_t)a.ldk * 2}, vs[2] = {D * 2, (uint64_t)a.ldv * 2};
  const uint32_t kb[3] = {64, 1, kKeys};
  if (!encode_tmap_bf16(&P.q_map, a.q, 4, qd, qs, qb)) return cudaErrorInvalidValue;
  if (!encode_tmap_bf16(&P.k_map, k, 3, kd, ks, kb)) return cudaErrorInvalidValue;
  if (!encode_tmap_bf16(&P.v_map, v, 3, kd, vs, kb)) return cudaErrorInvalidValue;
  const uint64_t os[3] = {D * 2, G * D * 2, (uint64_t)a.ldo * 2};
  const uint32_t ob[4] = {64, (uint32_t)G, 1, (uint32_t)(32 % G == 0 ? 32 / G : 1)};
  if (!encode_tmap_bf16(&P.o_map, a.out, 4, qd, os, ob)) return cudaErrorInvalidValue;
  P.a = a;
  P.group = p.group;
  P.tq = p.tq;
  P.levels = p.levels;
  P.tiles = p.tiles;
  P.splits = p.splits;
  P.scale_log2 = (float)(1.4426950408889634 * (double)a.scale);
  const Parts l = parts_layout(p, a.heads_k, D);
  uint8_t* ws = reinterpret_cast<uint8_t*>(a.parts);
  int2* list = reinterpret_cast<int2*>(ws + l.list);
  P.list = p.list ? list : nullptr;
  P.desc = reinterpret_cast<int2*>(ws + l.desc);
  P.ml = reinterpret_cast<float2*>(ws + l.ml);
  P.o = reinterpret_cast<float*>(ws + l.o);
  const size_t smem = Smem<D>::kBytes;
  auto kernel = p.splits > 1 ? text_attention_kernel<D, true> : text_attention_kernel<D, false>;
  int dev = 0;
  cudaGetDevice(&dev);
  const int slot = dev * 4 + (p.splits > 1) * 2 + (D == 64);
  if (dev >= 16 || !g_attr_set[slot].load(std::memory_order_acquire)) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    if (dev < 16) g_attr_set[slot].store(true, std::memory_order_release);
  }
  if (p.list) {
    LaunchScope scope(kClsTextAttention, s);
    cudaError_t e =
        launch_k(text_attention_list_kernel, dim3(1), dim3(1024), 0, s, a, p.tq * 2, p.levels, p.tiles, list);
    if (e != cudaSuccess) return e;
  }
  // Under 2^31 - 2^16 at any sizes that are accepted: pairs of tiles x key heads come to 1.55e9 at most (2^28
  // rows, groups of 44 heads), and keys are split only where that leaves fewer than an item per SM.
  const long long items = (long long)p.tiles * a.heads_k * p.splits;
  P.items = (int)items;
  const int sms = sm_count(), grid = items < sms ? (int)items : sms;
  {
    LaunchScope scope(kClsTextAttention, s);
    cudaError_t e = launch_k(kernel, dim3((unsigned)grid), dim3(kThreads), smem, s, P);
    if (e != cudaSuccess) return e;
  }
  if (p.splits > 1) {
    LaunchScope scope(kClsTextJoin, s);
    return launch_k(text_attention_join_kernel<D>, dim3((unsigned)(p.tiles * a.heads_k), 32), dim3(256), 0, s, P);
  }
  return cudaSuccess;
}

// ---- few query rows ---------------------------------------------------------------------------

// Tiles of 16 query rows of a key head (new tokens, heads of the group among them): with one tile reading
// the keys and values bounds the time, so what counts is bytes in flight, not the MMA rate.  One CTA
// per (run of keys, key head, sequence, tile), two per SM, each with three stages of 64 keys (64 * D * 4
// bytes) on their way by TMA; four warps take 16 keys of a stage each through mma.sync with their own
// running maximum and sum and add up at the end, in order.  Runs of several CTAs are joined by a second
// kernel.  A 128-row tcgen05 tile of mostly empty rows took 153 us where this takes 115 (48 tokens over
// 100 to 8192 keys, 8 key heads of 128).
constexpr int kFewMost = 2 * kSMs * 16;  // rows per key head that one wave can hold
constexpr int kFewRows = 16, kFewKeys = 64, kFewStages = 3, kFewThreads = 160;

struct FewPlan {
  int rows, tiles;    // query rows per key head, and tiles of 16 of them
  int chunk, splits;  // keys per CTA, CTAs per sequence, head and tile
};

// Runs of at most 1024 keys, so that ragged lengths even out over the CTAs, and of at least 256 (a
// run costs ~3 us besides its keys), that cut the longest sequences' keys into two waves of CTAs; and
// no more than 16384 runs in all, which bounds the workspace.  Eight waves of 128 keys or more took
// 27 tokens over 2021 to 3362 keys (3 heads of 128) from 27.6 to 40.6 us, one token over 8192 (8
// heads) from 13.4 to 20.4.
FewPlan few_plan(const TextAttnArgs& a) {
  FewPlan p;
  const long long rows = (long long)a.max_q * (a.heads_q / a.heads_k);
  p.rows = rows < kFewMost ? (int)rows : kFewMost;
  p.tiles = (p.rows + kFewRows - 1) / kFewRows;
  const long long items = (long long)a.seqs * a.heads_k * p.tiles;
  long long chunk = (long long)a.max_k * items / (4 * kSMs);
  if (chunk > 1024) chunk = 1024;
  const long long least = (long long)a.max_k * items / 16384;
  if (chunk < least) chunk = least;
  if (chunk > a.max_k) chunk = a.max_k;  // `least` passes 32 bits where many sequences may be long
  if (chunk < 256) chunk = 256;
  p.chunk = (int)((chunk + kFewKeys - 1) / kFewKeys * kFewKeys);
  p.splits = (a.max_k + p.chunk - 1) / p.chunk;
  if (p.splits < 1) p.splits = 1;
  return p;
}

// Up to 16 rows per key head always; more where all the CTAs run at once.  Then reading the keys again
// for every 16 rows costs less than the tile kernel's longer way to its first score: 40 causal tokens
// of 32 heads on 8 take 4.7 us against 7.9, 77 6.8 and 8.2, 8 single tokens of 32 heads on one over 4000
// keys 11.9 and 16.5; past one wave it turns (256 tokens 13.9 and 9.8, 4 x 64 tokens 11.5 and 8.3).
bool few_rows(const TextAttnArgs& a) {
  const long long rows = (long long)a.max_q * (a.heads_q / a.heads_k);
  if (rows <= kFewRows) return true;
  if (rows > kFewMost) return false;
  if ((long long)a.seqs * a.heads_k * ((rows + kFewRows - 1) / kFewRows) > 2 * kSMs) return false;
  const FewPlan p = few_plan(a);
  return (long long)a.seqs * a.heads_k * p.tiles * p.splits <= 2 * kSMs;
}

Parts few_parts(const FewPlan& p, const TextAttnArgs& a) {
  Parts l;
  const size_t n = p.splits > 1 ? (size_t)a.seqs * a.heads_k * p.splits * p.rows : 0;
  l.list = l.desc = l.ml = 0;
  l.o = up256(n * 8);
  l.total = l.o + up256(n * (size_t)a.head_dim * 4);
  return l;
}

struct alignas(64) FewParams {
  CUtensorMap k_map, v_map;
  TextAttnArgs a;
  int group, rows, tiles, chunk, splits;
  float scale_log2;
  float2* ml;
  float* o;
};

enum : uint32_t { kSiteFewFull = 0x521, kSiteFewEmpty };

// Keys that the tile of query rows [base, base + 16) of a sequence sees: those of its last row.
__device__ __forceinline__ int few_keys(const TextAttnArgs& a, const Span& sp, int G, int base) {
  if (!a.causal) return sp.nk;
  return min(sp.nk, max(0, min(base + kFewRows, sp.nq * G) - 1) / G + sp.nk - sp.nq + 1);
}

template <int D>
__global__ void __launch_bounds__(kFewThreads, 2) text_attention_few_kernel(const __grid_constant__ FewParams P) {
  constexpr uint32_t kHalf = kFewKeys * 128;            // 64 keys x 64 dims
  constexpr uint32_t kTile = (D / 64) * kHalf, kStage = 2 * kTile;
  constexpr int V = D / 32;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t full[kFewStages], empty[kFewStages];
  __shared__ float2 ml[4][kFewRows];
  __shared__ int abort_flag;
  const TextAttnArgs& a = P.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, G = P.group;
  // the tiles of the same keys run side by side
  const int run = blockIdx.x / P.tiles, base = (blockIdx.x - run * P.tiles) * kFewRows;
  const int split = run % P.splits, hk = (run / P.splits) % a.heads_k;
  const int seq = run / P.splits / a.heads_k;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kFewStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 4);
    }
    abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  grid_dependency_wait();
  allow_dependents();
  const Span sp = load_span(a, seq);
  if (!sp.ok) {
    if (split == 0 && hk == 0 && base == 0 && threadIdx.x == 0) report_bad_entry(a.status, kSiteTextLengths);
    return;
  }
  const int rows = min(kFewRows, sp.nq * G - base);  // this CTA's query rows
  if (rows <= 0) return;
  // this CTA's keys, none behind the last that its rows see
  const int first = split * P.chunk, last = min(few_keys(a, sp, G, base), first + P.chunk);
  const bool direct = sp.nk <= P.chunk;  // it has all the keys of its rows
  if (first >= last && split > 0) return;
  const int blocks = first < last ? (last - first + kFewKeys - 1) / kFewKeys : 0;
  const WaitCtx wc{a.status, &abort_flag, kWaitLimitNs};

  if (warp == 4) {
    if (lane == 0) {
      int issued = 0;
      bool ok = true;
      for (int j = 0; j < blocks; ++j) {
        const int st = j % kFewStages;
        if (!mbar_wait_sleep(&empty[st], ((uint32_t)(j / kFewStages) & 1u) ^ 1u, wc, kSiteFewEmpty)) {
          ok = false;
          break;
        }
        uint8_t* at = smem + st * kStage;
        mbar_arrive_expect_tx(&full[st], kStage);
        for (int h = 0; h < D / 64; ++h) {
          tma_load_3d(at + h * kHalf, &P.k_map, &full[st], h * 64, hk, sp.k0 + first + j * kFewKeys);
          tma_load_3d(at + kTile + h * kHalf, &P.v_map, &full[st], h * 64, hk, sp.k0 + first + j * kFewKeys);
        }
        issued = j + 1;
      }
      if (!ok) {
        const uint64_t t0 = global_timer_ns();
        for (int j = issued > kFewStages ? issued - kFewStages : 0; j < issued; ++j)
          while (!mbar_try(&full[j % kFewStages], (uint32_t)(j / kFewStages) & 1u) &&
                 global_timer_ns() - t0 < 200000000ull) {
          }
      }
    }
  }

  // Fragments: this lane's rows are lane / 4 and lane / 4 + 8, its columns 2 (lane % 4) + {0, 1}.
  const int r0 = lane >> 2, c0 = (lane & 3) * 2;
  float o[D / 8][4];
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  const float c = P.scale_log2;
  if (warp < 4) {
    uint32_t q[D / 16][4];
    int limit[2];  // keys that the lane's rows see
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = base + r0 + 8 * i, token = r / G;
      const bool ok = r0 + 8 * i < rows;
      const bf16* src = a.q + (long long)(sp.q0 + (ok ? token : 0)) * a.ldq + (hk * G + (ok ? r - token * G : 0)) * D + c0;
      limit[i] = !ok ? 0 : (a.causal ? min(sp.nk, token + sp.nk - sp.nq + 1) : sp.nk);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        q[k][i] = ok ? *reinterpret_cast<const uint32_t*>(src + k * 16) : 0u;
        q[k][i + 2] = ok ? *reinterpret_cast<const uint32_t*>(src + k * 16 + 8) : 0u;
      }
    }
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    // ldmatrix rows: K as (keys 0-7 | 0-7 | 8-15 | 8-15) x (dims 0-7 | 8-15 | 0-7 | 8-15), V transposed as
    // (keys 0-7 | 8-15 | 0-7 | 8-15) x (dims 0-7 | 0-7 | 8-15 | 8-15), each of this warp's 16 keys
    const int kk = warp * 16 + (lane & 7) + ((lane >> 4) << 3), kc = (lane >> 3) & 1;
    const int vk = warp * 16 + (lane & 15), vc = lane >> 4;
    for (int j = 0; j < blocks; ++j) {
      const int st = j % kFewStages;
      bool ok = mbar_wait(&full[st], (uint32_t)(j / kFewStages) & 1u, wc, kSiteFewFull);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      uint8_t* at = smem + st * kStage;
      const int key0 = first + j * kFewKeys + warp * 16;
      if (key0 < last) {
        if (key0 + 16 > last) {
          // V rows past this run's keys must read as zeros: a zero probability does not silence a NaN
          for (int h = 0; h < D / 64; ++h)
            for (int i = lane; i < 16 * 8; i += 32)
              if (key0 + (i >> 3) >= last)
                *reinterpret_cast<uint4*>(at + kTile + h * kHalf + (warp * 16 + (i >> 3)) * 128 + (i & 7) * 16) =
                    make_uint4(0u, 0u, 0u, 0u);
          __syncwarp();
        }
        float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          uint32_t b[4];
          ldmatrix4(b, smem_u32(at + (k >> 2) * kHalf + kk * 128 + (((((k & 3) * 2) + kc) ^ (kk & 7)) << 4)));
          mma_bf16(s[0], q[k], b[0], b[1]);
          mma_bf16(s[1], q[k], b[2], b[3]);
        }
        float alpha[2];
        uint32_t p[4];  // probabilities, rounded to bf16 for the product with V (see the top)
#pragma unroll
        for (int i = 0; i < 2; ++i) {  // the lane's two rows
          float x[4];
          float mx = -INFINITY;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = key0 + (e >> 1) * 8 + c0 + (e & 1);
            x[e] = key < min(limit[i], last) ? s[e >> 1][2 * i + (e & 1)] * c : -INFINITY;
            mx = fmaxf(mx, x[e]);
          }
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          const float mn = fmaxf(m[i], mx), ref = mn == -INFINITY ? 0.f : mn;
          alpha[i] = ex2_approx(m[i] - ref);
          m[i] = mn;
          float sum = 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[e] = ex2_approx(x[e] - ref);
            sum += x[e];
          }
          l[i] = l[i] * alpha[i] + sum;
          p[i] = pack_bf16x2(x[0], x[1]);
          p[i + 2] = pack_bf16x2(x[2], x[3]);
        }
        if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            o[i][0] *= alpha[0];
            o[i][1] *= alpha[0];
            o[i][2] *= alpha[1];
            o[i][3] *= alpha[1];
          }
        }
#pragma unroll
        for (int d = 0; d < D / 16; ++d) {
          uint32_t b[4];
          ldmatrix4_trans(b, smem_u32(at + kTile + (d >> 2) * kHalf + vk * 128 + (((((d & 3) * 2) + vc) ^ (vk & 7)) << 4)));
          mma_bf16(o[2 * d], p, b[0], b[1]);
          mma_bf16(o[2 * d + 1], p, b[2], b[3]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }
  }

  // The four warps' rows through shared memory (all stages have been read)
  __syncthreads();
  float* parts = reinterpret_cast<float*>(smem);  // [warp][row][dim]
  if (warp < 4) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      const int r = r0 + 8 * i;
      if ((lane & 3) == 0) ml[warp][r] = make_float2(m[i], l[i]);
      if (r < rows) {
#pragma unroll
        for (int d = 0; d < D / 8; ++d)
          *reinterpret_cast<float2*>(parts + (warp * kFewRows + r) * D + d * 8 + c0) = make_float2(o[d][2 * i], o[d][2 * i + 1]);
      }
    }
  }
  __syncthreads();
  if (warp == 4 || abort_flag) return;
  uint32_t odd = 0;  // rows that are not finite
  for (int r = warp; r < rows; r += 4) {
    float mr = -INFINITY, lr = 0.f, out[V];
#pragma unroll
    for (int w = 0; w < 4; ++w) mr = fmaxf(mr, ml[w][r].x);
    const float ref = mr == -INFINITY ? 0.f : mr;
#pragma unroll
    for (int e = 0; e < V; ++e) out[e] = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float2 x = ml[w][r];
      if (x.y == 0.f) continue;  // no key that the row sees
      const float f = ex2_approx(x.x - ref);
      lr += f * x.y;
#pragma unroll
      for (int e = 0; e < V; ++e) out[e] += f * parts[(w * kFewRows + r) * D + lane * V + e];
    }
    const int token = (base + r) / G, g = base + r - token * G;
    float zero = 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e) zero = fmaf(out[e], 0.f, zero);
    if (__any_sync(0xffffffffu, zero != 0.f)) odd |= 1u << r;
    if (direct) {
      const float inv = lr == 0.f ? 0.f : 1.0f / lr;
      bf16* dst = a.out + (long long)(sp.q0 + token) * a.ldo + (hk * G + g) * D + lane * V;
#pragma unroll
      for (int e = 0; e < V; e += 2)
        *reinterpret_cast<uint32_t*>(dst + e) = lr == 0.f ? 0u : pack_bf16x2(out[e] * inv, out[e + 1] * inv);
    } else {
      const long long at = (long long)run * P.rows + base + r;
      if (lane == 0) P.ml[at] = make_float2(mr, lr);
#pragma unroll
      for (int e = 0; e < V; e += 2)
        *reinterpret_cast<float2*>(P.o + at * D + lane * V + e) = make_float2(out[e], out[e + 1]);
    }
  }
  if (odd) {
    // was it a value behind the keys that the row sees?
    const bool mine = (odd >> lane) & 1u;
    const int token = (base + lane) / G, g = base + lane - token * G;
    const int seen = a.causal ? min(sp.nk, token + sp.nk - sp.nq + 1) : sp.nk;
    const bf16* vp = a.v + (long long)sp.k0 * a.ldv + hk * D;
    odd = __ballot_sync(0xffffffffu, mine && seen < last);
    if (odd) odd = spoiled_rows<D>(vp, a.ldv, odd, seen, first, last, lane);
    if (odd) {
      __syncwarp();  // the rows have been written by other lanes
      const bool redo = (odd >> lane) & 1u;
      const long long row = sp.q0 + (redo ? token : 0), at = (long long)run * P.rows + base + lane;
      const int col = (hk * G + (redo ? g : 0)) * D, keys = redo ? seen - first : 0;
      const bf16 *q = a.q + row * a.ldq + col, *k = a.k + (long long)(sp.k0 + first) * a.ldk + hk * D;
      vp += (long long)first * a.ldv;
      uint8_t* stage = smem + 4 * kFewRows * D * 4 + warp * 16 * D * 2;  // behind the warps' parts
      if (direct) attend_rows<D, false>(a, q, k, vp, keys, c, lane, a.out + row * a.ldo + col, nullptr, stage);
      else attend_rows<D, true>(a, q, k, vp, keys, c, lane, P.o + at * D, P.ml + at, stage);
    }
  }
}

// Adds up the runs of the sequences that took several, in order: one warp per row, grid (sequence
// and key head, four rows).
template <int D>
__global__ void __launch_bounds__(128) text_attention_few_join_kernel(const __grid_constant__ FewParams P) {
  grid_dependency_wait();
  allow_dependents();
  const TextAttnArgs& a = P.a;
  const int r = blockIdx.y * 4 + (threadIdx.x >> 5), G = P.group;
  const int hk = blockIdx.x % a.heads_k, seq = blockIdx.x / a.heads_k;
  const Span sp = load_span(a, seq);
  if (!sp.ok || sp.nk <= P.chunk || r >= sp.nq * G) return;
  const long long at = (long long)blockIdx.x * P.splits * P.rows + r;
  const int token = r / G, runs = (few_keys(a, sp, G, r / kFewRows * kFewRows) + P.chunk - 1) / P.chunk;
  join_row<D>(P.ml + at, P.o + at * D, P.rows, max(1, runs), threadIdx.x & 31,
              a.out + (long long)(sp.q0 + token) * a.ldo + (hk * G + r - token * G) * D);
}

std::atomic<bool> g_few_attr_set[32];  // (device, head_dim)

template <int D>
cudaError_t launch_few(const TextAttnArgs& a, cudaStream_t s) {
  const FewPlan p = few_plan(a);
  FewParams P;
  memset(&P, 0, sizeof(P));
  const uint64_t rk = a.rows_k > 0 ? a.rows_k : 1, Hk = a.heads_k;
  const uint64_t kd[3] = {D, Hk, rk}, ks[2] = {D * 2, (uint64_t)a.ldk * 2}, vs[2] = {D * 2, (uint64_t)a.ldv * 2};
  const uint32_t kb[3] = {64, 1, kFewKeys};
  if (a.rows_k > 0 &&
      (!encode_tmap_bf16(&P.k_map, a.k, 3, kd, ks, kb) || !encode_tmap_bf16(&P.v_map, a.v, 3, kd, vs, kb)))
    return cudaErrorInvalidValue;
  const Parts l = few_parts(p, a);
  uint8_t* ws = reinterpret_cast<uint8_t*>(a.parts);
  P.a = a;
  P.group = a.heads_q / a.heads_k;
  P.rows = p.rows;
  P.tiles = p.tiles;
  P.chunk = p.chunk;
  P.splits = p.splits;
  P.scale_log2 = (float)(1.4426950408889634 * (double)a.scale);
  P.ml = reinterpret_cast<float2*>(ws + l.ml);
  P.o = reinterpret_cast<float*>(ws + l.o);
  const size_t smem = 1024 + (size_t)kFewStages * kFewKeys * D * 4;
  int dev = 0;
  cudaGetDevice(&dev);
  const int slot = dev * 2 + (D == 64);
  if (dev >= 16 || !g_few_attr_set[slot].load(std::memory_order_acquire)) {
    cudaError_t e =
        cudaFuncSetAttribute(text_attention_few_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    if (dev < 16) g_few_attr_set[slot].store(true, std::memory_order_release);
  }
  // up to 2^24 sequences x key heads of one run, or about 16384 runs
  const long long grid = (long long)a.seqs * a.heads_k * p.splits * p.tiles;
  {
    LaunchScope scope(kClsTextAttention, s);
    cudaError_t e = launch_k(text_attention_few_kernel<D>, dim3((unsigned)grid), dim3(kFewThreads), smem, s, P);
    if (e != cudaSuccess) return e;
  }
  if (p.splits > 1) {
    LaunchScope scope(kClsTextJoin, s);
    return launch_k(text_attention_few_join_kernel<D>, dim3((unsigned)(a.seqs * a.heads_k), (unsigned)((p.rows + 3) / 4)),
                    dim3(128), 0, s, P);
  }
  return cudaSuccess;
}

}  // namespace

size_t text_attention_parts_bytes(const TextAttnArgs& a) {
  if (a.seqs == 0 || a.rows_q == 0 || a.max_q == 0) return 0;
  if (few_rows(a)) return few_parts(few_plan(a), a).total;
  return parts_layout(make_plan(a), a.heads_k, a.head_dim).total;
}

cudaError_t launch_text_attention(const TextAttnArgs& a, cudaStream_t s) {
  if (few_rows(a)) return a.head_dim == 64 ? launch_few<64>(a, s) : launch_few<128>(a, s);
  const Plan p = make_plan(a);
  return a.head_dim == 64 ? launch<64>(a, p, s) : launch<128>(a, p, s);
}

}  // namespace dit
