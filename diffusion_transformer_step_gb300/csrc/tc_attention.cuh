// Pieces of attention on the tensor cores that the kernels share: the softmax of one row of
// scores in Tensor Memory, and batches of tcgen05 MMAs.
#pragma once

#include <math.h>

#include "common.cuh"

namespace dit {

// ---- softmax arithmetic helpers -----------------------------------------------------

__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// (d0, d1) = (a0, a1) * b + c with one packed fp32x2 FMA.
__device__ __forceinline__ void ffma2(float& d0, float& d1, float a0, float a1, float b, float c) {
  uint64_t A, B, C, D;
  asm("mov.b64 %0, {%1, %2};" : "=l"(A) : "f"(a0), "f"(a1));
  asm("mov.b64 %0, {%1, %1};" : "=l"(B) : "f"(b));
  asm("mov.b64 %0, {%1, %1};" : "=l"(C) : "f"(c));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(D) : "l"(A), "l"(B), "l"(C));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d0), "=f"(d1) : "l"(D));
}

// (s0, s1) += (a0, a1) with one packed fp32x2 add.
__device__ __forceinline__ void fadd2(float& s0, float& s1, float a0, float a1) {
  uint64_t S, A;
  asm("mov.b64 %0, {%1, %2};" : "=l"(S) : "f"(s0), "f"(s1));
  asm("mov.b64 %0, {%1, %2};" : "=l"(A) : "f"(a0), "f"(a1));
  asm("add.f32x2 %0, %0, %1;" : "+l"(S) : "l"(A));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(s0), "=f"(s1) : "l"(S));
}

// One 32-key chunk of a softmax row: P = 2^(s c - m) packed to bf16 pairs and the two
// partial row sums; kMax: also the running key maximum (raw scores); kTail: keys at or past
// kv_valid masked to -inf.  Every exponential runs on MUFU: moving a share of them to an
// FMA-pipe polynomial was measured slower here.
template <bool kTail, bool kMax>
__device__ __forceinline__ void softmax_chunk(const uint32_t (&r)[32], int base, int kv_valid, float c, float mneg,
                                              float& smax, float& ps0, float& ps1, uint32_t* pk) {
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    float s0 = __uint_as_float(r[i]), s1 = __uint_as_float(r[i + 1]);
    if (kTail) {
      if (base + i >= kv_valid) s0 = -INFINITY;
      if (base + i + 1 >= kv_valid) s1 = -INFINITY;
    }
    if (kMax) smax = fmax3(smax, s0, s1);
    float x0, x1;
    ffma2(x0, x1, s0, s1, c, mneg);
    const float p0 = ex2_approx(x0);
    const float p1 = ex2_approx(x1);
    fadd2(ps0, ps1, p0, p1);
    pk[i / 2] = pack_bf16x2(p0, p1);
  }
}

template <bool kTail, bool kMax>
__device__ __forceinline__ void softmax_row(uint32_t tS, int kv_valid, float c, float mneg, float& smax, float& psum,
                                            uint32_t (&pk)[64]) {
  float ps0 = 0.f, ps1 = 0.f;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t r[32];
    tmem_load32(tS + q * 32, r);
    softmax_chunk<kTail, kMax>(r, q * 32, kv_valid, c, mneg, smax, ps0, ps1, &pk[q * 16]);
  }
  psum = ps0 + ps1;
}

// Eight back-to-back MMAs (K = 128) from one asm statement: D = A B (first) then D += A B.
__device__ __forceinline__ void umma8_ss(uint32_t d, const uint64_t (&a)[8], const uint64_t (&b)[8], uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred pf, pt;\n\t"
      "setp.ne.b32 pf, %18, %18;\n\t"
      "setp.eq.b32 pt, %18, %18;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %9, %17, pf;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %2, %10, %17, pt;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %3, %11, %17, pt;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %4, %12, %17, pt;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %5, %13, %17, pt;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %6, %14, %17, pt;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %7, %15, %17, pt;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %8, %16, %17, pt;\n\t}" ::"r"(d),
      "l"(a[0]), "l"(a[1]), "l"(a[2]), "l"(a[3]), "l"(a[4]), "l"(a[5]), "l"(a[6]), "l"(a[7]), "l"(b[0]), "l"(b[1]),
      "l"(b[2]), "l"(b[3]), "l"(b[4]), "l"(b[5]), "l"(b[6]), "l"(b[7]), "r"(idesc), "r"(0)
      : "memory");
}

// Four of them (K = 64).
__device__ __forceinline__ void umma4_ss(uint32_t d, const uint64_t (&a)[4], const uint64_t (&b)[4], uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred pf, pt;\n\t"
      "setp.ne.b32 pf, %10, %10;\n\t"
      "setp.eq.b32 pt, %10, %10;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %5, %9, pf;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %2, %6, %9, pt;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %3, %7, %9, pt;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %4, %8, %9, pt;\n\t}" ::"r"(d),
      "l"(a[0]), "l"(a[1]), "l"(a[2]), "l"(a[3]), "l"(b[0]), "l"(b[1]), "l"(b[2]), "l"(b[3]), "r"(idesc), "r"(0)
      : "memory");
}

// Eight MMAs with A read from TMEM at columns a_tmem + 8 kk: D (+)= A B.
__device__ __forceinline__ void umma8_ts(uint32_t d, uint32_t a_tmem, const uint64_t (&b)[8], uint32_t idesc,
                                         uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred pa, pt;\n\t.reg .b32 t1, t2, t3, t4, t5, t6, t7;\n\t"
      "setp.ne.b32 pa, %11, 0;\n\t"
      "setp.eq.b32 pt, %11, %11;\n\t"
      "add.u32 t1, %1, 8;\n\tadd.u32 t2, %1, 16;\n\tadd.u32 t3, %1, 24;\n\tadd.u32 t4, %1, 32;\n\t"
      "add.u32 t5, %1, 40;\n\tadd.u32 t6, %1, 48;\n\tadd.u32 t7, %1, 56;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %10, pa;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [t1], %3, %10, pt;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [t2], %4, %10, pt;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [t3], %5, %10, pt;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [t4], %6, %10, pt;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [t5], %7, %10, pt;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [t6], %8, %10, pt;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [t7], %9, %10, pt;\n\t}" ::"r"(d),
      "r"(a_tmem), "l"(b[0]), "l"(b[1]), "l"(b[2]), "l"(b[3]), "l"(b[4]), "l"(b[5]), "l"(b[6]), "l"(b[7]), "r"(idesc),
      "r"(acc)
      : "memory");
}

}  // namespace dit
