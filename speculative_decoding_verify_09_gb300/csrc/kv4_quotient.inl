// Quotients of many numbers by one.  Host code compiles this as well.
//
// A reciprocal y0 within a few steps of 1 / d is refined by one step of Newton's iteration,
//   y = y0 + y0 (1 - d y0),
// and the product q0 = x y corrected by its remainder,
//   q = q0 + y (x - d q0),
// all in fused products (P. W. Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", IBM Journal of Research and Development 34, 1990).  The remainder of a
// q0 within a step of x / d is exact, so that q differs from the rounded quotient by a step at
// most, and only where the quotient lies within 2^-22 of a step of the middle of two numbers; an
// exact quotient (a tie of two codes) is met exactly.
//
// Ops: T, mul(a, b), fma(a, b, c).
#pragma once

#ifdef __CUDACC__
#define SV_QUOTIENT __host__ __device__ __forceinline__
#else
#define SV_QUOTIENT inline
#endif

namespace sv {

namespace {

template <typename Ops, typename T = typename Ops::T>
SV_QUOTIENT T refined_reciprocal(T minus_d, T near, T one) {
  return Ops::fma(Ops::fma(minus_d, near, one), near, near);
}

template <typename Ops, typename T = typename Ops::T>
SV_QUOTIENT T corrected_quotient(T x, T minus_d, T reciprocal) {
  const T q = Ops::mul(x, reciprocal);
  return Ops::fma(Ops::fma(q, minus_d, x), reciprocal, q);
}

}  // namespace

}  // namespace sv
