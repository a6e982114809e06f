// Base-2 log-sum-exp states of the top-logits kernels.  Unlike the states of
// the dense loss they take rows with -inf entries anywhere (masked logits,
// words that are left out): while a state has seen nothing finite its offset
// is 0, so that -inf adds 0 and not NaN.  NaN and +inf stay visible as NaN.
#pragma once

#include "fct_common.cuh"

namespace fct {
namespace top {

// Folds a vector with maximum vm into a state.
template <int N>
__device__ __forceinline__ void fold(Lse2x& st, const float (&x)[N], float vm) {
  static_assert(N % 2 == 0, "pairs");
  const float m2n = vm * kLog2e;
  if (m2n > st.m2) {
    const float sc = ex2(st.m2 - m2n);
    st.s.x *= sc;
    st.s.y *= sc;
    st.m2 = m2n;
  }
  const float nm = st.m2 == -INFINITY ? 0.f : -st.m2;
  const float2 L2 = make_float2(kLog2e, kLog2e), n2 = make_float2(nm, nm);
#pragma unroll
  for (int j = 0; j < N; j += 2) {
    const float2 e = __ffma2_rn(make_float2(x[j], x[j + 1]), L2, n2);
    st.s = __fadd2_rn(st.s, make_float2(ex2(e.x), ex2(e.y)));
  }
}
template <int N>
__device__ __forceinline__ void fold(Lse2x& st, const float (&x)[N]) {
  fold(st, x, vec_max(x));
}

// A state's sum relative to the maximum m (at least its own).  An empty state
// has the sum 0; one of NaN alone has no maximum, and keeps its NaN.
__device__ __forceinline__ float rescaled(Lse2 a, float m) {
  return a.s == 0.f ? 0.f : a.m2 == -INFINITY ? a.s : a.s * ex2(a.m2 - m);
}
__device__ __forceinline__ Lse2 merge(Lse2 a, Lse2 b) {
  const float m = fmaxf(a.m2, b.m2);
  return Lse2{m, rescaled(a, m) + rescaled(b, m)};
}
__device__ __forceinline__ Lse2 warp_merge(Lse2 a) {
  float m = a.m2;
#pragma unroll
  for (int k = 16; k >= 1; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
  return Lse2{m, warp_sum(rescaled(a, m))};
}

// Natural log-sum-exp of a state, rounded once: the maximum and the
// logarithm's whole part are added to its fraction in 64 bits.  (In fp32 the
// three roundings would be of numbers near 20, and the backward takes
// exp(x - lse) of the result.)
__device__ __forceinline__ float finish(float m2, float s) {
  if (s == 0.f) return -INFINITY;
  if (!(s > 0.f) || !(fabsf(m2) < INFINITY)) return __uint_as_float(0x7fc00000u);
  int e;
  const float f = frexpf(s, &e);
  return static_cast<float>((double(m2) + double(e) + double(log2f(f))) * 0.6931471805599453);
}

}  // namespace top
}  // namespace fct
