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

// exp(x - l), the probability of a logit x under a log-sum-exp l held in fp32.
__device__ __forceinline__ float prob(float x, float l) { return ex2((x - l) * kLog2e); }

// The sign of p - q for logits x and y under log-sum-exps l and m held in
// fp32, with a row's sigma.  Where p and q are both near 1 (a student and a
// teacher that are sure of one word) l and m lose what tells them apart: their
// roundings, up to `doubt`, exceed 1 - p and 1 - q, and a sign that differs
// from the one in sigma leaves p (sign - sigma) near 1 or 2 where it should be
// 0.  A word or a rest with p > 3/4 is the only one, and its sign is that of
// sigma: |sigma| > 1/2 with a sign, < 1/4 with none.
__device__ __forceinline__ float sign_of(float x, float l, float y, float m, float doubt,
                                         float sigma) {
  const float p = prob(x, l);
  if (p > 0.75f && fabsf((x - l) - (y - m)) <= doubt)
    return sigma > 0.375f ? 1.f : sigma < -0.375f ? -1.f : 0.f;
  return sgn_pq(p, prob(y, m));
}

// What a row's gradient is made of.
struct Coefs {
  float gce, h;  // grad_ce, grad_tvd / 2
  float lse, t_lse, sigma;
  float doubt;   // most that (s - lse) - (t - t_lse) is off by the roundings of the two
  float outside; // coefficient of p_v outside U
  bool teacher;  // the list holds some probability
};
__device__ __forceinline__ Coefs make_coefs(float gce, float gtvd, float lse, float rest,
                                            float t_lse, float t_rest, float sigma) {
  const float doubt = (fabsf(lse) + fabsf(t_lse)) * 1.1920929e-07f;  // twice the half steps
  Coefs c{gce, 0.5f * gtvd, lse, t_lse, sigma, doubt, gce, !(t_lse == -INFINITY)};
  if (c.teacher)
    c.outside = fmaf(c.h, sign_of(rest, lse, t_rest, t_lse, doubt + fabsf(rest) * 1.1920929e-07f,
                                  sigma) - sigma, gce);
  return c;
}
// The gradient at a listed word with student logit s and teacher logit t.
__device__ __forceinline__ float listed_grad(const Coefs& c, float s, float t, bool target) {
  const float p = prob(s, c.lse);
  const float k =
      c.teacher ? fmaf(c.h, sign_of(s, c.lse, t, c.t_lse, c.doubt, c.sigma) - c.sigma, c.gce) : c.gce;
  return target ? fmaf(p, k, -c.gce) : p * k;
}

struct Sums {  // of one row's list, held by every lane of a warp
  float lse, rest, t_lse, tvd, sigma;
};

// The list's part of the loss, by one warp: the student's and the teacher's
// logits of K places (-inf where unused), and the student's state outside U.
// The signs are those of p and q from their sums, before any log-sum-exp is
// rounded.
static __device__ Sums list_sums(const float* s, const float* t, int K, float rest_m2, float rest_s,
                                 float t_rest) {
  const int lane = threadIdx.x & 31;
  float ms = -INFINITY, mt = t_rest;
  for (int k = lane; k < K; k += 32) {
    ms = fmaxf(ms, s[k]);
    mt = fmaxf(mt, t[k]);
  }
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) {
    ms = fmaxf(ms, __shfl_xor_sync(0xffffffffu, ms, m));
    mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, m));
  }
  const float ms2 = fmaxf(ms * kLog2e, rest_m2), mt2 = mt * kLog2e;
  const float ns = ms2 == -INFINITY ? 0.f : -ms2, nt = mt2 == -INFINITY ? 0.f : -mt2;
  float us = 0.f, ut = 0.f;
  for (int k = lane; k < K; k += 32) {
    us += ex2(fmaf(s[k], kLog2e, ns));
    ut += ex2(fmaf(t[k], kLog2e, nt));
  }
  us = warp_sum(us);
  ut = warp_sum(ut);
  const float rs = rest_s == 0.f ? 0.f : rest_s * ex2(rest_m2 + ns);
  const float rt = ex2(fmaf(t_rest, kLog2e, nt));
  const float zs = us + rs, zt = ut + rt;
  Sums o;
  o.lse = finish(ms2, zs);
  o.rest = finish(rest_m2, rest_s);
  o.t_lse = finish(mt2, zt);
  if (o.t_lse == -INFINITY) {  // no teacher: cross-entropy alone
    o.tvd = 0.f;
    o.sigma = 0.f;
    return o;
  }
  const float is = 1.f / zs, it = 1.f / zt;
  float d = 0.f, g = 0.f;
  for (int k = lane; k < K; k += 32) {
    // (products rounded by themselves: equal p and q differ by 0)
    const float p = __fmul_rn(ex2(fmaf(s[k], kLog2e, ns)), is);
    const float q = __fmul_rn(ex2(fmaf(t[k], kLog2e, nt)), it);
    d += fabsf(p - q);
    g += p * sgn_pq(p, q);
  }
  d = warp_sum(d);
  g = warp_sum(g);
  // where both sides have most of their mass outside U, the difference of the
  // two large numbers is that of the small ones inside
  const float p = __fmul_rn(rs, is), q = __fmul_rn(rt, it);
  const float gap = p > 0.5f && q > 0.5f ? __fmul_rn(ut, it) - __fmul_rn(us, is) : p - q;
  o.tvd = 0.5f * (d + fabsf(gap));
  const float side = sgn_pq(gap, 0.f);
  o.sigma = fmaf(p, side, g);
  // (a comparison with NaN gives the sign 0: a teacher's NaN is carried on here)
  if (o.t_lse != o.t_lse) o.sigma = o.t_lse;
  return o;
}

}  // namespace top
}  // namespace fct
