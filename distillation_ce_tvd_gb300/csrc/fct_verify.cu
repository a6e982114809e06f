// Verification of drafted tokens: the walk from a request's node 0 along the
// accepted children, and the next token from what is left (the rules are in
// include/fused_ce_tvd.h, fct_spec_verify).
//
// A node needs the log-sum-exp of its target row (and of its draft row, if it
// has children) to turn a few logits into probabilities; a rejection with a
// sibling left needs the mass of the residual r = max(p - S q, 0), and the end
// of the walk a race: the v with the largest r(v) / noise(v), which is
// distributed as r for exponential noise and, unlike the inversion of a
// running sum, needs no order between the elements.  Each is one pass over a
// row, so the bound is the bytes of the rows visited.  Rows of nodes that the
// walk does not reach are not read.
#include <climits>

#include "fct_common.cuh"
#include "fct_internal.h"

namespace fct {

namespace {

constexpr int kVThreads = 512;
constexpr int kVWarps = kVThreads / 32;
constexpr int kVUnroll = 4;  // vectors of a row in flight per thread

// log2-domain state of a row: p(v) = 2^(x_v * k - lse2).
struct RowNorm {
  float lse2;
  bool ok;  // a softmax exists
};

// Largest key and the lowest index that has it.
struct Best {
  float key;
  int v;
};
__device__ __forceinline__ Best best_of(Best a, Best b) {
  return (b.key > a.key || (b.key == a.key && b.v < a.v)) ? b : a;
}
__device__ __forceinline__ Best best_none() { return Best{-INFINITY, INT_MAX}; }

// Folds a vector into a base-2 log-sum-exp state.  Unlike the loss's update
// it takes rows with -inf entries (masked logits): while the state's maximum
// is -inf the exponent offset is 0, so -inf contributes 0 and not NaN.  NaN
// and +inf end in a state that is not finite.
template <int N>
__device__ __forceinline__ void fold(Lse2& st, const float (&x)[N], float k) {
  float vm = x[0];
#pragma unroll
  for (int j = 1; j < N; ++j) vm = fmaxf(vm, x[j]);
  const float m2 = vm * k;
  if (m2 > st.m2) {
    st.s *= ex2(st.m2 - m2);
    st.m2 = m2;
  }
  const float nm = st.m2 == -INFINITY ? 0.f : -st.m2;
  float acc = 0.f;
#pragma unroll
  for (int j = 0; j < N; ++j) acc += ex2(fmaf(x[j], k, nm));
  st.s += acc;
}

// What one CTA does over a request's rows.  T: the logits' element type; VE:
// elements per load (a 16-byte vector, or 1 for rows that are not 16-byte
// aligned).
template <typename T, int VE>
struct Rows {
  int V;
  float* red;  // 2 * kVWarps * 4 floats of shared memory
  int parity = 0;

  // f folded over the warps' values in warp order, for every thread.
  template <typename S, typename F>
  __device__ __forceinline__ S all(S mine, F f) {
    static_assert(sizeof(S) <= 16, "one slot");
    parity ^= 1;
    float* slot = red + parity * kVWarps * 4;
    if ((threadIdx.x & 31) == 0) *reinterpret_cast<S*>(slot + (threadIdx.x >> 5) * 4) = mine;
    __syncthreads();
    S r = *reinterpret_cast<S*>(slot);
#pragma unroll 1
    for (int w = 1; w < kVWarps; ++w) r = f(r, *reinterpret_cast<S*>(slot + w * 4));
    return r;
  }
  __device__ __forceinline__ float all_sum(float x) {
    return all(warp_sum(x), [](float p, float q) { return p + q; });
  }
  __device__ __forceinline__ Best all_best(Best x) {
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1)
      x = best_of(x, Best{__shfl_xor_sync(0xffffffffu, x.key, m),
                          __shfl_xor_sync(0xffffffffu, x.v, m)});
    return all(x, best_of);
  }
  __device__ __forceinline__ RowNorm all_norm(Lse2 st) {
    st = all(warp_merge(st), lse2_merge);
    const float lse2 = st.m2 + log2f(st.s);
    return RowNorm{lse2, lse2 > -INFINITY && lse2 < INFINITY};
  }

  // The thread whose sweep sees element v.
  __device__ __forceinline__ bool owns(int v) const {
    const int nvec = V / VE;
    return (v < nvec * VE ? (v / VE) % kVThreads : v - nvec * VE) == int(threadIdx.x);
  }

  // f(x0, x1, v) for the elements v .. v + n - 1 of a row, or of two at once.
  template <bool kTwo, typename F>
  __device__ __forceinline__ void sweep(const T* r0, const T* r1, F f) const {
    const uint64_t pol = policy_evict_normal();
    const int nvec = V / VE;
    for (int i = threadIdx.x; i < nvec; i += kVThreads * kVUnroll) {
      uint4 w0[kVUnroll], w1[kVUnroll];
#pragma unroll
      for (int u = 0; u < kVUnroll; ++u) {
        const int at = i + u * kVThreads;
        if (at < nvec) {
          w0[u] = load_raw<T, VE>(r0 + int64_t(at) * VE, pol);
          if constexpr (kTwo) w1[u] = load_raw<T, VE>(r1 + int64_t(at) * VE, pol);
        }
      }
#pragma unroll
      for (int u = 0; u < kVUnroll; ++u) {
        const int at = i + u * kVThreads;
        if (at < nvec) {
          float x0[VE], x1[VE];
          unpack_raw<T, VE>(w0[u], x0);
          if constexpr (kTwo) unpack_raw<T, VE>(w1[u], x1);
          f(x0, x1, at * VE);
        }
      }
    }
    // the ragged end, one element per thread
    const int v = nvec * VE + threadIdx.x;
    if (v < V) {
      float x0[1] = {Elem<T>::load1(r0 + v)}, x1[1] = {0.f};
      if constexpr (kTwo) x1[0] = Elem<T>::load1(r1 + v);
      f(x0, x1, v);
    }
  }
};

// Rejected tokens of a node without draft logits that fall to this thread.
// They are few (a node's children) and spread over the threads, so a handful
// per thread is kept; past that `all_of_them` makes the thread look through
// the node's children for every element.
constexpr int kOwn = 4;
struct Rejected {
  int own[kOwn];
  int n;
  __device__ __forceinline__ void add(int v) {
#pragma unroll
    for (int i = 0; i < kOwn; ++i)
      if (i == n) own[i] = v;
    ++n;
  }
};

template <typename T, int VE>
__global__ void __launch_bounds__(kVThreads) verify_kernel(VerifyArgs a) {
  __shared__ __align__(16) float red[2 * kVWarps * 4];
  Rows<T, VE> rows{static_cast<int>(a.V), red};
  const int V = static_cast<int>(a.V);
  const int64_t b = blockIdx.x;
  const int lane = threadIdx.x & 31;
  int64_t first = a.node_start[b], end = a.node_start[b + 1];
  int32_t status = 0;
  if (first < 0 || end > a.n_nodes || end < first) {
    status |= FCT_DEV_INDEX_OUT_OF_RANGE;
    end = first = 0;
  }
  const float temp = a.temperature ? a.temperature[b] : 1.f;
  const bool greedy = !(temp > 0.f);
  const float k = greedy ? kLog2e : kLog2e / temp;
  const float* noise = a.noise + b * a.ld_noise;
  int64_t* toks = a.out_tokens + b * (a.max_depth + 1);
  int32_t* path = a.path + b * a.max_depth;

  // The first child of `at` after node c, or -1 (nodes as rows of the batch).
  // Every warp looks for itself and gets the same answer.
  auto next_child = [&](int64_t at, int64_t c) -> int64_t {
    for (int64_t c0 = c + 1; c0 < end; c0 += 32) {
      const int64_t i = c0 + lane;
      const bool is = i < end && a.parent[i] >= 0 && first + a.parent[i] == at;
      const unsigned hit = __ballot_sync(0xffffffffu, is);
      if (hit) return c0 + __ffs(hit) - 1;
    }
    return -1;
  };
  // Whether a child of `at` before node c has token v (any thread by itself).
  auto among = [&](int64_t at, int64_t c, int64_t v) {
    for (int64_t e = at + 1; e < c; ++e)
      if (a.parent[e] >= 0 && first + a.parent[e] == at && a.tokens[e] == v) return true;
    return false;
  };

  int64_t at = first, depth = 0, last = -1;
  for (bool walking = end > first; walking;) {
    const T* tr = static_cast<const T*>(a.target) + at * a.ld_t;
    int64_t c = depth < a.max_depth ? next_child(at, at) : -1;
    int64_t accepted = -1;
    if (greedy) {
      Best best = best_none();
      bool bad = false;
      rows.template sweep<false>(tr, nullptr, [&](auto& x, auto&, int v) {
#pragma unroll
        for (int j = 0; j < int(sizeof(x) / sizeof(float)); ++j) {
          bad |= !(x[j] < INFINITY);
          if (x[j] > best.key) best = Best{x[j], v + j};
        }
      });
      best = rows.all_best(bad ? Best{INFINITY, -1} : best);
      if (best.v < 0 || best.v >= V) {
        status |= FCT_DEV_NO_DISTRIBUTION;
        break;
      }
      for (; c >= 0 && accepted < 0; c = next_child(at, c)) {
        if (a.tokens[c] < 0 || a.tokens[c] >= V) status |= FCT_DEV_TARGET_OUT_OF_RANGE;
        if (a.tokens[c] == best.v) accepted = c;
      }
      last = best.v;
    } else {
      const T* dr = a.draft && c >= 0 ? static_cast<const T*>(a.draft) + at * a.ld_d : nullptr;
      Lse2 sp = lse2_empty(), sq = lse2_empty();
      RowNorm p, q{0.f, true};
      if (dr) {
        rows.template sweep<true>(tr, dr, [&](auto& x, auto& y, int) {
          fold(sp, x, k);
          fold(sq, y, k);
        });
        q = rows.all_norm(sq);
      } else {
        rows.template sweep<false>(tr, nullptr, [&](auto& x, auto&, int) { fold(sp, x, k); });
      }
      p = rows.all_norm(sp);
      if (!p.ok || !q.ok) {
        status |= FCT_DEV_NO_DISTRIBUTION;
        break;
      }
      auto prob = [&](float x, RowNorm n) { return ex2(fmaf(x, k, -n.lse2)); };
      float S = 0.f, Z = 1.f;
      Rejected rej;
      rej.n = 0;
      int64_t tried = at;  // children up to this node have been rejected
      // r(v) of a vector, from the rows' values
      auto residual = [&](auto& x, auto& y, int v) {
        constexpr int n = int(sizeof(x) / sizeof(float));
#pragma unroll
        for (int j = 0; j < n; ++j) {
          x[j] = prob(x[j], p);
          if (dr) x[j] = fmaxf(fmaf(-S, prob(y[j], q), x[j]), 0.f);
        }
        if (rej.n > 0) {
#pragma unroll
          for (int j = 0; j < n; ++j) {
            bool out = rej.n > kOwn && among(at, tried + 1, v + j);
#pragma unroll
            for (int i = 0; i < kOwn; ++i) out |= i < rej.n && rej.own[i] == v + j;
            if (out) x[j] = 0.f;
          }
        }
      };
      while (c >= 0) {
        const int64_t x = a.tokens[c];
        if (x < 0 || x >= V) {
          status |= FCT_DEV_TARGET_OUT_OF_RANGE;
        } else {
          const float px = prob(Elem<T>::load1(tr + x), p);
          float rx, qx = 1.f;
          if (dr) {
            qx = prob(Elem<T>::load1(dr + x), q);
            rx = fmaxf(fmaf(-S, qx, px), 0.f);
          } else {
            rx = among(at, c, x) ? 0.f : px;
          }
          if (a.uniform[c] * Z * qx < rx) {
            accepted = c;
            break;
          }
          if (!dr && rows.owns(static_cast<int>(x))) rej.add(static_cast<int>(x));
        }
        // with draft logits a token outside the vocabulary has p = q = 0 and
        // still counts as one draw from q
        S += Z;
        tried = c;
        c = next_child(at, c);
        if (c >= 0) {  // another sibling: the mass that is left
          float z = 0.f;
          auto add = [&](auto& x, auto& y, int v) {
            residual(x, y, v);
#pragma unroll
            for (int j = 0; j < int(sizeof(x) / sizeof(float)); ++j) z += x[j];
          };
          if (dr)
            rows.template sweep<true>(tr, dr, add);
          else
            rows.template sweep<false>(tr, nullptr, add);
          Z = rows.all_sum(z);
        }
      }
      if (accepted < 0) {
        for (int round = 0; round < 2; ++round) {
          Best best = best_none();
          auto run = [&](auto& x, auto& y, int v) {
            residual(x, y, v);
#pragma unroll
            for (int j = 0; j < int(sizeof(x) / sizeof(float)); ++j) {
              const float key = __fdividef(x[j], noise[v + j]);
              if (x[j] > 0.f && key > best.key) best = Best{key, v + j};
            }
          };
          if (dr && S > 0.f)
            rows.template sweep<true>(tr, dr, run);
          else
            rows.template sweep<false>(tr, nullptr, run);
          best = rows.all_best(best);
          last = best.v;
          if (best.v < V) break;
          // nothing is left of p: it takes its own place
          S = 0.f;
          rej.n = 0;
          dr = nullptr;
        }
        if (last >= V) last = -1;
      }
    }
    walking = accepted >= 0;
    if (walking) {
      if (threadIdx.x == 0) {
        toks[depth] = a.tokens[accepted];
        path[depth] = static_cast<int32_t>(accepted - first);
      }
      ++depth;
      at = accepted;
      last = -1;
    }
  }
  if (threadIdx.x == 0) {
    toks[depth] = last;
    a.count[b] = static_cast<int32_t>(depth);
    if (status && a.dev_status) atomicOr(a.dev_status, status);
  }
  for (int64_t i = depth + threadIdx.x; i < a.max_depth; i += kVThreads) {
    toks[i + 1] = -1;
    path[i] = -1;
  }
}

template <typename T>
cudaError_t launch_typed(const VerifyArgs& a, cudaStream_t st) {
  auto rows16 = [&](const void* p, int64_t ld) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (size_t(ld) * sizeof(T)) % 16 == 0;
  };
  const unsigned n = static_cast<unsigned>(a.batch);
  if (rows16(a.target, a.ld_t) && (a.draft == nullptr || rows16(a.draft, a.ld_d)))
    verify_kernel<T, Elem<T>::kVec><<<n, kVThreads, 0, st>>>(a);
  else
    verify_kernel<T, 1><<<n, kVThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, int, int, cudaStream_t st) {
  return a.dtype == FCT_F32 ? launch_typed<float>(a, st) : launch_typed<bf16_t>(a, st);
}

}  // namespace fct
