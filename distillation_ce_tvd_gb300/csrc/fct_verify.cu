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
#include <cstring>
#include <mutex>

#include "fct_common.cuh"
#include "fct_internal.h"

namespace fct {

namespace {

constexpr int kVThreads = 256;
constexpr int kVWarps = kVThreads / 32;
constexpr int kVUnroll = 4;  // vectors of a row in flight per thread
constexpr int kMaxCtas = 16; // CTAs of a request's cluster
constexpr int kCtasPerSm = 2;

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

// States that reductions combine; 16 bytes at most.
struct NormPair {
  Lse2 p, q;
};
// As lse2_merge, but the NaN of a state that saw nothing else (its maximum is
// still -inf) is kept.
__device__ __forceinline__ Lse2 merge_norm(Lse2 a, Lse2 b) {
  const float m = fmaxf(a.m2, b.m2), base = m == -INFINITY ? 0.f : m;
  return Lse2{m, a.s * ex2(a.m2 - base) + b.s * ex2(b.m2 - base)};
}
__device__ __forceinline__ NormPair merge_pair(NormPair a, NormPair b) {
  return NormPair{merge_norm(a.p, b.p), merge_norm(a.q, b.q)};
}
__device__ __forceinline__ float add(float a, float b) { return a + b; }

template <typename S>
__device__ __forceinline__ S shuffle_xor(S x, int m) {
  constexpr int kWords = sizeof(S) / 4;
  uint32_t w[kWords];
  memcpy(w, &x, sizeof(S));
#pragma unroll
  for (int i = 0; i < kWords; ++i) w[i] = __shfl_xor_sync(0xffffffffu, w[i], m);
  memcpy(&x, w, sizeof(S));
  return x;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
               "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Reduction slots: per warp of this CTA, and per CTA of the cluster; two of
// each, used in turn, so that one barrier per reduction is enough.
struct Slots {
  uint4 warp[2][kVWarps];
  uint4 cta[2][kMaxCtas];
};

// What a cluster does over a request's rows: CTA `rank` of `ctas` holds the
// vectors [begin, end) of every row (and the last one the ragged end).  T: the
// logits' element type; VE: elements per load (a 16-byte vector, or 1 for rows
// that are not 16-byte aligned).
template <typename T, int VE>
struct Rows {
  int V, begin, end;
  int rank, ctas;
  Slots* slots;
  int parity = 0;

  // f (commutative) folded over every thread of the cluster, for every thread
  // of it.  Butterflies over lanes, then warps, then CTAs: the order does not
  // depend on timing, and all threads get the same bits.
  template <typename S, typename F>
  __device__ __forceinline__ S all(S x, S none, F f) {
    static_assert(sizeof(S) <= 16, "one slot");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    parity ^= 1;
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) x = f(x, shuffle_xor(x, m));
    if (lane == 0) memcpy(&slots->warp[parity][warp], &x, sizeof(S));
    __syncthreads();
    x = none;
    if (lane < kVWarps) memcpy(&x, &slots->warp[parity][lane], sizeof(S));
#pragma unroll
    for (int m = kVWarps / 2; m >= 1; m >>= 1) x = f(x, shuffle_xor(x, m));
    x = broadcast(x);  // lanes from kVWarps on have folded `none` only
    if (ctas > 1) {
      if (warp == 0 && lane < ctas) {
        uint32_t w[4] = {0, 0, 0, 0}, dst;
        memcpy(w, &x, sizeof(S));
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                     : "=r"(dst)
                     : "r"(smem_addr(&slots->cta[parity][rank])), "r"(lane));
        asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(w[0]),
                     "r"(w[1]), "r"(w[2]), "r"(w[3])
                     : "memory");
      }
      __syncwarp();
      cluster_barrier();
      x = none;
      if (lane < ctas) memcpy(&x, &slots->cta[parity][lane], sizeof(S));
#pragma unroll
      for (int m = kMaxCtas / 2; m >= 1; m >>= 1) x = f(x, shuffle_xor(x, m));
      x = broadcast(x);
    }
    return x;
  }
  template <typename S>
  __device__ __forceinline__ static S broadcast(S x) {
    constexpr int kWords = sizeof(S) / 4;
    uint32_t w[kWords];
    memcpy(w, &x, sizeof(S));
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = __shfl_sync(0xffffffffu, w[i], 0);
    memcpy(&x, w, sizeof(S));
    return x;
  }
  __device__ __forceinline__ float all_sum(float x) { return all(x, 0.f, add); }
  __device__ __forceinline__ Best all_best(Best x) { return all(x, best_none(), best_of); }
  __device__ __forceinline__ static RowNorm norm(Lse2 st) {
    const float lse2 = st.m2 + log2f(st.s);
    return RowNorm{lse2, lse2 > -INFINITY && lse2 < INFINITY};
  }

  // The thread of the cluster whose sweep sees element v.
  __device__ __forceinline__ bool owns(int v) const {
    const int i = v / VE, tail = V / VE * VE;
    if (v >= tail) return rank == ctas - 1 && v - tail == int(threadIdx.x);
    return i >= begin && i < end && (i - begin) % kVThreads == int(threadIdx.x);
  }

  // f(x0, x1, e, v) for the elements v .. v + n - 1 of up to three rows: r0,
  // r1 (kTwo) and fp32 values r2 (kNoise).
  template <bool kTwo, bool kNoise, typename F>
  __device__ __forceinline__ void sweep(const T* r0, const T* r1, const float* r2, F f) const {
    constexpr int kFloat4 = VE >= 4 ? VE / 4 : 1;
    constexpr int kUnroll = kNoise ? 2 : kVUnroll;
    const uint64_t pol = policy_evict_normal();
    for (int i = begin + threadIdx.x; i < end; i += kVThreads * kUnroll) {
      uint4 w0[kUnroll], w1[kUnroll], w2[kUnroll][kFloat4];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int at = i + u * kVThreads;
        if (at < end) {
          w0[u] = load_raw<T, VE>(r0 + int64_t(at) * VE, pol);
          if constexpr (kTwo) w1[u] = load_raw<T, VE>(r1 + int64_t(at) * VE, pol);
          if constexpr (kNoise) {
#pragma unroll
            for (int j = 0; j < kFloat4; ++j) {
              if constexpr (VE >= 4)
                w2[u][j] = ld16(r2 + int64_t(at) * VE + 4 * j, pol);
              else
                w2[u][j].x = __float_as_uint(r2[at]);
            }
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int at = i + u * kVThreads;
        if (at < end) {
          float x0[VE], x1[VE], e[VE];
          unpack_raw<T, VE>(w0[u], x0);
          if constexpr (kTwo) unpack_raw<T, VE>(w1[u], x1);
          if constexpr (kNoise) {
#pragma unroll
            for (int j = 0; j < VE; ++j) {
              const uint4 q = w2[u][VE >= 4 ? j / 4 : 0];
              e[j] = __uint_as_float(j % 4 == 0 ? q.x : j % 4 == 1 ? q.y : j % 4 == 2 ? q.z : q.w);
            }
          }
          f(x0, x1, e, at * VE);
        }
      }
    }
    // the ragged end, one element per thread
    const int v = V / VE * VE + threadIdx.x;
    if (rank == ctas - 1 && v < V) {
      float x0[1] = {Elem<T>::load1(r0 + v)}, x1[1] = {0.f}, e[1] = {0.f};
      if constexpr (kTwo) x1[0] = Elem<T>::load1(r1 + v);
      if constexpr (kNoise) e[0] = r2[v];
      f(x0, x1, e, v);
    }
  }
};

// Rejected tokens of a node without draft logits that fall to this thread.
// They are few (a node's children) and spread over the threads, so a handful
// per thread is kept; with more, the thread looks through the node's children
// for every element.
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

// A request's nodes as the walk needs them, read once (trees larger than
// kNodeCap are looked up where they are).
constexpr int kNodeCap = 256;
struct Nodes {
  int64_t tokens[kNodeCap];
  int32_t parent[kNodeCap];
  float uniform[kNodeCap];
};

// One cluster per request: kCtas CTAs share its rows (1, or a power of two up
// to kMaxCtas).
template <typename T, int VE>
__global__ void __launch_bounds__(kVThreads, kCtasPerSm) verify_kernel(const __grid_constant__ VerifyArgs a) {
  __shared__ Slots slots;
  __shared__ Nodes held;
  const int V = static_cast<int>(a.V);
  const int ctas = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
  const int nvec = V / VE, share = (nvec + ctas - 1) / ctas;
  Rows<T, VE> rows{V, min(rank * share, nvec), min((rank + 1) * share, nvec), rank, ctas, &slots};
  const int64_t b = blockIdx.x / ctas;
  const int lane = threadIdx.x & 31;
  const bool writer = rank == 0 && threadIdx.x == 0;
  int64_t first = a.node_start[b];
  int64_t n64 = a.node_start[b + 1] - first;
  int32_t status = 0;
  if (first < 0 || n64 < 0 || first + n64 > a.n_nodes) {
    status |= FCT_DEV_INDEX_OUT_OF_RANGE;
    first = n64 = 0;
  }
  const int nodes = static_cast<int>(n64);  // node indexes below are the request's
  for (int i = threadIdx.x; i < nodes && i < kNodeCap; i += kVThreads) {
    held.tokens[i] = a.tokens[first + i];
    held.parent[i] = a.parent[first + i];
    held.uniform[i] = a.uniform[first + i];
  }
  const float temp = a.temperature ? a.temperature[b] : 1.f;
  const bool greedy = !(temp > 0.f);
  const float k = greedy ? kLog2e : kLog2e / temp;
  const float* noise = a.noise + b * a.ld_noise;
  int64_t* toks = a.out_tokens + b * (a.max_depth + 1);
  int32_t* path = a.path + b * a.max_depth;
  // `held` is filled, and every CTA of the cluster runs: its shared memory may
  // be written from now on.  (The last reduction's barrier comes after all
  // such writes, so a CTA may also leave when it is done.)
  cluster_barrier();
  auto token = [&](int i) { return i < kNodeCap ? held.tokens[i] : a.tokens[first + i]; };
  auto parent = [&](int i) { return i < kNodeCap ? held.parent[i] : a.parent[first + i]; };
  auto uniform = [&](int i) { return i < kNodeCap ? held.uniform[i] : a.uniform[first + i]; };

  // The first child of `at` after node c, or -1.  Every warp looks for itself
  // and gets the same answer.
  auto next_child = [&](int at, int c) {
    for (int c0 = c + 1; c0 < nodes; c0 += 32) {
      const int i = c0 + lane;
      const unsigned hit = __ballot_sync(0xffffffffu, i < nodes && parent(i) == at);
      if (hit) return c0 + __ffs(hit) - 1;
    }
    return -1;
  };
  // Whether a child of `at` before node c has token v (any thread by itself).
  auto among = [&](int at, int c, int64_t v) {
    for (int e = at + 1; e < c; ++e)
      if (parent(e) == at && token(e) == v) return true;
    return false;
  };

  int at = 0;
  int64_t depth = 0, last = -1;
  for (bool walking = nodes > 0; walking;) {
    const T* tr = static_cast<const T*>(a.target) + (first + at) * a.ld_t;
    int c = depth < a.max_depth ? next_child(at, at) : -1;
    int accepted = -1;
    if (greedy) {
      Best best = best_none();
      bool bad = false;
      rows.template sweep<false, false>(tr, nullptr, nullptr, [&](auto& x, auto&, auto&, int v) {
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
        if (token(c) < 0 || token(c) >= V) status |= FCT_DEV_TARGET_OUT_OF_RANGE;
        if (token(c) == best.v) accepted = c;
      }
      last = best.v;
    } else if (c < 0) {
      // no child to test: r = p, and the race needs p up to a factor only, so
      // one pass does, on log2 of p(v) / noise(v)
      Best best = best_none();
      bool bad = false;
      rows.template sweep<false, true>(tr, nullptr, noise, [&](auto& x, auto&, auto& e, int v) {
#pragma unroll
        for (int j = 0; j < int(sizeof(x) / sizeof(float)); ++j) {
          bad |= !(x[j] < INFINITY);
          const float key = fmaf(x[j], k, -__log2f(e[j]));
          if (key > best.key) best = Best{key, v + j};
        }
      });
      best = rows.all_best(bad ? Best{INFINITY, -1} : best);
      if (best.v < 0 || best.v >= V)
        status |= FCT_DEV_NO_DISTRIBUTION;
      else
        last = best.v;
    } else {
      const T* dr = a.draft ? static_cast<const T*>(a.draft) + (first + at) * a.ld_d : nullptr;
      // the first child's logits, on their way while the rows are read
      const int64_t x0 = token(c);
      const bool in0 = x0 >= 0 && x0 < V;
      const float tx0 = in0 ? Elem<T>::load1(tr + x0) : 0.f;
      const float dx0 = in0 && dr ? Elem<T>::load1(dr + x0) : 0.f;
      NormPair st{lse2_empty(), lse2_empty()};
      if (dr)
        rows.template sweep<true, false>(tr, dr, nullptr, [&](auto& x, auto& y, auto&, int) {
          fold(st.p, x, k);
          fold(st.q, y, k);
        });
      else
        rows.template sweep<false, false>(tr, nullptr, nullptr,
                                          [&](auto& x, auto&, auto&, int) { fold(st.p, x, k); });
      st = rows.all(st, NormPair{lse2_empty(), lse2_empty()}, merge_pair);
      const RowNorm p = rows.norm(st.p), q = dr ? rows.norm(st.q) : RowNorm{0.f, true};
      if (!p.ok || !q.ok) {
        status |= FCT_DEV_NO_DISTRIBUTION;
        break;
      }
      auto prob = [&](float x, RowNorm n) { return ex2(fmaf(x, k, -n.lse2)); };
      float S = 0.f, Z = 1.f;
      Rejected rej;
      rej.n = 0;
      int tried = at;  // children up to this node have been rejected
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
      for (bool again = false; c >= 0; again = true) {
        const int64_t x = token(c);
        if (x < 0 || x >= V) {
          status |= FCT_DEV_TARGET_OUT_OF_RANGE;
        } else {
          const float px = prob(again ? Elem<T>::load1(tr + x) : tx0, p);
          float rx, qx = 1.f;
          if (dr) {
            qx = prob(again ? Elem<T>::load1(dr + x) : dx0, q);
            rx = fmaxf(fmaf(-S, qx, px), 0.f);
          } else {
            rx = again && among(at, c, x) ? 0.f : px;
          }
          if (uniform(c) * Z * qx < rx) {
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
          auto sum = [&](auto& x, auto& y, auto&, int v) {
            residual(x, y, v);
#pragma unroll
            for (int j = 0; j < int(sizeof(x) / sizeof(float)); ++j) z += x[j];
          };
          if (dr)
            rows.template sweep<true, false>(tr, dr, nullptr, sum);
          else
            rows.template sweep<false, false>(tr, nullptr, nullptr, sum);
          Z = rows.all_sum(z);
        }
      }
      if (accepted < 0) {
        for (int round = 0; round < 2; ++round) {
          Best best = best_none();
          auto run = [&](auto& x, auto& y, auto& e, int v) {
            residual(x, y, v);
#pragma unroll
            for (int j = 0; j < int(sizeof(x) / sizeof(float)); ++j) {
              const float key = __fdividef(x[j], e[j]);
              if (x[j] > 0.f && key > best.key) best = Best{key, v + j};
            }
          };
          if (dr)
            rows.template sweep<true, true>(tr, dr, noise, run);
          else
            rows.template sweep<false, true>(tr, nullptr, noise, run);
          best = rows.all_best(best);
          last = best.v < V ? best.v : -1;
          if (last >= 0) break;
          // nothing is left of p: it takes its own place
          rej.n = 0;
          dr = nullptr;
        }
      }
    }
    walking = accepted >= 0;
    if (walking) {
      if (writer) {
        toks[depth] = token(accepted);
        path[depth] = accepted;
      }
      ++depth;
      at = accepted;
      last = -1;
    }
  }
  if (writer) {
    toks[depth] = last;
    a.count[b] = static_cast<int32_t>(depth);
    if (status && a.dev_status) atomicOr(a.dev_status, status);
  }
  if (rank == 0)
    for (int64_t i = depth + threadIdx.x; i < a.max_depth; i += kVThreads) {
      toks[i + 1] = -1;
      path[i] = -1;
    }
}

template <typename T, int VE>
cudaError_t launch_rows(const VerifyArgs& a, int sms, int device, cudaStream_t st) {
  static std::once_flag once[64];
  static cudaError_t ready[64];
  auto kernel = verify_kernel<T, VE>;
  if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
  std::call_once(once[device], [&] {
    ready[device] = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  });
  if (ready[device] != cudaSuccess) return ready[device];
  int ctas = 1;
  while (ctas < kMaxCtas && a.batch * ctas * 2 <= int64_t(sms) * kCtasPerSm) ctas *= 2;
  if (a.batch * ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.batch * ctas));
  cfg.blockDim = dim3(kVThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <typename T>
cudaError_t launch_typed(const VerifyArgs& a, int sms, int device, cudaStream_t st) {
  auto rows16 = [&](const void* p, int64_t ld, size_t e) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (size_t(ld) * e) % 16 == 0;
  };
  const bool vec = rows16(a.target, a.ld_t, sizeof(T)) && rows16(a.noise, a.ld_noise, 4) &&
                   (a.draft == nullptr || rows16(a.draft, a.ld_d, sizeof(T)));
  return vec ? launch_rows<T, Elem<T>::kVec>(a, sms, device, st)
             : launch_rows<T, 1>(a, sms, device, st);
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, int sms, int device, cudaStream_t st) {
  return a.dtype == FCT_F32 ? launch_typed<float>(a, sms, device, st)
                            : launch_typed<bf16_t>(a, sms, device, st);
}

}  // namespace fct
