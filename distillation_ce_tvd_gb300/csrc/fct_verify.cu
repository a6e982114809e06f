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
//
// The nodes follow one another, so what a request costs is mostly latency: at
// 64 requests of 7 drafted tokens and V = 151936 bf16 (93 us, 197 MB expected)
// a node takes 6 us on its four CTAs, 3 of them the sweep of the rows, 1.1 the
// reduction over the cluster, the rest the decision and the next row's copies.
// One request of 4 drafted tokens at V = 32000 fp32 takes 16 us, 24 trees of 32
// nodes 40 us.  Rows read straight from global memory, not staged,
// took 171, 19 and 75 us; one CTA per request 303, 50 and 177.
#include <climits>
#include <cstring>
#include <mutex>

#include "fct_common.cuh"
#include "fct_internal.h"

namespace fct {

namespace {

constexpr int kVThreads = 512;
constexpr int kVWarps = kVThreads / 32;
constexpr int kVUnroll = 4;   // vectors of a row in flight per thread
constexpr int kMaxCtas = 16;  // CTAs of a request's cluster
// Staged rows: buffers for up to kMaxBufs nodes, each a CTA's share of a
// target and a draft row, filled in kChunks pieces.
constexpr int kMaxBufs = 4;
constexpr int kChunks = 4;
constexpr int kStageBytes = 216 * 1024;

// A row's softmax: p(v) = 2^(x_v * k - m2) * inv, with m2 the largest x_v * k and
// inv = 1 / sum_v 2^(x_v * k - m2).  Kept apart: the exponent's rounding is then
// that of the distance from the maximum.  In one number, m2 + log2(sum), it is
// that of the logits themselves, and a constant added to a row, or a low
// temperature, costs bits of every probability (1024 at T = 1: 4e-5).
struct RowNorm {
  float m2, inv;
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

// Best in a race whose keys are log2 of p(v) / noise(v), p up to a factor: x_v is
// taken relative to `top`, the largest x seen (by the thread, then by all), so
// that a key's rounding is that of a distance from it, not of the logit.
struct Race {
  float key;
  int v;
  float top;
};
__device__ __forceinline__ Race race_none() { return Race{-INFINITY, INT_MAX, -INFINITY}; }
// `top` raised to the larger t: the key, if there is one, goes down by what
// that is.
__device__ __forceinline__ void raise(Race& r, float t, float k) {
  if (r.v >= 0 && r.v < INT_MAX) r.key = fmaf(r.top - t, k, r.key);
  r.top = t;
}

// Folds a vector into a base-2 log-sum-exp state.  Unlike the loss's update
// it takes rows with -inf entries (masked logits): while the state's maximum
// is -inf the exponent offset is 0, so -inf contributes 0 and not NaN.  NaN
// and +inf end in a state that is not finite.
template <int N>
__device__ __forceinline__ void fold(Lse2x& st, const float (&x)[N], float k) {
  const float m2 = vec_max(x) * k;
  if (m2 > st.m2) {
    const float sc = ex2(st.m2 - m2);
    st.s.x *= sc;
    st.s.y *= sc;
    st.m2 = m2;
  }
  const float nm = st.m2 == -INFINITY ? 0.f : -st.m2;
  if constexpr (N % 2 == 0) {
    const float2 k2 = make_float2(k, k), n2 = make_float2(nm, nm);
#pragma unroll
    for (int j = 0; j < N; j += 2) {
      const float2 e = __ffma2_rn(make_float2(x[j], x[j + 1]), k2, n2);
      st.s = __fadd2_rn(st.s, make_float2(ex2(e.x), ex2(e.y)));
    }
  } else {
    st.s.x += ex2(fmaf(x[0], k, nm));
  }
}

// States that reductions combine; 16 bytes at most.
struct NormPair {
  Lse2 p, q;
};
// Both states folded over `width` (a power of two) neighbouring lanes: the
// maxima first, then each sum rescaled once.  The NaN of a state that saw
// nothing else (its maximum is still -inf) is kept.
struct FoldNorms {
  __device__ __forceinline__ NormPair operator()(NormPair x, int width) const {
    float mp = x.p.m2, mq = x.q.m2;
    for (int m = width / 2; m >= 1; m >>= 1) {
      mp = fmaxf(mp, __shfl_xor_sync(0xffffffffu, mp, m));
      mq = fmaxf(mq, __shfl_xor_sync(0xffffffffu, mq, m));
    }
    float sp = x.p.s * ex2(x.p.m2 - (mp == -INFINITY ? 0.f : mp));
    float sq = x.q.s * ex2(x.q.m2 - (mq == -INFINITY ? 0.f : mq));
    for (int m = width / 2; m >= 1; m >>= 1) {
      sp += __shfl_xor_sync(0xffffffffu, sp, m);
      sq += __shfl_xor_sync(0xffffffffu, sq, m);
    }
    return NormPair{Lse2{mp, sp}, Lse2{mq, sq}};
  }
};
struct FoldSum {
  __device__ __forceinline__ float operator()(float x, int width) const {
    for (int m = width / 2; m >= 1; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
  }
};
struct FoldBest {
  __device__ __forceinline__ Best operator()(Best x, int width) const {
    for (int m = width / 2; m >= 1; m >>= 1)
      x = best_of(x, Best{__shfl_xor_sync(0xffffffffu, x.key, m), __shfl_xor_sync(0xffffffffu, x.v, m)});
    return x;
  }
};

struct FoldRace {
  float k;
  __device__ __forceinline__ Race operator()(Race x, int width) const {
    float top = x.top;
    for (int m = width / 2; m >= 1; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
    if (x.top < top) raise(x, top, k);
    const Best best = FoldBest()(Best{x.key, x.v}, width);
    return Race{best.key, best.v, top};
  }
};

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

// Reduction slots: per warp of this CTA, and per CTA of the cluster, filled
// by the CTAs with stores that complete on `bar`.  Two of each, used in turn:
// a CTA sends for the next reduction but one only after it has received for
// the next one from every CTA, and those sent after they had read this one's.
struct Slots {
  uint4 warp[2][kVWarps];
  uint4 cta[2][kMaxCtas];
  uint64_t bar[2];
};

// The staged rows of a CTA: which pieces have landed.
struct Stage {
  uint64_t bar[kMaxBufs][kChunks];
  int abort;
};

// What a cluster does over a request's rows: CTA `rank` of `ctas` holds the
// vectors [begin, end) of every row (and the last one the ragged end).  T: the
// logits' element type; VE: elements per load (a 16-byte vector, or 1 for rows
// that are not 16-byte aligned).  kStaged: rows are swept from shared memory,
// where bulk copies put the CTA's share (the ragged end stays where it is),
// else from global memory.
template <typename T, int VE, bool kStaged>
struct Rows {
  int V, begin, end;
  int rank, ctas;
  Slots* slots;
  uint32_t reductions = 0;
  // staged: pieces of the share and vectors per piece, and the current node's
  // rows from vector `begin` on with the barriers their pieces land on
  int pieces = 1, piece = 0;
  uint64_t* bar = nullptr;
  uint32_t bar_parity = 0;
  int* abort = nullptr;
  const T* t_share = nullptr;
  const T* d_share = nullptr;

  // The fold of every thread's x over the cluster, for every thread of it.
  // Butterflies over lanes, then (in warp 0) warps, then CTAs: the order does
  // not depend on timing, and all threads get the same bits.
  template <typename S, typename F>
  __device__ __forceinline__ S all(S x, S none, F fold) {
    static_assert(sizeof(S) <= 16, "one slot");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int turn = reductions & 1;
    uint64_t* bar = &slots->bar[turn];
    x = fold(x, 32);
    if (lane == 0) memcpy(&slots->warp[turn][warp], &x, sizeof(S));
    __syncthreads();
    if (warp == 0) {
      if (lane == 0) mbar_arrive_expect_tx(bar, uint32_t(ctas) * 16);
      x = none;
      if (lane < kVWarps) memcpy(&x, &slots->warp[turn][lane], sizeof(S));
      x = broadcast(fold(x, kVWarps));  // lanes from kVWarps on have folded `none` only
      if (lane < ctas) {
        uint32_t w[4] = {0, 0, 0, 0};
        memcpy(w, &x, sizeof(S));
        asm volatile(
            "{\n\t.reg .b32 dst, bar;\n\t"
            "mapa.shared::cluster.u32 dst, %0, %2;\n\t"
            "mapa.shared::cluster.u32 bar, %1, %2;\n\t"
            "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [dst], {%3, %4, %5, %6}, "
            "[bar];\n\t}" ::"r"(smem_addr(&slots->cta[turn][rank])),
            "r"(smem_addr(bar)), "r"(lane), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
            : "memory");
      }
      __syncwarp();
    }
    if (lane == 0) mbar_wait(bar, (reductions >> 1) & 1u, abort, false);
    __syncwarp();
    ++reductions;
    x = none;
    if (lane < ctas) memcpy(&x, &slots->cta[turn][lane], sizeof(S));
    return broadcast(fold(x, ctas));
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
  __device__ __forceinline__ float all_sum(float x) { return all(x, 0.f, FoldSum()); }
  __device__ __forceinline__ Best all_best(Best x) { return all(x, best_none(), FoldBest()); }
  __device__ __forceinline__ static RowNorm norm(Lse2 st) {
    const bool ok = st.m2 > -INFINITY && st.m2 < INFINITY && st.s > 0.f && st.s < INFINITY;
    return RowNorm{st.m2, 1.f / st.s, ok};
  }

  // The thread of the cluster whose sweep sees element v.
  __device__ __forceinline__ bool owns(int v) const {
    const int i = v / VE, tail = V / VE * VE;
    if (v >= tail) return rank == ctas - 1 && v - tail == int(threadIdx.x);
    if (i < begin || i >= end) return false;
    const int in_piece = kStaged ? (i - begin) % piece : i - begin;
    return in_piece % kVThreads == int(threadIdx.x);
  }

  // f(x0, x1, e, v) for the elements v .. v + n - 1 of up to three rows: r0,
  // r1 (kTwo) and fp32 values r2 (kNoise).  r0 and r1 are the node's rows;
  // `fresh`: the first sweep of a staged node, which waits for its pieces.
  template <bool kTwo, bool kNoise, int kUnroll, typename F>
  __device__ __forceinline__ void sweep(const T* r0, const T* r1, const float* r2, bool fresh,
                                        F f) const {
    constexpr int kFloat4 = VE >= 4 ? VE / 4 : 1;
    const uint64_t pol = policy_evict_normal();
    for (int c = 0; c < (kStaged ? pieces : 1); ++c) {
      const int from = kStaged ? min(begin + c * piece, end) : begin;
      const int to = kStaged ? min(from + piece, end) : end;
      if (kStaged && fresh && from < to) {
        if ((threadIdx.x & 31) == 0) mbar_wait(&bar[c], bar_parity, abort, false);
        __syncwarp();
      }
      for (int i = from + threadIdx.x; i < to; i += kVThreads * kUnroll) {
        uint4 w0[kUnroll], w1[kUnroll], w2[kUnroll][kFloat4];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          const int at = i + u * kVThreads;
          if (at < to) {
            if constexpr (kNoise) {
#pragma unroll
              for (int j = 0; j < kFloat4; ++j) {
                if constexpr (VE >= 4)
                  w2[u][j] = ld16(r2 + int64_t(at) * VE + 4 * j, pol);
                else
                  w2[u][j].x = __float_as_uint(r2[at]);
              }
            }
            if constexpr (kStaged) {
              w0[u] = *reinterpret_cast<const uint4*>(t_share + (at - begin) * VE);
              if constexpr (kTwo) w1[u] = *reinterpret_cast<const uint4*>(d_share + (at - begin) * VE);
            } else {
              w0[u] = load_raw<T, VE>(r0 + int64_t(at) * VE, pol);
              if constexpr (kTwo) w1[u] = load_raw<T, VE>(r1 + int64_t(at) * VE, pol);
            }
          }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          const int at = i + u * kVThreads;
          if (at < to) {
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
  int32_t child[kNodeCap];    // the first one, INT_MAX if none
  int32_t sibling[kNodeCap];  // the next one, -1 if none
};

__device__ __forceinline__ void bulk_copy(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_addr(dst)),
      "l"(src), "r"(bytes), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void bulk_prefetch(const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}

// One cluster per request, whose CTAs share its rows (1, or a power of two up
// to kMaxCtas).  kStaged: the walk's likely next nodes, each the first child
// of the one before, are copied to shared memory ahead of it, as far as `bufs`
// buffers of buf_bytes reach, and a node's later passes read them there.
template <typename T, int VE, bool kStaged>
__global__ void __launch_bounds__(kVThreads, 1)
    verify_kernel(const __grid_constant__ VerifyArgs a, int bufs, int buf_bytes) {
  constexpr int kUnroll = kStaged ? 1 : kVUnroll;       // vectors in flight per thread
  constexpr int kNoiseUnroll = 4;
  extern __shared__ __align__(128) uint8_t stage_smem[];
  __shared__ Slots slots;
  __shared__ Nodes held;
  __shared__ Stage stage;
  const int V = static_cast<int>(a.V);
  const int ctas = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
  const int nvec = V / VE, share = (nvec + ctas - 1) / ctas;
  Rows<T, VE, kStaged> rows{V, min(rank * share, nvec), min((rank + 1) * share, nvec), rank, ctas, &slots};
  rows.pieces = share >= 4 * kVThreads ? kChunks : 1;
  rows.piece = (share + rows.pieces - 1) / rows.pieces;
  rows.abort = &stage.abort;
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
  if (threadIdx.x == 0) {
    stage.abort = 0;
    mbar_init(&slots.bar[0], 1);
    mbar_init(&slots.bar[1], 1);
    if (kStaged)
      for (int i = 0; i < bufs; ++i)
        for (int c = 0; c < kChunks; ++c) mbar_init(&stage.bar[i][c], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  for (int i = threadIdx.x; i < nodes && i < kNodeCap; i += kVThreads) {
    held.tokens[i] = a.tokens[first + i];
    held.parent[i] = a.parent[first + i];
    held.uniform[i] = a.uniform[first + i];
    held.child[i] = INT_MAX;
  }
  __syncthreads();
  const bool small = nodes <= kNodeCap;  // children are looked up in the tables
  if (small)
    for (int i = threadIdx.x; i < nodes; i += kVThreads) {
      const int p = held.parent[i];
      if (p >= 0 && p < i) atomicMin(&held.child[p], i);
      int next = i + 1;
      while (next < nodes && held.parent[next] != p) ++next;
      held.sibling[i] = p >= 0 && next < nodes ? next : -1;
    }
  const float temp = a.temperature ? a.temperature[b] : 1.f;
  const bool no_temp = !(temp >= 0.f), greedy = !(temp > 0.f);
  if (no_temp && nodes > 0) status |= FCT_DEV_NO_DISTRIBUTION;
  const float k = greedy ? kLog2e : kLog2e / temp;
  const float* noise = a.noise + b * a.ld_noise;
  int64_t* toks = a.out_tokens + b * (a.max_depth + 1);
  int32_t* path = a.path + b * a.max_depth;
  // `held` is filled, and every CTA of the cluster runs: its shared memory may
  // be written from now on.
  __syncwarp();
  cluster_barrier();
  auto token = [&](int i) { return i < kNodeCap ? held.tokens[i] : a.tokens[first + i]; };
  auto parent = [&](int i) { return i < kNodeCap ? held.parent[i] : a.parent[first + i]; };
  auto uniform = [&](int i) { return i < kNodeCap ? held.uniform[i] : a.uniform[first + i]; };

  // The first child of `at` after node c, or -1.  Every warp looks for itself
  // and gets the same answer.
  auto next_child = [&](int at, int c) {
    if (small) {
      const int next = c == at ? held.child[at] : held.sibling[c];
      return next == INT_MAX ? -1 : next;
    }
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

  if (kStaged && threadIdx.x == 0 && rows.begin < rows.end)  // read once, at the walk's end
    bulk_prefetch(noise + int64_t(rows.begin) * VE, uint32_t(rows.end - rows.begin) * VE * 4);
  auto target_row = [&](int i) { return static_cast<const T*>(a.target) + (first + i) * a.ld_t; };
  auto draft_row = [&](int i) { return static_cast<const T*>(a.draft) + (first + i) * a.ld_d; };

  // Staging.  Buffers are taken in turn, and every thread keeps the same
  // counts: nodes copied and walked, and for each of the two the buffer that is
  // next and the parity of its barriers' phase.  Warp 0 issues the copies.
  uint32_t issued = 0, used = 0;
  int in_buf = 0, out_buf = 0;
  uint32_t out_parity = 0;
  int ahead = -1;  // the next node to copy, or -1, and its depth and first child
  int64_t ahead_depth = 0;
  int ahead_child = -1;
  auto set_ahead = [&](int node, int64_t d) {
    ahead = node;
    ahead_depth = d;
    ahead_child = node >= 0 && d < a.max_depth ? next_child(node, node) : -1;
  };
  auto stage_next = [&]() {
    if (threadIdx.x < 32) {
      // lane 2 c (2 c + 1): piece c of the target (draft) row
      const bool two = a.draft && !greedy && ahead_child >= 0;
      const int c = lane >> 1;
      const bool second = lane & 1;
      const int from = min(rows.begin + c * rows.piece, rows.end);
      const int n = c < rows.pieces ? min(from + rows.piece, rows.end) - from : 0;
      const uint32_t bytes = uint32_t(n) * 16;
      uint64_t* bar = &stage.bar[in_buf][c < kChunks ? c : 0];
      if (n > 0 && !second) mbar_arrive_expect_tx(bar, two ? 2 * bytes : bytes);
      __syncwarp();
      if (n > 0 && (two || !second))
        bulk_copy(reinterpret_cast<T*>(stage_smem + size_t(in_buf) * buf_bytes) +
                      size_t(second ? share : 0) * VE + size_t(from - rows.begin) * VE,
                  (second ? draft_row(ahead) : target_row(ahead)) + int64_t(from) * VE, bytes, bar);
    }
    ++issued;
    in_buf = in_buf + 1 == bufs ? 0 : in_buf + 1;
    set_ahead(ahead_child, ahead_depth + 1);
  };
  auto take = [&]() {  // the next staged node's buffer has been used (or dropped)
    ++used;
    out_buf = out_buf + 1 == bufs ? 0 : out_buf + 1;
    out_parity ^= out_buf == 0;
  };
  // Waits for the copies of all staged nodes that were not walked.  Every warp
  // does, so that none is a phase behind when it waits for a buffer's next node.
  auto drop = [&]() {
    while (used < issued) {
      if (lane == 0)
        for (int c = 0; c < rows.pieces && rows.begin + c * rows.piece < rows.end; ++c)
          mbar_wait(&stage.bar[out_buf][c], out_parity, &stage.abort, false);
      __syncwarp();
      take();
    }
  };

  int at = 0, staged = -1;  // staged: the node whose copies are next in turn
  int64_t depth = 0, last = -1;
  for (bool walking = nodes > 0 && !no_temp; walking;) {
    const T* tr = target_row(at);
    int c = depth < a.max_depth ? next_child(at, at) : -1;
    if constexpr (kStaged) {
      // Every thread is past its reads of the last node (a reduction's barrier
      // came after them), so that node's buffer is free.
      if (at != staged) {
        // not the node that was copied ahead: drop what is on its way
        drop();
        set_ahead(at, depth);
      }
      while (ahead >= 0 && issued - used < uint32_t(bufs)) stage_next();
      // with room for one node only, the next one's rows at least come to L2
      if (bufs == 1 && ahead >= 0 && threadIdx.x == 0 && rows.begin < rows.end) {
        const uint32_t bytes = uint32_t(rows.end - rows.begin) * 16;
        bulk_prefetch(target_row(ahead) + int64_t(rows.begin) * VE, bytes);
        if (a.draft && !greedy && ahead_child >= 0)
          bulk_prefetch(draft_row(ahead) + int64_t(rows.begin) * VE, bytes);
      }
      rows.t_share = reinterpret_cast<const T*>(stage_smem + size_t(out_buf) * buf_bytes);
      rows.d_share = rows.t_share + size_t(share) * VE;
      rows.bar = stage.bar[out_buf];
      rows.bar_parity = out_parity;
      staged = c;
      take();
    }
    int accepted = -1;
    if (greedy) {
      Best best = best_none();
      bool bad = false;
      rows.template sweep<false, false, kUnroll>(tr, nullptr, nullptr, true, [&](auto& x, auto&, auto&, int v) {
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
      // one pass does, on log2 of p(v) / noise(v) (the logarithm's 2^-20 is the
      // largest error)
      Race best = race_none();
      bool bad = false;
      rows.template sweep<false, true, kNoiseUnroll>(tr, nullptr, noise, true, [&](auto& x, auto&, auto& e, int v) {
        const float top = vec_max(x);
        if (top > best.top) raise(best, top, k);
#pragma unroll
        for (int j = 0; j < int(sizeof(x) / sizeof(float)); ++j) {
          bad |= !(x[j] < INFINITY);
          const float key = fmaf(x[j] - best.top, k, -__log2f(e[j]));
          if (key > best.key) best = Race{key, v + j, best.top};
        }
      });
      best = rows.all(bad ? Race{INFINITY, -1, -INFINITY} : best, race_none(), FoldRace{k});
      if (best.v < 0 || best.v >= V)
        status |= FCT_DEV_NO_DISTRIBUTION;
      else
        last = best.v;
    } else {
      const T* dr = a.draft ? draft_row(at) : nullptr;
      // the first child's logits, on their way while the rows are read
      const int64_t x0 = token(c);
      const bool in0 = x0 >= 0 && x0 < V;
      const float tx0 = in0 ? Elem<T>::load1(tr + x0) : 0.f;
      const float dx0 = in0 && dr ? Elem<T>::load1(dr + x0) : 0.f;
      Lse2x sp = lse2x_empty(), sq = lse2x_empty();
      if (dr)
        rows.template sweep<true, false, kUnroll>(tr, dr, nullptr, true, [&](auto& x, auto& y, auto&, int) {
          fold(sp, x, k);
          fold(sq, y, k);
        });
      else
        rows.template sweep<false, false, kUnroll>(tr, nullptr, nullptr, true,
                                          [&](auto& x, auto&, auto&, int) { fold(sp, x, k); });
      NormPair st{lse2x_fold(sp), lse2x_fold(sq)};
      st = rows.all(st, NormPair{lse2_empty(), lse2_empty()}, FoldNorms());
      const RowNorm p = rows.norm(st.p), q = dr ? rows.norm(st.q) : RowNorm{0.f, 1.f, true};
      if (!p.ok || !q.ok) {
        status |= FCT_DEV_NO_DISTRIBUTION;
        break;
      }
      auto prob = [&](float x, RowNorm n) { return ex2(fmaf(x, k, -n.m2)) * n.inv; };
      float S = 0.f, Z = 1.f, left = 1.f;
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
          if (!dr) {
            if (rows.owns(static_cast<int>(x))) rej.add(static_cast<int>(x));
            left -= rx;
          }
        }
        // with draft logits a token outside the vocabulary has p = q = 0 and
        // still counts as one draw from q
        S += Z;
        tried = c;
        c = next_child(at, c);
        if (c < 0) break;
        // another sibling: the mass that is left.  Without draft logits it is 1
        // less the rejected ones' probabilities; each is within some 2^-19 of
        // itself (the distance from the maximum times 3 * 2^-24, the exponential
        // and the sum), so the difference is good to 2^-16 while an eighth or
        // more is left.
        if (!dr && left >= 0.125f) {
          Z = left;
        } else {
          float z = 0.f;
          auto sum = [&](auto& x, auto& y, auto&, int v) {
            residual(x, y, v);
#pragma unroll
            for (int j = 0; j < int(sizeof(x) / sizeof(float)); ++j) z += x[j];
          };
          if (dr)
            rows.template sweep<true, false, 1>(tr, dr, nullptr, false, sum);
          else
            rows.template sweep<false, false, 1>(tr, nullptr, nullptr, false, sum);
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
            rows.template sweep<true, true, 1>(tr, dr, noise, false, run);
          else
            rows.template sweep<false, true, 1>(tr, nullptr, noise, false, run);
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
  __syncwarp();
  // no CTA leaves while another may still write to it (each has everything
  // that was sent to it, unless a wait ran out)
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  if constexpr (kStaged) drop();  // copies ahead of the walk's end have landed
  if (threadIdx.x == 0 && stage.abort) status |= FCT_DEV_WAIT_TIMEOUT;
  if (writer) {
    toks[depth] = last;
    a.count[b] = static_cast<int32_t>(depth);
  }
  if (threadIdx.x == 0 && status && a.dev_status) atomicOr(a.dev_status, status);
  if (rank == 0)
    for (int64_t i = depth + threadIdx.x; i < a.max_depth; i += kVThreads) {
      toks[i + 1] = -1;
      path[i] = -1;
    }
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <typename T, int VE, bool kStaged>
cudaError_t launch_rows(const VerifyArgs& a, int ctas, int bufs, int buf_bytes, int device,
                        cudaStream_t st) {
  static std::once_flag once[64];
  static cudaError_t ready[64];
  auto kernel = verify_kernel<T, VE, kStaged>;
  if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
  std::call_once(once[device], [&] {
    ready[device] = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (kStaged && ready[device] == cudaSuccess)
      ready[device] =
          cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kStageBytes);
  });
  if (ready[device] != cudaSuccess) return ready[device];
  if (a.batch * ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.batch * ctas));
  cfg.blockDim = dim3(kVThreads);
  cfg.dynamicSmemBytes = size_t(bufs) * size_t(buf_bytes);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, bufs, buf_bytes);
}

template <typename T>
cudaError_t launch_typed(const VerifyArgs& a, int sms, int device, cudaStream_t st) {
  constexpr int kVec = Elem<T>::kVec;
  auto rows16 = [&](const void* p, int64_t ld, size_t e) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (size_t(ld) * e) % 16 == 0;
  };
  const bool vec = rows16(a.target, a.ld_t, sizeof(T)) && rows16(a.noise, a.ld_noise, 4) &&
                   (a.draft == nullptr || rows16(a.draft, a.ld_d, sizeof(T)));
  const int n_rows = a.draft ? 2 : 1;
  auto share_bytes = [&](int c) { return (a.V / kVec + c - 1) / c * 16 * n_rows; };
  // as many CTAs as keep every SM at work, and at least so many that a node's
  // rows fit their shared memory
  int ctas = 1;
  while (ctas < kMaxCtas && (a.batch * ctas * 2 <= sms || share_bytes(ctas) > kStageBytes)) ctas *= 2;
  if (!vec) return launch_rows<T, 1, false>(a, ctas, 0, 0, device, st);
  const int64_t bytes = share_bytes(ctas);
  if (bytes == 0 || bytes > kStageBytes) return launch_rows<T, kVec, false>(a, ctas, 0, 0, device, st);
  const int64_t fit = kStageBytes / bytes;
  const int bufs = static_cast<int>(fit < kMaxBufs ? fit : kMaxBufs);
  return launch_rows<T, kVec, true>(a, ctas, bufs, static_cast<int>(bytes), device, st);
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, int sms, int device, cudaStream_t st) {
  return a.dtype == FCT_F32 ? launch_typed<float>(a, sms, device, st)
                            : launch_typed<bf16_t>(a, sms, device, st);
}

}  // namespace fct
