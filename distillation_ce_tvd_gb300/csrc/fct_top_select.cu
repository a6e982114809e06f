// The K largest logits of each row, and the log-sum-exp of the others.
//
// One pass over the row, V e bytes, which bound it.  A threshold that at least
// K logits seen so far exceed or equal splits what comes: logits at or below
// it are folded into the log-sum-exp of the rest at once; the few above it
// ("candidates") are kept in shared memory with their index.  When those are
// many, or the row ends, a histogram selection keeps the K largest (and a few
// more), raises the threshold, and hands what it drops to the rest.
//
// So the rest is summed from its own terms, never as a difference: it keeps
// its relative precision however little it holds.  What a selection drops is
// added as integers (2^40 = its largest term), in any order the same; the
// order of the other terms is fixed by the row's layout.  Repeated calls give
// the same bits.
//
// Equal logits rank by index.  The row is taken in rounds of increasing index,
// and a threshold only ever meets later rounds: there, an equal logit has a
// larger index than K logits that rank before it.
#include <climits>
#include <mutex>

#include "fct_internal.h"
#include "fct_top.cuh"

namespace fct {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;  // vectors in flight per thread: the rounds of a step
constexpr int kBins = 1024;

// A selection may keep this many more than K: it need not split a bin.
__host__ __device__ constexpr int slack(int K) { return K / 4 + 32; }
// Room for candidates: what a selection keeps and one round of vectors.
__host__ __device__ constexpr int capacity(int K, int vec) {
  return K + slack(K) + kThreads * vec;
}

__host__ __device__ constexpr int hist_size(int K) {
  return kBins > K + slack(K) ? kBins : K + slack(K);
}

// Unsigned key that increases with the float (no NaN comes here; -0 is +0).
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
constexpr uint32_t kKeyNegInf = 0x007fffffu;  // key_of(-inf)

// Entries rank by value, then by lower index.
__device__ __forceinline__ uint64_t rank_key(uint32_t key, int idx) {
  return (uint64_t(key) << 32) | uint32_t(~idx);
}

struct Shared {
  uint32_t* key;  // [cap]
  int* idx;       // [cap]
  int* hist;      // [hist_size(K)]: a selection's bins, then the entries' places
};

struct Scratch {  // static shared memory of a CTA
  int pushed[3];  // candidates of this step, the last and the next
  uint32_t lo, hi;
  int warp_count[kWarps];
  int bin, above, inside;
  int kept;
  uint32_t drop_key;
  unsigned long long drop_sum;
  float2 warp_state[kWarps];
  uint32_t warp_key[kWarps];
};

// What has been dropped, as a base-2 state (all threads hold the same).
__device__ __forceinline__ void add_state(float2& a, float m2, float s) {
  const Lse2 r = top::merge(Lse2{a.x, a.y}, Lse2{m2, s});
  a = make_float2(r.m2, r.s);
}

// Adds the entries that `is_dropped(i)` names, of n, to `out`: integers in
// units of 2^-40 of the largest, so that their order does not matter.
template <typename F>
__device__ void drop(const Shared& sh, Scratch& sc, int n, float2& out, F is_dropped) {
  const int tid = threadIdx.x;
  if (tid == 0) {
    sc.drop_key = 0;
    sc.drop_sum = 0;
  }
  __syncthreads();
  uint32_t m = 0;
  for (int i = tid; i < n; i += kThreads)
    if (is_dropped(i)) m = max(m, sh.key[i]);
  m = __reduce_max_sync(0xffffffffu, m);
  if ((tid & 31) == 0 && m) atomicMax(&sc.drop_key, m);
  __syncthreads();
  const uint32_t top = sc.drop_key;
  if (top == 0) return;  // nothing dropped (a candidate's key is above that of -inf)
  const float m2 = value_of(top) * kLog2e;
  unsigned long long sum = 0;
  for (int i = tid; i < n; i += kThreads)
    if (is_dropped(i))
      sum += static_cast<unsigned long long>(ex2(fmaf(value_of(sh.key[i]), kLog2e, -m2)) *
                                             1099511627776.f);
#pragma unroll
  for (int k = 16; k >= 1; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
  if ((tid & 31) == 0 && sum) atomicAdd(&sc.drop_sum, sum);
  __syncthreads();
  add_state(out, m2, static_cast<float>(sc.drop_sum) * (1.f / 1099511627776.f));
}

// Keeps the K highest-ranking of n > K + slack entries, or up to `slack` more,
// at the front; drops the others.  Returns how many are kept and the value
// below or at which nothing of a later round can rank.
//
// Levels of a histogram over a range of rank keys: the range first spans all
// entries, then the bin that holds the K-th, until the bins up to that one
// hold few enough.  The K-th bin narrows by 1024 a level; single keys are
// unique, so that it ends.
__device__ int select(const Shared& sh, Scratch& sc, int n, int K, float2& dropped, float& thr) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    sc.lo = 0xffffffffu;
    sc.hi = 0;
    sc.kept = 0;
  }
  __syncthreads();
  uint32_t lo = 0xffffffffu, hi = 0;
  for (int i = tid; i < n; i += kThreads) {
    lo = min(lo, sh.key[i]);
    hi = max(hi, sh.key[i]);
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) {
    atomicMin(&sc.lo, lo);
    atomicMax(&sc.hi, hi);
  }
  __syncthreads();
  uint64_t from = uint64_t(sc.lo) << 32, to = (uint64_t(sc.hi) << 32) | 0xffffffffu;
  int above = 0;  // entries ranking above the range
  for (int level = 0; level < 8; ++level) {
    const uint64_t span = to - from;
    const int shift = max(0, 54 - __clzll(static_cast<long long>(span | 1)));
    for (int i = tid; i < kBins; i += kThreads) sh.hist[i] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
      const uint64_t k = rank_key(sh.key[i], sh.idx[i]);
      if (k >= from && k <= to) atomicAdd(&sh.hist[(k - from) >> shift], 1);
    }
    __syncthreads();
    // bins from the highest down, two per thread
    const int b0 = kBins - 1 - 2 * tid, c0 = sh.hist[b0], c1 = sh.hist[b0 - 1];
    int run = c0 + c1;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, run, d);
      if (lane >= d) run += o;
    }
    if (lane == 31) sc.warp_count[warp] = run;
    __syncthreads();
    int before = above + run - (c0 + c1);
    for (int w = 0; w < warp; ++w) before += sc.warp_count[w];
    if (before < K && before + c0 + c1 >= K) {
      const bool second = before + c0 < K;
      sc.bin = second ? b0 - 1 : b0;
      sc.above = second ? before + c0 : before;
      sc.inside = second ? c1 : c0;
    }
    __syncthreads();
    above = sc.above;
    const uint64_t start = from + (uint64_t(sc.bin) << shift);
    const uint64_t end = start + ((uint64_t(1) << shift) - 1);
    from = start;
    if (end < to) to = end;
    if (above + sc.inside <= K + slack(K)) break;
    __syncthreads();  // the result is read before the next level writes it
  }
  drop(sh, sc, n, dropped, [&](int i) { return rank_key(sh.key[i], sh.idx[i]) < from; });
  // moved towards the front, a block of entries at a time: writes stay behind reads
  for (int base = 0; base < n; base += kThreads) {
    const int i = base + tid;
    uint32_t k = 0;
    int v = 0;
    bool keep = false;
    if (i < n) {
      k = sh.key[i];
      v = sh.idx[i];
      keep = rank_key(k, v) >= from;
    }
    __syncthreads();
    if (keep) {
      const int at = atomicAdd(&sc.kept, 1);
      sh.key[at] = k;
      sh.idx[at] = v;
    }
    __syncthreads();
  }
  thr = value_of(static_cast<uint32_t>(from >> 32));
  return sc.kept;
}

// The largest t such that `want` of the warp's values are at or above it, by
// the top 16 bits of its key (0: fewer have one).
__device__ __forceinline__ uint32_t warp_threshold(const uint32_t (&key)[kUnroll], int want) {
  uint32_t t = 0;
#pragma unroll
  for (int bit = 31; bit >= 16; --bit) {
    const uint32_t trial = t | (1u << bit);
    int c = 0;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) c += __popc(__ballot_sync(0xffffffffu, key[u] >= trial));
    if (c >= want) t = trial;
  }
  return t;
}

// One CTA per row at a time.
template <typename T>
__global__ void __launch_bounds__(kThreads, 3) top_select_kernel(TopSelectArgs a, int cap) {
  constexpr int VE = Elem<T>::kVec;
  extern __shared__ uint32_t select_smem[];
  __shared__ Scratch sc;
  const Shared sh{select_smem, reinterpret_cast<int*>(select_smem + cap),
                  reinterpret_cast<int*>(select_smem + 2 * cap)};
  const int K = static_cast<int>(a.K), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int V = static_cast<int>(a.V);
  const uint64_t once = policy_evict_first();
  for (int64_t row = blockIdx.x; row < a.BT; row += gridDim.x) {
    const T* p = static_cast<const T*>(a.logits) + row * a.ld;
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(p) % 16 / sizeof(T));
    const int head = off ? min(VE - off, V) : 0;
    const int nvec = (V - head) / VE, tail0 = head + nvec * VE;
    const uint4* vecs = reinterpret_cast<const uint4*>(p + head);
    if (tid < 3) sc.pushed[tid] = 0;
    __syncthreads();

    Lse2x st = lse2x_empty();
    float2 dropped = make_float2(-INFINITY, 0.f);
    float thr = -INFINITY;
    int n = 0, slot = 0;
    auto push = [&](float x, int v) {
      const int at = n + atomicAdd(&sc.pushed[slot], 1);
      if (at < cap) {
        sh.key[at] = key_of(x);
        sh.idx[at] = v;
      }
    };
    // one vector: candidates pushed, the others folded
    auto take = [&](uint4 raw, int i) {
      float x[VE];
      Elem<T>::unpack(raw, x);
      float vm = vec_max(x);
      if (vm > thr) {
        const int e0 = head + i * VE;
#pragma unroll
        for (int j = 0; j < VE; ++j)
          if (x[j] > thr) {
            push(x[j], e0 + j);
            x[j] = -INFINITY;
          }
        vm = vec_max(x);
      }
      top::fold(st, x, vm);
    };
    // the end of a step: everybody knows the candidates pushed in it
    auto settle = [&]() {
      __syncthreads();
      const int got = sc.pushed[slot];
      slot = slot == 2 ? 0 : slot + 1;
      if (tid == 0) sc.pushed[slot == 2 ? 0 : slot + 1] = 0;
      return got;
    };

    if (tid < head) {  // fewer than a vector: always room
      const float x = Elem<T>::load1(p + tid);
      if (x > thr) {
        push(x, tid);
      } else {
        const float one[2] = {x, -INFINITY};
        top::fold(st, one, x);
      }
    }
    n += settle();
    for (int c = 0; c < nvec; c += kUnroll * kThreads) {
      uint4 raw[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int i = c + u * kThreads + tid;
        if (i < nvec) raw[u] = ld16(vecs + i, once);
      }
      if (c == 0) {
        // A first threshold: the vectors' maxima are logits of their own, so
        // what K of them reach, K logits reach.  Each warp finds what its
        // share of K reach, and the least of those holds for all.
        uint32_t key[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          key[u] = 0;
          if (c + u * kThreads + tid < nvec) {
            float x[VE];
            Elem<T>::unpack(raw[u], x);
            key[u] = key_of(vec_max(x));
          }
        }
        const uint32_t t = warp_threshold(key, (K + kWarps - 1) / kWarps);
        if (lane == 0) sc.warp_key[warp] = t;
        __syncthreads();
        uint32_t least = sc.warp_key[0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) least = min(least, sc.warp_key[w]);
        // logits at it are candidates too: the threshold is the float before
        if (least > kKeyNegInf + 1) thr = value_of(least - 1);
      }
      const Lse2x st0 = st;
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int i = c + u * kThreads + tid;
        if (i < nvec) take(raw[u], i);
      }
      const int got = settle();
      if (n + got <= cap) {
        n += got;
      } else {  // too many: the step again, round by round, with room made before each
        st = st0;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          if (n + kThreads * VE > cap) n = select(sh, sc, n, K, dropped, thr);
          const int i = c + u * kThreads + tid;
          if (i < nvec) take(raw[u], i);
          n += settle();
        }
      }
      if (n > 4 * K + 512) n = select(sh, sc, n, K, dropped, thr);
    }
    if (tail0 + tid < V) {
      const float x = Elem<T>::load1(p + tail0 + tid);
      if (x > thr) {
        push(x, tail0 + tid);
      } else {
        const float one[2] = {x, -INFINITY};
        top::fold(st, one, x);
      }
    }
    n += settle();
    if (n > K + slack(K)) n = select(sh, sc, n, K, dropped, thr);
    // every entry's place is the number of entries that rank before it
    for (int i = tid; i < n; i += kThreads) {
      const uint64_t mine = rank_key(sh.key[i], sh.idx[i]);
      int place = 0;
      for (int j = 0; j < n; ++j) place += rank_key(sh.key[j], sh.idx[j]) > mine;
      if (place < K) {
        a.values[row * a.ld_v + place] = value_of(sh.key[i]);
        a.index[row * a.ld_i + place] = sh.idx[i];
      }
      sh.hist[i] = place;
    }
    for (int i = n + tid; i < K; i += kThreads) {
      a.values[row * a.ld_v + i] = -INFINITY;
      a.index[row * a.ld_i + i] = -1;
    }
    const Lse2 w = top::warp_merge(lse2x_fold(st));
    if (lane == 0) sc.warp_state[warp] = make_float2(w.m2, w.s);
    __syncthreads();
    if (n > K) drop(sh, sc, n, dropped, [&](int i) { return sh.hist[i] >= K; });
    if (warp == 0) {
      const float2 mine = lane < kWarps ? sc.warp_state[lane] : make_float2(-INFINITY, 0.f);
      const Lse2 r = top::merge(top::warp_merge(Lse2{mine.x, mine.y}), Lse2{dropped.x, dropped.y});
      bool inf = false;
      for (int i = lane; i < n; i += 32) inf = inf || value_of(sh.key[i]) == INFINITY;
      inf = __any_sync(0xffffffffu, inf);
      if (lane == 0) {
        const float rest = inf ? __uint_as_float(0x7fc00000u) : top::finish(r.m2, r.s);
        a.rest[row] = rest;
        if ((rest != rest || n == 0) && a.dev_status) atomicOr(a.dev_status, FCT_DEV_NO_DISTRIBUTION);
      }
    }
    __syncthreads();  // shared memory is read: the next row may come
  }
}

template <typename T>
cudaError_t run(const TopSelectArgs& a, int sms, int device, cudaStream_t st) {
  const int K = static_cast<int>(a.K);
  const int cap = capacity(K, Elem<T>::kVec);
  const size_t smem = (2 * size_t(cap) + hist_size(K)) * 4;
  auto kernel = top_select_kernel<T>;
  static std::once_flag once[64];
  static cudaError_t set[64];
  std::call_once(once[device], [&] {
    set[device] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kTopSmemMax);
  });
  if (set[device] != cudaSuccess) return set[device];
  int64_t grid = int64_t(sms) * 3;
  if (grid > a.BT) grid = a.BT;
  kernel<<<static_cast<unsigned>(grid), kThreads, smem, st>>>(a, cap);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_top_select(const TopSelectArgs& a, int sms, int device, cudaStream_t st) {
  return a.dtype == FCT_BF16 ? run<bf16_t>(a, sms, device, st) : run<float>(a, sms, device, st);
}

}  // namespace fct
