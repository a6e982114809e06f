// The K largest logits of each row, and the log-sum-exp of the others.
//
// V e bytes from memory, which bound it, in two sweeps: the second reads from
// L2.  The first finds the largest logit of each thread's part of the row.
// These maxima are logits of their own, so what K of them reach, K logits of
// the row reach: their K-th largest is a threshold that about K logits are
// above (70 at K = 64 and 512 threads, 355 at K = 256).  The second sweep
// keeps those few ("candidates") in shared memory and folds all others into
// the log-sum-exp of the rest.  (One sweep with a threshold that rises as it
// goes has 300 to 1200 candidates at K = 64, in nearly every warp's vectors:
// 1218 us at 8192 x 151936 bf16, against ??.)
//
// So the rest is summed from its own terms, never as a difference: it keeps
// its relative precision however little it holds.  Candidates beyond the K-th
// are added as integers (2^40 = the largest of them), in any order the same;
// the order of the other terms is fixed by the row's layout.  Repeated calls
// give the same bits.
//
// Equal logits rank by index.  Where more candidates come than there is room
// for (rows of few values), the second sweep is done again in rounds of rising
// index with a selection in between: its threshold only ever meets later
// rounds, where an equal logit has a larger index than K that rank before it.
#include <climits>
#include <mutex>

#include "fct_internal.h"
#include "fct_top.cuh"

namespace fct {

namespace {

using namespace top;

constexpr int kThreads = kRowThreads;
constexpr int kWarps = kRowWarps;
constexpr int kBins = 1024;
// Up to this K a thread's part has one maximum, above it one per vector of a
// chunk: the maxima have to be several times K for the threshold to be near
// the K-th logit.
constexpr int kFewMaxima = 384;

// A selection may keep this many more than K: it need not split a bin.
__host__ __device__ constexpr int slack(int K) { return K / 4 + 32; }
// Room for candidates: what a selection keeps and one round of vectors.
__host__ __device__ constexpr int capacity(int K, int vec) {
  return K + slack(K) + kThreads * vec;
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
constexpr uint32_t kKeyZero = 0x80000000u;    // key_of(0)

// Entries rank by value, then by lower index.
__device__ __forceinline__ uint64_t rank_key(uint32_t key, int idx) {
  return (uint64_t(key) << 32) | uint32_t(~idx);
}

struct Shared {
  uint64_t* entry;  // [cap] rank keys of the candidates
  int* hist;        // [kBins]
};
__device__ __forceinline__ float entry_value(uint64_t e) {
  return value_of(static_cast<uint32_t>(e >> 32));
}
__device__ __forceinline__ int entry_index(uint64_t e) {
  return static_cast<int>(~static_cast<uint32_t>(e));
}

struct Scratch {  // static shared memory of a CTA
  int pushed;     // candidates
  uint32_t lo, hi;
  int warp_count[kWarps];
  int bin, above, inside;
  int kept;
  uint32_t drop_key;
  unsigned long long drop_sum;
  float2 warp_state[kWarps];
  uint64_t state; // for CTA 0 of the cluster: the CTA's part of the rest
  uint64_t n;     // and its candidates
};

// What has been dropped, as a base-2 state (all threads hold the same).
__device__ __forceinline__ void add_state(float2& a, float m2, float s) {
  const Lse2 r = merge(Lse2{a.x, a.y}, Lse2{m2, s});
  a = make_float2(r.m2, r.s);
}

// Adds those of entries [from, n) that is_dropped says to `out`: integers in
// units of 2^-40 of the largest, so that their order does not matter.
template <typename F>
__device__ void drop(const Shared& sh, Scratch& sc, int from, int n, float2& out, F is_dropped) {
  const int tid = threadIdx.x;
  if (tid == 0) {
    sc.drop_key = 0;
    sc.drop_sum = 0;
  }
  row_sync();
  uint32_t m = 0;
  for (int i = from + tid; i < n; i += kThreads)
    if (is_dropped(sh.entry[i])) m = max(m, static_cast<uint32_t>(sh.entry[i] >> 32));
  m = __reduce_max_sync(0xffffffffu, m);
  if ((tid & 31) == 0 && m) atomicMax(&sc.drop_key, m);
  row_sync();
  const uint32_t top = sc.drop_key;
  if (top == 0) return;  // nothing dropped (a candidate's key is above that of -inf)
  const float m2 = value_of(top) * kLog2e;
  unsigned long long sum = 0;
  for (int i = from + tid; i < n; i += kThreads)
    if (is_dropped(sh.entry[i]))
      sum += static_cast<unsigned long long>(ex2(fmaf(entry_value(sh.entry[i]), kLog2e, -m2)) *
                                             1099511627776.f);
#pragma unroll
  for (int k = 16; k >= 1; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
  if ((tid & 31) == 0 && sum) atomicAdd(&sc.drop_sum, sum);
  row_sync();
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
__device__ __noinline__ int select(const Shared& sh, Scratch& sc, int n, int K, float2& dropped,
                                   float& thr) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    sc.lo = 0xffffffffu;
    sc.hi = 0;
    sc.kept = 0;
  }
  row_sync();
  uint32_t lo = 0xffffffffu, hi = 0;
  for (int i = tid; i < n; i += kThreads) {
    const uint32_t k = static_cast<uint32_t>(sh.entry[i] >> 32);
    lo = min(lo, k);
    hi = max(hi, k);
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) {
    atomicMin(&sc.lo, lo);
    atomicMax(&sc.hi, hi);
  }
  row_sync();
  uint64_t from = uint64_t(sc.lo) << 32, to = (uint64_t(sc.hi) << 32) | 0xffffffffu;
  int above = 0;  // entries ranking above the range
  for (int level = 0; level < 8; ++level) {
    const uint64_t span = to - from;
    const int shift = max(0, 54 - __clzll(static_cast<long long>(span | 1)));
    for (int i = tid; i < kBins; i += kThreads) sh.hist[i] = 0;
    row_sync();
    for (int i = tid; i < n; i += kThreads) {
      const uint64_t k = sh.entry[i];
      if (k >= from && k <= to) atomicAdd(&sh.hist[(k - from) >> shift], 1);
    }
    row_sync();
    // bins from the highest down, two per thread
    const int b0 = kBins - 1 - 2 * tid, c0 = sh.hist[b0], c1 = sh.hist[b0 - 1];
    int run = c0 + c1;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, run, d);
      if (lane >= d) run += o;
    }
    if (lane == 31) sc.warp_count[warp] = run;
    row_sync();
    int before = above + run - (c0 + c1);
    for (int w = 0; w < warp; ++w) before += sc.warp_count[w];
    if (before < K && before + c0 + c1 >= K) {
      const bool second = before + c0 < K;
      sc.bin = second ? b0 - 1 : b0;
      sc.above = second ? before + c0 : before;
      sc.inside = second ? c1 : c0;
    }
    row_sync();
    above = sc.above;
    const uint64_t start = from + (uint64_t(sc.bin) << shift);
    const uint64_t end = start + ((uint64_t(1) << shift) - 1);
    from = start;
    if (end < to) to = end;
    if (above + sc.inside <= K + slack(K)) break;
    row_sync();  // the result is read before the next level writes it
  }
  drop(sh, sc, 0, n, dropped, [&](uint64_t e) { return e < from; });
  // moved towards the front, a block of entries at a time: writes stay behind reads
  for (int base = 0; base < n; base += kThreads) {
    const int i = base + tid;
    const uint64_t e = i < n ? sh.entry[i] : 0;
    row_sync();
    if (i < n && e >= from) sh.entry[atomicAdd(&sc.kept, 1)] = e;
    row_sync();
  }
  thr = value_of(static_cast<uint32_t>(from >> 32));
  return sc.kept;
}

// Sorts n entries, highest rank first (bitonic; the room up to a power of two
// is there).  Pairs of up to 64 entries stay within a warp's entries.
__device__ __noinline__ void sort_entries(const Shared& sh, int n) {
  const int tid = threadIdx.x;
  int P = 64;
  while (P < n) P *= 2;
  for (int i = n + tid; i < P; i += kThreads) sh.entry[i] = 0;
  row_sync();
  for (int size = 2; size <= P; size *= 2) {
    for (int step = size / 2; step > 0; step /= 2) {
      for (int i = tid; i < P / 2; i += kThreads) {
        const int lo = 2 * i - (i & (step - 1)), hi = lo + step;
        const uint64_t x = sh.entry[lo], y = sh.entry[hi];
        if ((x < y) == ((lo & size) == 0)) {
          sh.entry[lo] = y;
          sh.entry[hi] = x;
        }
      }
      // the next step's pairs: 2 step entries apart at most
      if (step > 32 || (step == 1 && size >= 64))
        row_sync();
      else
        __syncwarp();
    }
  }
  row_sync();
}

// The largest t, with 16 bits, such that K of the block's values reach it (0:
// fewer than K are above -inf): a bit a round.
template <int N>
__device__ __forceinline__ uint32_t block_threshold(const uint32_t (&key)[N], int K) {
  uint32_t t = 0;
  for (int bit = 31; bit >= 16; --bit) {
    const uint32_t trial = t | (1u << bit);
    int c = 0;
#pragma unroll
    for (int u = 0; u < N; ++u) c += row_count(key[u] >= trial);
    if (c >= K) t = trial;
  }
  return t;
}

__device__ __forceinline__ float raw_max(uint4 w, float) {
  return fmaxf(max3(__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z)),
               __uint_as_float(w.w));
}
__device__ __forceinline__ float raw_max(uint4 w, bf16_t) {
  float x[8];
  Elem<bf16_t>::unpack(w, x);
  return vec_max(x);
}

// One cluster of C CTAs per row at a time, C by V and the element type alone.
// Each CTA finds the candidates of its share of the row; CTA 0 then takes over
// the others' candidates and states.
template <typename T>
__global__ void __launch_bounds__(kStreamThreads, 2)
    top_select_kernel(TopSelectArgs a, int cap, int stages) {
  constexpr int VE = Elem<T>::kVec;
  extern __shared__ uint4 select_smem[];
  __shared__ Scratch sc;
  __shared__ __align__(8) RingBars bars;
  // CTA 0's: the others' candidates are ready; the others': CTA 0 has taken them over
  __shared__ __align__(8) uint64_t ready_bar, taken_bar;
  const Shared sh{reinterpret_cast<uint64_t*>(select_smem + stages * kChunkVecs),
                  reinterpret_cast<int*>(select_smem + stages * kChunkVecs) + 2 * cap};
  const int K = static_cast<int>(a.K), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int V = static_cast<int>(a.V);
  const int C = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
  const int64_t n_clusters = gridDim.x / C;
  Ring ring(&bars, select_smem, stages);
  if (tid == 0) {
    mbar_init(&ready_bar, C > 1 ? C - 1 : 1);
    mbar_init(&taken_bar, 1);
    ring.init();
  }
  __syncthreads();
  cluster_barrier();  // every CTA's barriers exist
  auto share_of = [&](const Row<T>& r, int* v0, int* v1) {
    const int per = static_cast<int>(share(r.nvec, C));
    *v0 = min(rank * per, r.nvec);
    *v1 = min(*v0 + per, r.nvec);
  };

  if (tid >= kThreads) {
    if (tid == kThreads) {  // ---- copies: every share twice
      const uint64_t once = policy_evict_first(), again = policy_evict_last();
      uint32_t copied = 0;
      for (int64_t row = blockIdx.x / C; row < a.BT; row += n_clusters) {
        const Row<T> r(static_cast<const T*>(a.logits) + row * a.ld, V);
        int v0, v1;
        share_of(r, &v0, &v1);
        if (!ring.copy(r, v0, v1, again)) break;
        copied += chunks_of(v0, v1);
        if (!ring.copy(r, v0, v1, once)) break;
        copied += chunks_of(v0, v1);
      }
      ring.drain(copied);
    }
  } else {
    uint32_t turn = 0;
    for (int64_t row = blockIdx.x / C; row < a.BT; row += n_clusters, ++turn) {
      const Row<T> r(static_cast<const T*>(a.logits) + row * a.ld, V);
      int v0, v1;
      share_of(r, &v0, &v1);

      // ---- first sweep: the threshold
      float mx[kPerThread];
#pragma unroll
      for (int u = 0; u < kPerThread; ++u) mx[u] = -INFINITY;
      ring.each(v0, v1,
                [&](uint4 w, int, int u) { mx[u] = fmaxf(mx[u], raw_max(w, T{})); });
      uint32_t least;
      if (K <= kFewMaxima) {
        const uint32_t key[1] = {key_of(fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]))};
        least = block_threshold(key, K);
      } else {
        const uint32_t key[4] = {key_of(mx[0]), key_of(mx[1]), key_of(mx[2]), key_of(mx[3])};
        least = block_threshold(key, K);
      }
      // logits at it are candidates too: the threshold is the number before it
      // (before 0, not the other 0)
      float thr = least == kKeyZero          ? -__uint_as_float(1u)
                  : least > kKeyNegInf + 1 ? value_of(least - 1)
                                           : -INFINITY;
      if (tid == 0) sc.pushed = 0;
      // CTA 0 has taken over the last row's candidates
      if (rank != 0 && turn > 0) wait_cluster(&taken_bar, (turn - 1) & 1u, &bars.abort);
      row_sync();

      // ---- second sweep
      Run st = run_empty();
      float2 dropped = make_float2(-INFINITY, 0.f);
      auto push = [&](float x, int v) {
        const int at = atomicAdd(&sc.pushed, 1);
        if (at < cap) sh.entry[at] = rank_key(key_of(x), v);
      };
      // one vector: candidates pushed, the others folded
      auto take = [&](uint4 raw, int i) {
        float x[VE];
        Elem<T>::unpack(raw, x);
        float vm = vec_max(x);
        if (vm > thr) {
          const int e0 = r.head + i * VE;
#pragma unroll
          for (int j = 0; j < VE; ++j)
            if (x[j] > thr) {
              push(x[j], e0 + j);
              x[j] = -INFINITY;
            }
          vm = vec_max(x);
        }
        fold(st, x, vm);
      };
      auto take_loose = [&](int v) {
        const float x = Elem<T>::load1(r.p + v);
        if (x > thr) {
          push(x, v);
        } else {
          const float one[2] = {x, -INFINITY};
          fold(st, one, x);
        }
      };
      const bool has_head = rank == 0 && tid < r.head;
      const bool has_tail = rank == C - 1 && r.tail0 + tid < V;
      if (has_head) take_loose(tid);
      ring.each(v0, v1, [&](uint4 w, int i, int) { take(w, i); });
      if (has_tail) take_loose(r.tail0 + tid);
      row_sync();
      int n = sc.pushed;
      if (n > cap) {  // too many: again, a round of one vector per thread at a time
        row_sync();
        if (tid == 0) sc.pushed = 0;
        row_sync();
        st = run_empty();
        auto room = [&](int more) {  // the candidates so far, with room for a round
          row_sync();
          n = sc.pushed;
          row_sync();
          if (n + more > cap) {
            n = select(sh, sc, n, K, dropped, thr);
            row_sync();
            if (tid == 0) sc.pushed = n;
            row_sync();
          }
        };
        if (has_head) take_loose(tid);
        for (int c = v0; c < v1; c += kThreads) {
          room(kThreads * VE);
          if (c + tid < v1) take(*r.vec(c + tid), c + tid);
        }
        room(VE);
        if (has_tail) take_loose(r.tail0 + tid);
        row_sync();
        n = sc.pushed;
      }
      if (n > K + slack(K)) n = select(sh, sc, n, K, dropped, thr);
      const Lse2 w = merge_warp(folded(st));
      if (lane == 0) sc.warp_state[warp] = make_float2(w.m2, w.s);
      row_sync();
      Lse2 rest{-INFINITY, 0.f};  // warp 0 of CTA 0: the row's, but for what is dropped below
      if (warp == 0) {
        const float2 own = lane < kWarps ? sc.warp_state[lane] : make_float2(-INFINITY, 0.f);
        rest = merge(merge_warp(Lse2{own.x, own.y}), Lse2{dropped.x, dropped.y});
      }
      dropped = make_float2(-INFINITY, 0.f);
      if (rank != 0) {
        if (tid == 0) {
          sc.state = (uint64_t(__float_as_uint(rest.m2)) << 32) | __float_as_uint(rest.s);
          sc.n = static_cast<uint64_t>(n);
          arrive_at(&ready_bar, 0);  // and all entries, written before the last barrier
        }
        continue;
      }
      if (C > 1) {
        wait_cluster(&ready_bar, turn & 1u, &bars.abort);
        for (int p = 1; p < C; ++p) {
          const uint64_t o = peer_word(&sc.state, static_cast<uint32_t>(p));
          rest = merge(rest, Lse2{__uint_as_float(static_cast<uint32_t>(o >> 32)),
                                  __uint_as_float(static_cast<uint32_t>(o))});
          // (a CTA keeps no more than this; after a wait that ran out, anything is read)
          const int more = static_cast<int>(
              min(peer_word(&sc.n, static_cast<uint32_t>(p)), uint64_t(K + slack(K))));
          if (n + more > cap) n = select(sh, sc, n, K, dropped, thr);
          for (int i = tid; i < more; i += kThreads)
            sh.entry[n + i] = peer_word(sh.entry + i, static_cast<uint32_t>(p));
          n += more;
          row_sync();
        }
        if (tid > 0 && tid < C) arrive_at(&taken_bar, static_cast<uint32_t>(tid));
        if (n > K + slack(K)) n = select(sh, sc, n, K, dropped, thr);
      }
      sort_entries(sh, n);
      for (int i = tid; i < K; i += kThreads) {
        const uint64_t e = i < n ? sh.entry[i] : 0;
        a.values[row * a.ld_v + i] = i < n ? entry_value(e) : -INFINITY;
        a.index[row * a.ld_i + i] = i < n ? entry_index(e) : -1;
      }
      if (n > K) drop(sh, sc, K, n, dropped, [](uint64_t) { return true; });
      if (tid == 0) {
        rest = merge(rest, Lse2{dropped.x, dropped.y});
        const bool inf = n > 0 && entry_value(sh.entry[0]) == INFINITY;
        const float out = inf ? __uint_as_float(0x7fc00000u) : finish(rest.m2, rest.s);
        a.rest[row] = out;
        if ((out != out || n == 0) && a.dev_status) atomicOr(a.dev_status, FCT_DEV_NO_DISTRIBUTION);
      }
      row_sync();
    }
  }
  __syncthreads();
  cluster_barrier();  // no CTA leaves while a peer may send to it or read from it
  if (tid == 0 && bars.abort && a.dev_status) atomicOr(a.dev_status, FCT_DEV_WAIT_TIMEOUT);
}

// CTAs per row: the rows in flight (two CTAs per SM) fit in 0.8 of L2, from
// which the second sweep reads.
int ctas_per_row(int64_t V, int dtype, int sms, int l2) {
  const double row = double(V) * (dtype == FCT_BF16 ? 2 : 4);
  int C = 1;
  while (C < 8 && 2.0 * sms / C * row > 0.8 * l2) C *= 2;
  return C;
}

template <typename T>
cudaError_t run(const TopSelectArgs& a, int sms, int device, int l2, cudaStream_t st) {
  const int K = static_cast<int>(a.K);
  const int cap = capacity(K, Elem<T>::kVec);
  const size_t lists = size_t(cap) * 8 + kBins * 4;
  auto kernel = top_select_kernel<T>;
  static std::once_flag once[64];
  static cudaError_t set[64];
  std::call_once(once[device], [&] {
    set[device] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kStreamSmem);
  });
  if (set[device] != cudaSuccess) return set[device];
  const int C = ctas_per_row(a.V, a.dtype, sms, l2);
  const int stages = static_cast<int>((kStreamSmem / 2 - lists) / (kChunkVecs * 16));
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(C);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(kStreamThreads);
  cfg.dynamicSmemBytes = size_t(stages) * kChunkVecs * 16 + lists;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = st;
  int64_t clusters = int64_t(sms) * 2 / C;
  if (clusters < 1) clusters = 1;
  if (clusters > a.BT) clusters = a.BT;
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * C));
  return cudaLaunchKernelEx(&cfg, kernel, a, cap, stages);
}

}  // namespace

cudaError_t launch_top_select(const TopSelectArgs& a, int sms, int device, int l2,
                              cudaStream_t st) {
  return a.dtype == FCT_BF16 ? run<bf16_t>(a, sms, device, l2, st)
                             : run<float>(a, sms, device, l2, st);
}

}  // namespace fct
