// Cross-entropy + total-variation distance against a teacher's top logits.
//
// The teacher of a row is a list of K (index, logit) pairs and the log-sum-exp
// `rest` of its logits outside the list (include/fused_ce_tvd.h has the
// formulas).  With U the listed words, every word outside U shares one sign,
// sign(p_rest - q_rest), so the loss needs of the V student logits
//   one log-sum-exp over the words outside U, and the K logits of U,
// and the gradient is p_v times one coefficient per row outside U.  Both
// directions are one pass over the row: V e bytes read, and V e written by the
// backward pass, which bound them.
//
// The words of U are left out of the sum as it is taken, not subtracted from
// it: p_rest keeps its relative precision where the list holds nearly all of
// the mass.  A bit per word in shared memory says which those are; a vector of
// 16 bytes looks up its own few bits.
#include <climits>
#include <mutex>

#include "fct_internal.h"
#include "fct_top.cuh"

namespace fct {

namespace {

using top::Coefs;
using top::list_sums;
using top::listed_grad;
using top::make_coefs;
using top::prob;
using top::Sums;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;  // vectors of a row in flight per thread

// ---------------------------------------------------------------- rows

// A row of V elements as `head` elements before the first 16-byte boundary,
// nvec vectors, and the rest from element tail0.  Element v has position
// v - head + kVec: vector i starts at position (i + 1) kVec.
template <typename T>
struct Row {
  const T* p;
  int head, nvec, tail0, V;
  __device__ __forceinline__ Row(const T* row, int V) : p(row), V(V) {
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(row) % 16 / sizeof(T));
    constexpr int kVec = Elem<T>::kVec;
    head = off ? min(kVec - off, V) : 0;
    nvec = (V - head) / kVec;
    tail0 = head + nvec * kVec;
  }
  __device__ __forceinline__ const uint4* vec(int i) const {
    return reinterpret_cast<const uint4*>(p + head) + i;
  }
  // The j-th of the elements that are in no vector.
  __device__ __forceinline__ int loose(int j) const { return j < head ? j : tail0 + (j - head); }
  __device__ __forceinline__ int n_loose() const { return head + (V - tail0); }
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
__device__ __forceinline__ float2 peer_state(const float2* mine, uint32_t rank) {
  float2 v;
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %2, %3;\n\t"
      "ld.shared::cluster.v2.f32 {%0, %1}, [a];\n\t}"
      : "=f"(v.x), "=f"(v.y)
      : "r"(smem_addr(mine)), "r"(rank)
      : "memory");
  return v;
}

template <int N>
__device__ __forceinline__ void outside_grad(const Coefs& c, const float (&x)[N], int off,
                                             float (&g)[N]) {
  const float2 nl = make_float2(-c.lse, -c.lse), L2 = make_float2(kLog2e, kLog2e);
#pragma unroll
  for (int j = 0; j < N; j += 2) {
    const float2 e = __fmul2_rn(__fadd2_rn(make_float2(x[j], x[j + 1]), nl), L2);
    g[j] = ex2(e.x) * c.outside;
    g[j + 1] = ex2(e.y) * c.outside;
  }
  if (static_cast<uint32_t>(off) < uint32_t(N)) {  // the target is in this vector
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (j == off) g[j] = fmaf(prob(x[j], c.lse), c.outside, -c.gce);
  }
}

// Vectors [v0, v1) of a row's gradient outside U, by all threads, and the
// elements in no vector: the head's and the tail's where asked for.
template <typename T>
__device__ __forceinline__ void stream_grad(const Row<T>& r, T* grow, const Coefs& c, int target,
                                            int v0, int v1, bool head, bool tail, uint64_t pol) {
  constexpr int VE = Elem<T>::kVec;
  const int tid = threadIdx.x;
  const bool same = (reinterpret_cast<uintptr_t>(r.p) % 16) == (reinterpret_cast<uintptr_t>(grow) % 16);
  for (int i = v0 + tid; i < v1; i += kUnroll * kThreads) {
    uint4 raw[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (i + u * kThreads < v1) raw[u] = ld16(r.vec(i + u * kThreads), pol);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int iv = i + u * kThreads;
      if (iv >= v1) break;
      float x[VE], g[VE];
      Elem<T>::unpack(raw[u], x);
      const int e0 = r.head + iv * VE;
      outside_grad(c, x, target - e0, g);
      if (same) {
        st16(grow + e0, Elem<T>::pack(g), pol);
      } else {
#pragma unroll
        for (int j = 0; j < VE; ++j) Elem<T>::store1(grow + e0 + j, g[j]);
      }
    }
  }
  if (tid < r.n_loose() && (tid < r.head ? head : tail)) {
    const int v = r.loose(tid);
    const float p = prob(Elem<T>::load1(r.p + v), c.lse);
    Elem<T>::store1(grow + v, v == target ? fmaf(p, c.outside, -c.gce) : p * c.outside);
  }
}

// A gradient row, or its part [v0, v1), set to one value.
template <typename T>
__device__ __forceinline__ void fill_grad(T* grow, int64_t v0, int64_t v1, float value) {
  for (int64_t v = v0 + threadIdx.x; v < v1; v += kThreads) Elem<T>::store1(grow + v, value);
}

// ---------------------------------------------------------------- forward

// Shared memory of a CTA: the bits, then the list's student and teacher logits
// and indices.
struct Shared {
  uint32_t* bits;
  float* s;
  float* t;
  int* idx;
};
__host__ __device__ constexpr size_t list_bytes(int64_t K) { return size_t(K) * 12; }
// Words of bits for `vecs` vectors of a row and the elements in none.
__host__ __device__ constexpr int64_t bit_words(int64_t vecs, int vec) {
  return ((vecs + 2) * vec + 31) / 32 + 1;
}

// Vectors of a row that each of C CTAs takes: a multiple of eight, so that a
// share's bits start on a byte.
__host__ __device__ constexpr int64_t share(int64_t nvec, int C) {
  return ((nvec + C - 1) / C + 7) / 8 * 8;
}

// One cluster of C CTAs per row, C fixed by V and the element type.  Each CTA
// streams its share of the row; every CTA then has the row's sums (the
// forward alone: CTA 0) from its peers' shared memory.
//
// kGrad: the same CTAs go over their share once more, which L2 still holds,
// and write the gradient.
template <typename T, bool kGrad>
__global__ void __launch_bounds__(kThreads, kGrad ? 2 : 3) top_forward_kernel(TopArgs a, int words) {
  constexpr int VE = Elem<T>::kVec;
  extern __shared__ uint32_t top_smem[];
  __shared__ float2 warp_state[kWarps];
  __shared__ float2 cta_state[2];
  __shared__ int bad_flag[2];
  __shared__ Sums sums;
  const int K = static_cast<int>(a.K), V = static_cast<int>(a.V), tid = threadIdx.x;
  const int C = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
  const Shared sh{top_smem, reinterpret_cast<float*>(top_smem + words),
                  reinterpret_cast<float*>(top_smem + words) + K,
                  reinterpret_cast<int*>(top_smem + words) + 2 * K};
  const uint8_t* bytes = reinterpret_cast<const uint8_t*>(sh.bits);
  const uint64_t once = policy_evict_first(), again = policy_evict_last();
  for (int i = tid; i < words; i += kThreads) sh.bits[i] = 0;
  __syncthreads();
  const int64_t n_clusters = gridDim.x / C;
  int turn = 0;
  for (int64_t row = blockIdx.x / C; row < a.BT; row += n_clusters) {
    const T* srow = static_cast<const T*>(a.student) + row * a.ld_s;
    const Row<T> r(srow, V);
    const int per = static_cast<int>(share(r.nvec, C));
    const int v0 = min(rank * per, r.nvec), v1 = min(v0 + per, r.nvec);
    const int64_t tg = a.target[row];
    T* grow = kGrad ? static_cast<T*>(a.grad) + row * a.ld_g : nullptr;
    if (tg == a.ignore_index) {
      if (rank == 0 && tid == 0) {
        a.ce[row] = 0.f;
        a.tvd[row] = 0.f;
        a.lse[row] = 0.f;
        a.rest_lse[row] = 0.f;
        a.t_lse[row] = 0.f;
        a.sigma[row] = 0.f;
      }
      if constexpr (kGrad) {
        const int64_t per_cta = (a.V + C - 1) / C;
        fill_grad(grow, rank * per_cta, min(a.V, (rank + 1) * per_cta), 0.f);
      }
      continue;
    }
    const bool tg_ok = tg >= 0 && tg < V;
    // ---- the list: its logits, and the bits of the words in this CTA's share
    bool bad = false;
    for (int k = tid; k < K; k += kThreads) {
      const int v = a.index[row * a.ld_i + k];
      float s = -INFINITY, t = -INFINITY;
      int at = -1;
      if (v != -1) {
        if (v < 0 || v >= V) {
          bad = true;
        } else {
          at = v;
          s = Elem<T>::load1(srow + v);
          t = a.values[row * a.ld_v + k];
          const int pos = v - r.head + VE - v0 * VE;
          const bool mine = (pos >= VE || rank == 0) && (pos < (v1 - v0 + 1) * VE || rank == C - 1);
          if (mine && (atomicOr(&sh.bits[pos >> 5], 1u << (pos & 31)) >> (pos & 31) & 1u)) bad = true;
        }
      }
      sh.s[k] = s;
      sh.t[k] = t;
      sh.idx[k] = at;
    }
    const float tg_logit = tg_ok ? Elem<T>::load1(srow + tg) : 0.f;
    const int any_bad = __syncthreads_or(bad);
    // ---- the log-sum-exp of the words outside U
    Lse2x st = lse2x_empty();
    for (int i = v0 + tid; i < v1; i += kUnroll * kThreads) {
      uint4 raw[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (i + u * kThreads < v1) raw[u] = ld16(r.vec(i + u * kThreads), kGrad ? again : once);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int iv = i + u * kThreads;
        if (iv >= v1) break;
        float x[VE];
        Elem<T>::unpack(raw[u], x);
        const int pos = (iv - v0 + 1) * VE;
        const uint32_t m = VE == 8 ? bytes[pos >> 3] : (bytes[pos >> 3] >> (pos & 4)) & 15u;
        if (m) {
#pragma unroll
          for (int j = 0; j < VE; ++j)
            if ((m >> j) & 1u) x[j] = -INFINITY;
        }
        top::fold(st, x);
      }
    }
    // the elements in no vector: the head with CTA 0, the tail with the last
    if (tid < r.n_loose() && rank == (tid < r.head ? 0 : C - 1)) {
      const int v = r.loose(tid), pos = v - r.head + VE - v0 * VE;
      const float x = Elem<T>::load1(srow + v);
      const float one[2] = {(sh.bits[pos >> 5] >> (pos & 31)) & 1u ? -INFINITY : x, -INFINITY};
      top::fold(st, one);
    }
    const Lse2 w = top::warp_merge(lse2x_fold(st));
    if ((tid & 31) == 0) warp_state[tid >> 5] = make_float2(w.m2, w.s);
    __syncthreads();
    // the bits go back to 0 for the next row
    for (int k = tid; k < K; k += kThreads) {
      const int pos = sh.idx[k] - r.head + VE - v0 * VE;
      if (sh.idx[k] >= 0 && pos >= 0 && pos < words * 32) sh.bits[pos >> 5] = 0;
    }
    if (tid < 32) {
      const float2 mine = tid < kWarps ? warp_state[tid] : make_float2(-INFINITY, 0.f);
      const Lse2 b = top::warp_merge(Lse2{mine.x, mine.y});
      if (tid == 0) {
        cta_state[turn] = make_float2(b.m2, b.s);
        bad_flag[turn] = any_bad;
      }
    }
    if (C > 1)
      cluster_barrier();  // the states of this turn; those of the last one have been read
    if (tid < 32 && (kGrad || rank == 0)) {
      __syncwarp();
      float2 s = make_float2(-INFINITY, 0.f);
      int b = 0;
      if (tid < C) {
        s = C > 1 ? peer_state(&cta_state[turn], tid) : cta_state[turn];
        if (C > 1)
          asm volatile(
              "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\t"
              "ld.shared::cluster.s32 %0, [a];\n\t}"
              : "=r"(b)
              : "r"(smem_addr(&bad_flag[turn])), "r"(tid)
              : "memory");
        else
          b = bad_flag[turn];
      }
      const bool wrong = __any_sync(0xffffffffu, b != 0);
      const Lse2 rest = top::warp_merge(Lse2{s.x, s.y});
      const float t_rest = a.rest ? a.rest[row] : -INFINITY;
      Sums o = list_sums(sh.s, sh.t, K, rest.m2, rest.s, t_rest);
      const float nan = __uint_as_float(0x7fc00000u);
      if (wrong) o = Sums{nan, nan, nan, nan, nan};
      if (tid == 0) {
        if (rank == 0) {
          a.ce[row] = tg_ok ? o.lse - tg_logit : nan;
          a.tvd[row] = o.tvd;
          a.lse[row] = o.lse;
          a.rest_lse[row] = o.rest;
          a.t_lse[row] = o.t_lse;
          a.sigma[row] = o.sigma;
          const int status = (tg_ok ? 0 : FCT_DEV_TARGET_OUT_OF_RANGE) | (wrong ? FCT_DEV_BAD_LIST : 0);
          if (status && a.dev_status) atomicOr(a.dev_status, status);
        }
        if constexpr (kGrad) sums = o;
      }
    }
    turn ^= 1;
    __syncthreads();
    if constexpr (kGrad) {
      if (!tg_ok) {
        const int64_t per_cta = (a.V + C - 1) / C;
        fill_grad(grow, rank * per_cta, min(a.V, (rank + 1) * per_cta),
                  __uint_as_float(0x7fc00000u));
        __syncthreads();
        continue;
      }
      const Coefs c = make_coefs(a.grad_ce[row * a.grad_stride], a.grad_tvd[row * a.grad_stride],
                                 sums.lse, sums.rest, sums.t_lse,
                                 a.rest ? a.rest[row] : -INFINITY, sums.sigma);
      stream_grad(r, grow, c, static_cast<int>(tg), v0, v1, rank == 0, rank == C - 1, once);
      __syncthreads();  // the words of U over what the stream wrote there
      for (int k = tid; k < K; k += kThreads) {
        const int v = sh.idx[k];
        if (v < 0) continue;
        const int pos = v - r.head + VE - v0 * VE;
        const bool mine = (pos >= VE || rank == 0) && (pos < (v1 - v0 + 1) * VE || rank == C - 1);
        if (mine) Elem<T>::store1(grow + v, listed_grad(c, sh.s[k], sh.t[k], v == tg));
      }
      __syncthreads();  // the list and the sums are read: the next row may come
    }
  }
  if (C > 1) cluster_barrier();  // a peer may still read this CTA's shared memory
}

// ---------------------------------------------------------------- backward

// One CTA per kSeg vectors of a row (the elements in no vector go with the
// last).  It reads the student's logits at the listed words of its segment
// first, streams the segment as if no word were listed, and then writes those
// words again: so the gradient may overwrite the student.
constexpr int kSeg = kUnroll * kThreads;
constexpr int kListRegs = (kTopMax + kThreads - 1) / kThreads;

template <typename T>
__global__ void __launch_bounds__(kThreads, 3) top_backward_kernel(TopArgs a, int64_t segs) {
  constexpr int VE = Elem<T>::kVec;
  const uint64_t once = policy_evict_first();
  const int tid = threadIdx.x, V = static_cast<int>(a.V), K = static_cast<int>(a.K);
  const int64_t row = blockIdx.x / segs;
  const int seg = static_cast<int>(blockIdx.x - row * segs);
  const T* srow = static_cast<const T*>(a.student) + row * a.ld_s;
  T* grow = static_cast<T*>(a.grad) + row * a.ld_g;
  const Row<T> r(srow, V);
  const int v0 = min(seg * kSeg, r.nvec), v1 = min(v0 + kSeg, r.nvec);
  const bool first = seg == 0, last = seg == segs - 1;
  // the segment's elements: its vectors, the head with the first, the tail with the last
  const int e0 = first ? 0 : r.head + v0 * VE, e1 = last ? V : r.head + v1 * VE;
  const int64_t tg = a.target[row];
  if (tg == a.ignore_index || tg < 0 || tg >= V) {
    const bool ignored = tg == a.ignore_index;
    if (!ignored && first && tid == 0 && a.dev_status)
      atomicOr(a.dev_status, FCT_DEV_TARGET_OUT_OF_RANGE);
    fill_grad(grow, e0, e1, ignored ? 0.f : __uint_as_float(0x7fc00000u));
    return;
  }
  const Coefs c = make_coefs(a.grad_ce[row * a.grad_stride], a.grad_tvd[row * a.grad_stride],
                             a.lse[row], a.rest_lse[row], a.t_lse[row],
                             a.rest ? a.rest[row] : -INFINITY, a.sigma[row]);
  int at[kListRegs];
  float g[kListRegs];
#pragma unroll
  for (int j = 0; j < kListRegs; ++j) {
    const int k = tid + j * kThreads;
    at[j] = -1;
    g[j] = 0.f;
    if (k < K) {
      const int v = a.index[row * a.ld_i + k];
      if (v >= e0 && v < e1) {
        at[j] = v;
        g[j] = listed_grad(c, Elem<T>::load1(srow + v), a.values[row * a.ld_v + k], v == tg);
      }
    }
  }
  __syncthreads();
  stream_grad(r, grow, c, static_cast<int>(tg), v0, v1, first, last, once);
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kListRegs; ++j)
    if (at[j] >= 0) Elem<T>::store1(grow + at[j], g[j]);
}

// ---------------------------------------------------------------- launch

// CTAs per row, by V and the element type alone: never the number of rows, so
// that results do not depend on how rows are batched, and the same with and
// without the gradient, so that those give the same bits.  The bits of a CTA's
// share take at most 32 KB, and the rows in flight (two CTAs per SM) fit in
// 0.8 of L2, from which the single launch reads them again.
int ctas_per_row(int64_t V, int dtype, int sms, int l2) {
  const double row = double(V) * (dtype == FCT_BF16 ? 2 : 4);
  int C = 1;
  while (C < 8 && (V > int64_t(C) * 262144 || 2.0 * sms / C * row > 0.8 * l2)) C *= 2;
  return C;
}

template <typename T, bool kGrad>
cudaError_t run_forward(const TopArgs& a, int sms, int device, int l2, cudaStream_t st) {
  constexpr int VE = Elem<T>::kVec;
  const int C = ctas_per_row(a.V, a.dtype, sms, l2);
  const int64_t words = bit_words(share(a.V / VE, C), VE);
  const size_t smem = size_t(words) * 4 + list_bytes(a.K);
  auto kernel = top_forward_kernel<T, kGrad>;
  static std::once_flag once[64];
  static cudaError_t set[64];
  std::call_once(once[device], [&] {
    set[device] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kTopSmemMax);
  });
  if (set[device] != cudaSuccess) return set[device];
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(C);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = st;
  int resident = kGrad ? 2 : 3;
  const int by_smem = static_cast<int>((227 * 1024) / (smem + 1280));
  if (by_smem < resident) resident = by_smem > 0 ? by_smem : 1;
  int64_t clusters = int64_t(sms) * resident / C;
  if (clusters < 1) clusters = 1;
  if (clusters > a.BT) clusters = a.BT;
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * C));
  return cudaLaunchKernelEx(&cfg, kernel, a, static_cast<int>(words));
}

template <typename T>
cudaError_t run_backward(const TopArgs& a, cudaStream_t st) {
  const int64_t nvec = a.V / Elem<T>::kVec;  // at most, whatever a row's alignment
  const int64_t segs = nvec > 0 ? (nvec + kSeg - 1) / kSeg : 1;
  const int64_t rows_per = (int64_t(1) << 31) / segs / 2;
  for (int64_t r0 = 0; r0 < a.BT; r0 += rows_per) {
    TopArgs b = a;
    b.BT = a.BT - r0 < rows_per ? a.BT - r0 : rows_per;
    b.student = static_cast<const T*>(a.student) + r0 * a.ld_s;
    b.grad = static_cast<T*>(a.grad) + r0 * a.ld_g;
    b.target += r0;
    b.index += r0 * a.ld_i;
    b.values += r0 * a.ld_v;
    if (b.rest) b.rest += r0;
    b.lse += r0;
    b.rest_lse += r0;
    b.t_lse += r0;
    b.sigma += r0;
    b.grad_ce += a.grad_stride * r0;
    b.grad_tvd += a.grad_stride * r0;
    top_backward_kernel<T><<<static_cast<unsigned>(b.BT * segs), kThreads, 0, st>>>(b, segs);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_top_forward(const TopArgs& a, int sms, int device, int l2, cudaStream_t st) {
  if (a.dtype == FCT_BF16)
    return a.grad ? run_forward<bf16_t, true>(a, sms, device, l2, st)
                  : run_forward<bf16_t, false>(a, sms, device, l2, st);
  return a.grad ? run_forward<float, true>(a, sms, device, l2, st)
                : run_forward<float, false>(a, sms, device, l2, st);
}

cudaError_t launch_top_backward(const TopArgs& a, cudaStream_t st) {
  return a.dtype == FCT_BF16 ? run_backward<bf16_t>(a, st) : run_backward<float>(a, st);
}

}  // namespace fct
