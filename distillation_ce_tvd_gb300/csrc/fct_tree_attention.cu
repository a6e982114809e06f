// Attention of drafted trees (and of single tokens) over a paged cache; the
// operation is described in include/fused_ce_tvd.h, fct_tree_attention.
#include <cuda_fp16.h>

#include "fct_common.cuh"
#include "fct_internal.h"

namespace fct {

namespace {

// ---------------------------------------------------------------- general layouts
//
// One CTA per node and query head; its warps take every kGWarps-th group of
// keys.  In a warp, `lanes` threads (a power of two, head_dim / 8 rounded up)
// hold a key's vector, 8 elements each, so a warp looks at 32 / lanes keys at
// a time.  Any page size, head_dim and stride that fct_kv_cache takes.

constexpr int kGWarps = 4;

// 8 elements of a cached vector, payload only.
__device__ __forceinline__ void load_cached(const void* pool, int dtype, int64_t at, float (&x)[8]) {
  if (dtype == FCT_BF16) {
    Elem<bf16_t>::unpack(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(pool) + at), x);
  } else {
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(pool) + at);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const uint16_t two = static_cast<uint16_t>((j < 4 ? w.x : w.y) >> (8 * (j % 4)));
      uint32_t h;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      x[j] = f.x;
      x[j + 1] = f.y;
    }
  }
}

// 2^(byte - 127), NaN for byte 255.
__device__ __forceinline__ float scale_of(uint8_t byte) {
  return byte == 255 ? __int_as_float(0x7fc00000)
                     : byte == 0 ? __int_as_float(0x00400000) : __uint_as_float(uint32_t(byte) << 23);
}

__global__ void __launch_bounds__(kGWarps * 32) attention_general_kernel(AttnArgs a, int lanes) {
  __shared__ float sm_m[kGWarps], sm_l[kGWarps];
  __shared__ float sm_o[kGWarps][256];
  const fct_kv_cache& c = a.cache;
  const int64_t node = blockIdx.x / a.n_q_heads;
  const int h = static_cast<int>(blockIdx.x % a.n_q_heads);
  const int kvh = h / (a.n_q_heads / c.n_heads);
  // the request: the last b with node_start[b] <= node
  int64_t lo = 0, hi = a.pages.batch;
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) / 2;
    if (a.node_start[mid] <= node) lo = mid; else hi = mid;
  }
  const int64_t b = lo, first = a.node_start[b], end = a.node_start[b + 1];
  if (node < first || node >= end) return;
  const int64_t i = node - first, nodes = end - first;
  int64_t ctx = a.pages.context_len[b], len = ctx + nodes;
  const int64_t room = a.pages.max_pages * c.page_size;
  int32_t status = 0;
  if (ctx < 0 || len > room) {
    status |= FCT_DEV_INDEX_OUT_OF_RANGE;
    ctx = ctx < 0 ? 0 : ctx;
    len = len < 0 ? 0 : (len > room ? room : len);
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane % lanes, group = lane / lanes, groups = 32 / lanes;
  const bool active = sub * 8 < c.head_dim;
  const int e = c.dtype == FCT_E4M3;
  float q[8] = {}, o[8] = {};
  if (active)
#pragma unroll
    for (int j = 0; j < 8; ++j)
      q[j] = Elem<bf16_t>::load1(static_cast<const bf16_t*>(a.q) + node * a.ld_qn + h * a.ld_qh +
                                 sub * 8 + j) * a.scale * kLog2e;
  float m = -INFINITY, l = 0.f;
  for (int64_t j0 = int64_t(warp) * groups; j0 < len; j0 += kGWarps * groups) {
    const int64_t j = j0 + group;
    bool sees = j < len;
    if (sees && j >= ctx) {
      const int64_t n = j - ctx;
      sees = a.mask == nullptr
                 ? n <= i
                 : n < 64 * a.mask_words && ((a.mask[node * a.mask_words + n / 64] >> (n % 64)) & 1);
    }
    int64_t at = 0, sc = 0;
    if (sees) {
      const int64_t id = a.pages.table[b * a.pages.ld + j / c.page_size];
      if (id < 0 || id >= c.num_pages) {
        status |= FCT_DEV_INDEX_OUT_OF_RANGE;
        sees = false;
      } else {
        const int64_t off = j % c.page_size;
        at = id * c.page_stride + off * c.slot_stride + kvh * c.head_stride + sub * 8;
        sc = id * c.scale_page_stride + off * c.scale_slot_stride + kvh * c.scale_head_stride;
      }
    }
    float k[8] = {}, v[8] = {};
    if (sees && active) {
      load_cached(c.k, c.dtype, at, k);
      load_cached(c.v, c.dtype, at, v);
    }
    float s = 0.f;
#pragma unroll
    for (int d = 0; d < 8; ++d) s = fmaf(q[d], k[d], s);
    for (int x = lanes / 2; x >= 1; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    float vs = 1.f;
    if (e && sees) {
      s *= scale_of(c.k_scale[sc]);
      vs = scale_of(c.v_scale[sc]);
    }
    if (sees) {
      const float mn = fmaxf(m, s);
      const float base = mn == -INFINITY ? 0.f : mn;
      const float r = ex2(m - base), p = ex2(s - base);
      l = l * r + p;
#pragma unroll
      for (int d = 0; d < 8; ++d) o[d] = o[d] * r + p * vs * v[d];
      m = mn;
    }
  }
  // merge the groups of the warp, then the warps
  for (int x = lanes; x < 32; x <<= 1) {
    const float om = __shfl_xor_sync(0xffffffffu, m, x), ol = __shfl_xor_sync(0xffffffffu, l, x);
    const float mn = fmaxf(m, om), base = mn == -INFINITY ? 0.f : mn;
    const float r = ex2(m - base), ro = ex2(om - base);
    l = l * r + ol * ro;
#pragma unroll
    for (int d = 0; d < 8; ++d) o[d] = o[d] * r + __shfl_xor_sync(0xffffffffu, o[d], x) * ro;
    m = mn;
  }
  if (lane < lanes && active) {
#pragma unroll
    for (int d = 0; d < 8; ++d) sm_o[warp][sub * 8 + d] = o[d];
  }
  if (lane == 0) sm_m[warp] = m, sm_l[warp] = l;
  __syncthreads();
  float top = -INFINITY, total = 0.f;
#pragma unroll
  for (int w = 0; w < kGWarps; ++w) top = fmaxf(top, sm_m[w]);
  const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
  for (int w = 0; w < kGWarps; ++w) total += sm_l[w] * ex2(sm_m[w] - base);
  for (int d = threadIdx.x; d < c.head_dim; d += kGWarps * 32) {
    float r = 0.f;
#pragma unroll
    for (int w = 0; w < kGWarps; ++w) r += sm_o[w][d] * ex2(sm_m[w] - base);
    Elem<bf16_t>::store1(static_cast<bf16_t*>(a.out) + node * a.ld_on + h * a.ld_oh + d,
                         total == 0.f ? 0.f : r / total);
  }
  if (a.lse && threadIdx.x == 0)
    a.lse[node * a.n_q_heads + h] = total == 0.f ? -INFINITY : (top + log2f(total)) * kLn2;
  if (status && a.dev_status) atomicOr(a.dev_status, status);
}

cudaError_t launch_general(const AttnArgs& a, cudaStream_t st) {
  int lanes = 1;
  while (lanes * 8 < a.cache.head_dim) lanes *= 2;
  const int64_t blocks = a.n_nodes * a.n_q_heads;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  attention_general_kernel<<<static_cast<unsigned>(blocks), kGWarps * 32, 0, st>>>(a, lanes);
  return cudaGetLastError();
}

}  // namespace

size_t attn_workspace_bytes(int64_t, int, int, int, int) { return 0; }

cudaError_t launch_attention(const AttnArgs& a, int, int, cudaStream_t st) {
  return launch_general(a, st);
}

}  // namespace fct
