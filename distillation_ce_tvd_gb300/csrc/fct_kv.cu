// The paged key/value cache: new tokens written (and quantised to e4m3 as
// they are), and an accepted path's tokens moved to the front of their tree.
//
// Both are copies: a token's key (value) of one head is read once and written
// once, so the bound is the bytes.  A thread owns 8 elements (16 bytes of
// bf16, 8 of e4m3), the threads of one vector are neighbours in a warp.
#include "fct_common.cuh"
#include "fct_internal.h"

namespace fct {

namespace {

constexpr int kKvThreads = 256;

__device__ __forceinline__ void set_status(int32_t* status, int32_t bit) {
  if (status) atomicOr(status, bit);
}

// ---------------------------------------------------------------- write

// 8 consecutive source elements as floats.  A bf16 vector is 16 bytes and an
// fp32 one 32; a source whose rows are not aligned to that goes one element
// at a time.
template <typename T, bool kVecSrc>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
  if constexpr (!kVecSrc) {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = Elem<T>::load1(p + j);
  } else if constexpr (Elem<T>::kVec == 8) {
    Elem<T>::unpack(*reinterpret_cast<const uint4*>(p), x);
  } else {
    const float4 a = *reinterpret_cast<const float4*>(p);
    const float4 b = *reinterpret_cast<const float4*>(p + 4);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
}

// Two floats to e4m3, lo in the lower byte, round to nearest even.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// The smallest e >= -126 with amax <= 448 * 2^e = 1.75 * 2^(e + 8), from the
// bits of a finite amax >= 0.
__device__ __forceinline__ int e4m3_exponent(uint32_t amax_bits) {
  const int top = static_cast<int>(amax_bits >> 23) - 127;
  const int e = (amax_bits & 0x7fffffu) <= 0x600000u ? top - 8 : top - 7;
  return e < -126 ? -126 : e;
}

// Vector i of the call is (token, key or value, head), heads fastest, so that
// neighbouring vectors are neighbours in both the source and the cache.
// `lanes` (a power of two, head_dim / 8 rounded up) threads share one.
template <typename T, bool kVecSrc, bool kE4m3>
__global__ void __launch_bounds__(kKvThreads) kv_write_kernel(KvWriteArgs a, int lanes) {
  const int sub = threadIdx.x % lanes;
  const int64_t per_block = kKvThreads / lanes;
  const int64_t total = a.n_tokens * 2 * a.cache.n_heads;
  const int64_t i = blockIdx.x * per_block + threadIdx.x / lanes;
  const bool live = i < total && sub * 8 < a.cache.head_dim;
  const uint32_t both = static_cast<uint32_t>(i % (2 * a.cache.n_heads));
  const int64_t token = i / (2 * a.cache.n_heads);
  const bool is_v = both >= static_cast<uint32_t>(a.cache.n_heads);
  const int64_t head = is_v ? both - a.cache.n_heads : both;
  int64_t slot = live ? a.slots[token] : -1;
  if (slot >= a.cache.num_pages * a.cache.page_size) {
    set_status(a.dev_status, FCT_DEV_INDEX_OUT_OF_RANGE);
    slot = -1;
  }
  float x[8] = {};
  if (slot >= 0)
    load8<T, kVecSrc>(static_cast<const T*>(is_v ? a.v : a.k) + token * a.ld_token +
                          head * a.ld_head + sub * 8,
                      x);
  const int64_t page = slot / a.cache.page_size, off = slot % a.cache.page_size;
  const int64_t at = page * a.cache.page_stride + off * a.cache.slot_stride +
                     head * a.cache.head_stride + sub * 8;
  void* pool = is_v ? a.cache.v : a.cache.k;
  if constexpr (!kE4m3) {
    if (slot >= 0) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(pool) + at) = Elem<bf16_t>::pack(x);
  } else {
    // |x| as bits orders like |x|, and puts infinities and NaNs on top
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(x[j]) & 0x7fffffffu);
    for (int k = lanes / 2; k >= 1; k >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, k));
    const bool finite = top < 0x7f800000u;
    const int e = finite ? e4m3_exponent(top) : 0;
    const float mul = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);  // 2^-e, exact
    uint32_t w[2] = {0, 0};
    if (finite) {
#pragma unroll
      for (int j = 0; j < 8; j += 2)
        w[j / 4] |= pack_e4m3x2(x[j] * mul, x[j + 1] * mul) << (8 * (j % 4));
    }
    if (slot >= 0) {
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(pool) + at) = make_uint2(w[0], w[1]);
      if (sub == 0)
        (is_v ? a.cache.v_scale : a.cache.k_scale)[page * a.cache.scale_page_stride +
                                                   off * a.cache.scale_slot_stride +
                                                   head * a.cache.scale_head_stride] =
            finite ? static_cast<uint8_t>(e + 127) : uint8_t(255);
    }
  }
}

template <typename T, bool kVecSrc>
cudaError_t write_typed(const KvWriteArgs& a, cudaStream_t st) {
  int lanes = 1;
  while (lanes * 8 < a.cache.head_dim) lanes *= 2;
  const int64_t per_block = kKvThreads / lanes;
  const int64_t blocks = (a.n_tokens * 2 * a.cache.n_heads + per_block - 1) / per_block;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  if (a.cache.dtype == FCT_E4M3)
    kv_write_kernel<T, kVecSrc, true><<<static_cast<unsigned>(blocks), kKvThreads, 0, st>>>(a, lanes);
  else
    kv_write_kernel<T, kVecSrc, false><<<static_cast<unsigned>(blocks), kKvThreads, 0, st>>>(a, lanes);
  return cudaGetLastError();
}

// ---------------------------------------------------------------- move

// The pool offset (in units of the given strides) of a request's position, or
// -1 where the table or the pool does not hold it.
__device__ __forceinline__ int64_t place(const KvMoveArgs& a, int64_t b, int64_t pos, int64_t ps,
                                         int64_t ss) {
  const int64_t page = pos / a.cache.page_size;
  if (pos < 0 || page >= a.pages.max_pages) return -1;
  const int64_t id = a.pages.table[b * a.pages.ld + page];
  if (id < 0 || id >= a.cache.num_pages) return -1;
  return id * ps + (pos % a.cache.page_size) * ss;
}

// One thread moves one 8-element column (or one scale byte) of a request: it
// is the only one to touch that column's bytes, and it reads up to kMoveStep
// tokens before it writes any.  Paths ascend with path[j] >= j + 1, so a
// later step's source lies past every earlier destination, and a step's
// sources are read before its destinations are written.
constexpr int kMoveStep = 8;

template <typename W>
__device__ __forceinline__ void move_column(const KvMoveArgs& a, int64_t b, int64_t n, W* pool,
                                            int64_t col, int64_t ps, int64_t ss) {
  const int64_t start = a.pages.context_len[b];
  const int32_t* path = a.path + b * a.ld_path;
  for (int64_t j0 = 0; j0 < n; j0 += kMoveStep) {
    W held[kMoveStep];
    int64_t to[kMoveStep];
    bool stop = false;
#pragma unroll
    for (int s = 0; s < kMoveStep; ++s) {
      const int64_t j = j0 + s;
      to[s] = -1;
      if (j >= n || stop) continue;
      const int64_t from_node = path[j];
      const bool ok = from_node >= j + 1 && (j == 0 || from_node > path[j - 1]);
      const int64_t from = ok && start >= 0 ? place(a, b, start + from_node, ps, ss) : -1;
      const int64_t dest = ok && start >= 0 ? place(a, b, start + 1 + j, ps, ss) : -1;
      if (from < 0 || dest < 0) {
        set_status(a.dev_status, FCT_DEV_INDEX_OUT_OF_RANGE);
        stop = true;
      } else if (from_node != j + 1) {
        held[s] = *reinterpret_cast<const W*>(reinterpret_cast<const uint8_t*>(pool) + col + from);
        to[s] = dest;
      }
    }
#pragma unroll
    for (int s = 0; s < kMoveStep; ++s)
      if (to[s] >= 0) *reinterpret_cast<W*>(reinterpret_cast<uint8_t*>(pool) + col + to[s]) = held[s];
    if (stop) return;
  }
}

__global__ void __launch_bounds__(kKvThreads) kv_move_kernel(KvMoveArgs a, int blocks_per_request) {
  const fct_kv_cache& c = a.cache;
  const int64_t b = blockIdx.x / blocks_per_request;
  int64_t n = a.count[b];
  if (n < 0 || n > a.path_len) {
    set_status(a.dev_status, FCT_DEV_INDEX_OUT_OF_RANGE);
    n = n < 0 ? 0 : a.path_len;
  }
  const int per_head = c.head_dim / 8;
  const int columns = 2 * c.n_heads * per_head;  // of K and V; then one per scale
  int i = static_cast<int>(blockIdx.x % blocks_per_request) * kKvThreads + threadIdx.x;
  if (i < columns) {
    const bool is_v = i >= columns / 2;
    if (is_v) i -= columns / 2;
    const int64_t e = c.dtype == FCT_E4M3 ? 1 : 2;
    const int64_t col = ((i / per_head) * c.head_stride + (i % per_head) * 8) * e;
    if (c.dtype == FCT_E4M3)
      move_column(a, b, n, static_cast<uint2*>(is_v ? c.v : c.k), col, c.page_stride,
                  c.slot_stride);
    else
      move_column(a, b, n, static_cast<uint4*>(is_v ? c.v : c.k), col, c.page_stride * e,
                  c.slot_stride * e);
  } else if (c.dtype == FCT_E4M3 && i < columns + 2 * c.n_heads) {
    i -= columns;
    const bool is_v = i >= c.n_heads;
    if (is_v) i -= c.n_heads;
    move_column(a, b, n, is_v ? c.v_scale : c.k_scale, i * c.scale_head_stride,
                c.scale_page_stride, c.scale_slot_stride);
  }
}

}  // namespace

cudaError_t launch_kv_write(const KvWriteArgs& a, cudaStream_t st) {
  const size_t e = a.src_dtype == FCT_F32 ? 4 : 2;
  auto rows16 = [&](const void* p) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (size_t(a.ld_token) * e) % 16 == 0 &&
           (size_t(a.ld_head) * e) % 16 == 0;
  };
  const bool vec = rows16(a.k) && rows16(a.v);
  if (a.src_dtype == FCT_F32)
    return vec ? write_typed<float, true>(a, st) : write_typed<float, false>(a, st);
  return vec ? write_typed<bf16_t, true>(a, st) : write_typed<bf16_t, false>(a, st);
}

cudaError_t launch_kv_move(const KvMoveArgs& a, cudaStream_t st) {
  const int64_t columns = int64_t(2) * a.cache.n_heads * (a.cache.head_dim / 8) +
                          (a.cache.dtype == FCT_E4M3 ? 2 * a.cache.n_heads : 0);
  const int64_t per = (columns + kKvThreads - 1) / kKvThreads;
  if (per * a.pages.batch > 0x7fffffff) return cudaErrorInvalidConfiguration;
  kv_move_kernel<<<static_cast<unsigned>(per * a.pages.batch), kKvThreads, 0, st>>>(
      a, static_cast<int>(per));
  return cudaGetLastError();
}

}  // namespace fct
