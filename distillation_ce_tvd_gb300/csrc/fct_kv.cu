// The paged key/value cache: new tokens written (and quantised to e4m3 as
// they are), and an accepted path's tokens moved to the front of their tree.
//
// Both are copies: a token's key (value) of one head is read once and written
// once, so the bound is the bytes, and for a few tokens the latency of a launch
// and of loads that depend on one another.  A thread owns 8 elements (16 bytes
// of bf16, 8 of e4m3), the threads of one vector are neighbours in a warp.
#include "fct_common.cuh"
#include "fct_internal.h"

namespace fct {

namespace {

constexpr int kKvThreads = 256;
constexpr int kBlocksPerSm = 8;  // of the write kernel's grid, at most

__device__ __forceinline__ void set_status(int32_t* status, int32_t bit) {
  if (status) atomicOr(status, bit);
}

// ---------------------------------------------------------------- write

// 8 consecutive source elements as loaded (16 bytes of bf16, 32 of fp32), and
// as floats.  A source whose rows are not aligned to 16 bytes goes one element
// at a time.
template <typename T>
struct Raw8 {
  uint4 w[sizeof(T) / 2];
};
template <typename T, bool kVecSrc>
__device__ __forceinline__ Raw8<T> load8(const T* p) {
  Raw8<T> r;
  if constexpr (kVecSrc) {
#pragma unroll
    for (int i = 0; i < int(sizeof(T) / 2); ++i) r.w[i] = reinterpret_cast<const uint4*>(p)[i];
  } else {
    uint32_t b[4 * sizeof(T) / 2];
#pragma unroll
    for (int i = 0; i < int(2 * sizeof(T)); ++i) {
      if constexpr (sizeof(T) == 4)
        b[i] = __float_as_uint(p[i]);
      else
        b[i] = uint32_t(p[2 * i].bits) | (uint32_t(p[2 * i + 1].bits) << 16);
    }
#pragma unroll
    for (int i = 0; i < int(sizeof(T) / 2); ++i)
      r.w[i] = make_uint4(b[4 * i], b[4 * i + 1], b[4 * i + 2], b[4 * i + 3]);
  }
  return r;
}
template <typename T>
__device__ __forceinline__ void floats8(const Raw8<T>& r, float (&x)[8]) {
  if constexpr (sizeof(T) == 2) {
    Elem<bf16_t>::unpack(r.w[0], x);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      x[4 * i] = __uint_as_float(r.w[i].x);
      x[4 * i + 1] = __uint_as_float(r.w[i].y);
      x[4 * i + 2] = __uint_as_float(r.w[i].z);
      x[4 * i + 3] = __uint_as_float(r.w[i].w);
    }
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

// Where things are in the division of a call over threads.  A token's places
// are (key or value, head, 8 elements), `lanes` (a power of two, head_dim / 8
// rounded up) of them to a vector; a block takes `tokens` tokens at a time and
// blockIdx.y its share of the places where a token has more than a block.
struct WriteShape {
  int lanes, places, tokens;
};

// page * a + offset * b of a slot, the division in 32 bits where they hold it.
struct Slot {
  int64_t page;
  int offset;
};
__device__ __forceinline__ Slot slot_of(int64_t slot, int page_size) {
  if ((slot >> 32) == 0) {
    const uint32_t s = static_cast<uint32_t>(slot), p = s / static_cast<uint32_t>(page_size);
    return Slot{p, static_cast<int>(s - p * static_cast<uint32_t>(page_size))};
  }
  const int64_t p = slot / page_size;
  return Slot{p, static_cast<int>(slot - p * page_size)};
}

// kTokens tokens per thread at a time; the next ones' loads are under way while
// these are written, in a grid of at most kBlocksPerSm blocks per SM (four of the
// two-token kernels, with 56 registers, are resident at a time, so that a large
// call runs in two waves).  At 16389 tokens of 8 heads of 128 in bf16: into a
// bf16 cache 25 us (134 MB, 5.5 TB/s), into e4m3 31 us (101 MB, 3.3 TB/s); in
// fp32 34 us into either (201 and 168 MB, 5.9 and 4.9 TB/s); one block per token
// took 33 and 40 us from bf16, four tokens at a time into e4m3 33.
template <typename T, bool kVecSrc, bool kE4m3, int kTokens>
__global__ void __launch_bounds__(kKvThreads) kv_write_kernel(const __grid_constant__ KvWriteArgs a,
                                                              WriteShape w) {
  const int own = threadIdx.x / w.places;  // which of the block's tokens at once
  const int place = blockIdx.y * kKvThreads + threadIdx.x - own * w.places;
  const int vec = place / w.lanes, sub = place - vec * w.lanes;
  const bool is_v = vec >= a.cache.n_heads;
  const int head = is_v ? vec - a.cache.n_heads : vec;
  // (threads without a place take part in the shuffles)
  const bool mine = own < w.tokens && place < w.places && sub * 8 < a.cache.head_dim;
  const T* src = static_cast<const T*>(is_v ? a.v : a.k) + head * a.ld_head + sub * 8;
  const int64_t held = a.cache.num_pages * a.cache.page_size;
  const int64_t step = int64_t(gridDim.x) * w.tokens * kTokens;
  void* pool = is_v ? a.cache.v : a.cache.k;
  int64_t first = int64_t(blockIdx.x) * w.tokens * kTokens;
  Raw8<T> raw[kTokens];
  int64_t slot[kTokens];
  auto load = [&](int64_t from) {
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
      const int64_t token = from + own + i * w.tokens;
      slot[i] = -1;
      raw[i] = Raw8<T>{};
      if (mine && token < a.n_tokens) {
        slot[i] = a.slots[token];
        raw[i] = load8<T, kVecSrc>(src + token * a.ld_token);
      }
    }
  };
  load(first);
  for (; first < a.n_tokens; first += step) {
    Raw8<T> now[kTokens];
    int64_t to[kTokens];
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
      now[i] = raw[i];
      to[i] = slot[i];
    }
    if (first + step < a.n_tokens) load(first + step);
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
      if (to[i] >= held) {
        set_status(a.dev_status, FCT_DEV_INDEX_OUT_OF_RANGE);
        to[i] = -1;
      }
      float x[8];
      floats8<T>(now[i], x);
      const Slot s = slot_of(to[i] < 0 ? 0 : to[i], a.cache.page_size);
      const int64_t at = s.page * a.cache.page_stride + s.offset * a.cache.slot_stride +
                         head * a.cache.head_stride + sub * 8;
      if constexpr (!kE4m3) {
        if (to[i] >= 0)
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(pool) + at) = Elem<bf16_t>::pack(x);
      } else {
        // |x| as bits orders like |x|, and puts infinities and NaNs on top
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) top = max(top, __float_as_uint(x[k]) & 0x7fffffffu);
        for (int k = w.lanes / 2; k >= 1; k >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, k));
        const bool finite = top < 0x7f800000u;
        const int e = finite ? e4m3_exponent(top) : 0;
        const float mul = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);  // 2^-e, exact
        uint32_t out[2] = {0, 0};
        if (finite) {
#pragma unroll
          for (int k = 0; k < 8; k += 2)
            out[k / 4] |= pack_e4m3x2(x[k] * mul, x[k + 1] * mul) << (8 * (k % 4));
        }
        if (to[i] >= 0) {
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(pool) + at) = make_uint2(out[0], out[1]);
          if (sub == 0)
            (is_v ? a.cache.v_scale : a.cache.k_scale)[s.page * a.cache.scale_page_stride +
                                                       s.offset * a.cache.scale_slot_stride +
                                                       head * a.cache.scale_head_stride] =
                finite ? static_cast<uint8_t>(e + 127) : uint8_t(255);
        }
      }
    }
  }
}

template <typename T, bool kVecSrc, int kTokens>
cudaError_t write_tokens(const KvWriteArgs& a, const WriteShape& w, int sms, cudaStream_t st) {
  const int64_t per_block = int64_t(w.tokens) * kTokens;
  int64_t blocks = (a.n_tokens + per_block - 1) / per_block;
  if (blocks > int64_t(sms) * kBlocksPerSm) blocks = int64_t(sms) * kBlocksPerSm;
  const int64_t shares = (w.places + kKvThreads - 1) / kKvThreads;
  if (shares > 65535) return cudaErrorInvalidConfiguration;
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(shares));
  if (a.cache.dtype == FCT_E4M3)
    kv_write_kernel<T, kVecSrc, true, kTokens><<<grid, kKvThreads, 0, st>>>(a, w);
  else
    kv_write_kernel<T, kVecSrc, false, kTokens><<<grid, kKvThreads, 0, st>>>(a, w);
  return cudaGetLastError();
}

template <typename T, bool kVecSrc>
cudaError_t write_typed(const KvWriteArgs& a, int sms, cudaStream_t st) {
  WriteShape w{1, 0, 1};
  while (w.lanes * 8 < a.cache.head_dim) w.lanes *= 2;
  w.places = 2 * a.cache.n_heads * w.lanes;
  if (w.places < kKvThreads) w.tokens = kKvThreads / w.places;
  // several tokens per thread once every SM has its share of threads without
  constexpr int kMost = sizeof(T) == 2 ? 2 : 1;
  return a.n_tokens * w.places >= int64_t(sms) * kKvThreads * kBlocksPerSm
             ? write_tokens<T, kVecSrc, kMost>(a, w, sms, st)
             : write_tokens<T, kVecSrc, 1>(a, w, sms, st);
}

// ---------------------------------------------------------------- move

// A request's position as page and slot, or page -1 where the table or the
// pool does not hold it.
__device__ __forceinline__ Slot place(const KvMoveArgs& a, int64_t b, int64_t pos) {
  if (pos < 0) return Slot{-1, 0};
  const Slot s = slot_of(pos, a.cache.page_size);
  if (s.page >= a.pages.max_pages) return Slot{-1, 0};
  const int64_t id = a.pages.table[b * a.pages.ld + s.page];
  return Slot{id < 0 || id >= a.cache.num_pages ? -1 : id, s.offset};
}

// One thread moves one 8-element column (or one scale byte) of a request: it
// is the only one to touch that column's bytes, and it reads up to kMoveStep
// tokens before it writes any.  Paths ascend with path[j] >= j + 1, so a
// later step's source lies past every earlier destination, and a step's
// sources are read before its destinations are written.  Where the step's
// tokens lie is looked up once per block, by one thread each.  Latency is what
// a call costs (a count, a path, a table entry and the data follow one another).
constexpr int kMoveStep = 8;
struct Moves {
  Slot from[kMoveStep], to[kMoveStep];
  int n;  // tokens of this step, up to the first that is not valid
};

template <typename W>
__device__ __forceinline__ void move_column(const Moves& m, void* pool, int64_t col, int64_t ps, int64_t ss) {
  uint8_t* base = static_cast<uint8_t*>(pool) + col;
  W held[kMoveStep];
#pragma unroll
  for (int s = 0; s < kMoveStep; ++s)
    if (s < m.n) held[s] = *reinterpret_cast<const W*>(base + m.from[s].page * ps + m.from[s].offset * ss);
#pragma unroll
  for (int s = 0; s < kMoveStep; ++s)
    if (s < m.n) *reinterpret_cast<W*>(base + m.to[s].page * ps + m.to[s].offset * ss) = held[s];
}

__global__ void __launch_bounds__(kKvThreads) kv_move_kernel(const __grid_constant__ KvMoveArgs a,
                                                             int blocks_per_request) {
  __shared__ Moves moves;
  const fct_kv_cache& c = a.cache;
  const int64_t b = blockIdx.x / blocks_per_request;
  const int64_t start = a.pages.context_len[b];
  int64_t n = a.count[b];
  if (n < 0 || n > a.path_len) {
    set_status(a.dev_status, FCT_DEV_INDEX_OUT_OF_RANGE);
    n = n < 0 ? 0 : a.path_len;
  }
  const int32_t* path = a.path + b * a.ld_path;
  const int per_head = c.head_dim / 8;
  const int columns = 2 * c.n_heads * per_head;  // of K and V; then one per scale
  int i = static_cast<int>(blockIdx.x % blocks_per_request) * kKvThreads + threadIdx.x;
  for (int64_t j0 = 0; j0 < n; j0 += kMoveStep) {
    if (threadIdx.x < 32) {
      const int64_t j = j0 + threadIdx.x;
      bool ok = true;
      if (threadIdx.x < kMoveStep && j < n) {
        const int64_t node = path[j];
        ok = start >= 0 && node >= j + 1 && (j == 0 || node > path[j - 1]);
        const Slot from = place(a, b, ok ? start + node : -1), to = place(a, b, ok ? start + 1 + j : -1);
        ok = ok && from.page >= 0 && to.page >= 0;
        if (!ok) set_status(a.dev_status, FCT_DEV_INDEX_OUT_OF_RANGE);
        moves.from[threadIdx.x] = from;
        moves.to[threadIdx.x] = to;
      }
      const unsigned bad = __ballot_sync(0xffffffffu, !ok);
      const int most = n - j0 < kMoveStep ? static_cast<int>(n - j0) : kMoveStep;
      if (threadIdx.x == 0) moves.n = bad ? __ffs(bad) - 1 : most;
    }
    __syncthreads();
    if (i < columns) {
      const int at = i >= columns / 2 ? i - columns / 2 : i;
      void* pool = i >= columns / 2 ? c.v : c.k;
      const int64_t e = c.dtype == FCT_E4M3 ? 1 : 2;
      const int64_t col = ((at / per_head) * c.head_stride + (at % per_head) * 8) * e;
      if (c.dtype == FCT_E4M3)
        move_column<uint2>(moves, pool, col, c.page_stride, c.slot_stride);
      else
        move_column<uint4>(moves, pool, col, c.page_stride * e, c.slot_stride * e);
    } else if (c.dtype == FCT_E4M3 && i < columns + 2 * c.n_heads) {
      const int at = i - columns;
      const bool is_v = at >= c.n_heads;
      move_column<uint8_t>(moves, is_v ? c.v_scale : c.k_scale,
                           (is_v ? at - c.n_heads : at) * c.scale_head_stride, c.scale_page_stride,
                           c.scale_slot_stride);
    }
    if (moves.n < kMoveStep) return;  // (the same for every thread)
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_kv_write(const KvWriteArgs& a, int sms, cudaStream_t st) {
  const size_t e = a.src_dtype == FCT_F32 ? 4 : 2;
  auto rows16 = [&](const void* p) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (size_t(a.ld_token) * e) % 16 == 0 &&
           (size_t(a.ld_head) * e) % 16 == 0;
  };
  const bool vec = rows16(a.k) && rows16(a.v);
  if (a.src_dtype == FCT_F32)
    return vec ? write_typed<float, true>(a, sms, st) : write_typed<float, false>(a, sms, st);
  return vec ? write_typed<bf16_t, true>(a, sms, st) : write_typed<bf16_t, false>(a, sms, st);
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
