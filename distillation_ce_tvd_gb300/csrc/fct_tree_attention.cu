// Attention of drafted trees (and of single tokens) over a paged cache; the
// operation is described in include/fused_ce_tvd.h, fct_tree_attention.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_fp16.h>

#include <mutex>

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
// Every query head of every node reads its keys for itself, so what bounds it
// is loads and CUDA-core arithmetic: 48 requests x 5 nodes, 32 query and 8 kv
// heads of 128, 450 to 8190 keys in bf16 took it 4.7 ms.

constexpr int kGWarps = 4;

// Four e4m3 payloads.
__device__ __forceinline__ float4 e4m3_floats(uint32_t w) {
  uint32_t lo, hi;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"(static_cast<uint16_t>(w)));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"(static_cast<uint16_t>(w >> 16)));
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  return make_float4(a.x, a.y, b.x, b.y);
}

// 8 elements of a cached vector, payload only.
__device__ __forceinline__ void load_cached(const void* pool, int dtype, int64_t at, float (&x)[8]) {
  if (dtype == FCT_BF16) {
    Elem<bf16_t>::unpack(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(pool) + at), x);
  } else {
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(pool) + at);
#pragma unroll
    for (int j = 0; j < 8; j += 4) {
      const float4 f = e4m3_floats(j < 4 ? w.x : w.y);
      x[j] = f.x;
      x[j + 1] = f.y;
      x[j + 2] = f.z;
      x[j + 3] = f.w;
    }
  }
}

// 2^(byte - 127), NaN for byte 255.
__device__ __forceinline__ float scale_of(uint8_t byte) {
  return byte == 255 ? __int_as_float(0x7fc00000)
                     : byte == 0 ? __int_as_float(0x00400000) : __uint_as_float(uint32_t(byte) << 23);
}
// From this byte on a payload times its scale can be 2^128 or more, which reads
// as an infinity.
constexpr int kLargeScale = 247;

// Whether node_start[b] .. node_start[b + 1] is not a range of the nodes, or is
// the first (last) and does not start at 0 (end at n_nodes).
__device__ __forceinline__ bool bad_nodes(const AttnArgs& a, int64_t b) {
  const int64_t n0 = a.node_start[b], n1 = a.node_start[b + 1];
  return n0 < 0 || n1 > a.n_nodes || n1 < n0 || (b == 0 && n0 != 0) ||
         (b == a.pages.batch - 1 && n1 != a.n_nodes);
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
  if (blockIdx.x == 0) {
    bool bad = false;
    for (int64_t r = threadIdx.x; r < a.pages.batch; r += kGWarps * 32) bad |= bad_nodes(a, r);
    if (bad && a.dev_status) atomicOr(a.dev_status, FCT_DEV_INDEX_OUT_OF_RANGE);
  }
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
    float s = 0.f, ks = 1.f, vs = 1.f;
    if (e && sees) {
      ks = scale_of(c.k_scale[sc]);
      vs = scale_of(c.v_scale[sc]);
      if (max(c.k_scale[sc], c.v_scale[sc]) >= kLargeScale) {
#pragma unroll
        for (int d = 0; d < 8; ++d) {
          k[d] *= ks;
          v[d] *= vs;
        }
        ks = vs = 1.f;
      }
    }
#pragma unroll
    for (int d = 0; d < 8; ++d) s = fmaf(q[d], k[d], s);
    for (int x = lanes / 2; x >= 1; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= ks;
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

// ---------------------------------------------------------------- tensor cores
//
// head_dim 64 and 128 over pages of whole 8-token rows.  The rows of a kv
// head's query tile are the (node, query head of the group) pairs: every key
// is read once for all of them.
//
//   S = Q K^T  (128 rows x 128 keys, fp32 in tensor memory, tcgen05.mma)
//   P = 2^(S * scale * log2 e - m) as two bf16, over S's own columns
//   O += P V   (P from tensor memory, V as it lies in the cache: MN-major)
//
// A weight goes through the second product as its bf16 value and the bf16 of
// what that rounding left, 16 bits together: with the first alone an output is
// off by up to 2^-8 of the largest weight's value, at any number of keys.
//
// A unit of work is a request, a kv head and up to 256 rows; its keys come in
// tiles of 128.  A unit of at most 128 rows gives its even key tiles to
// softmax group A and its odd ones to group B, each with an S and an O of its
// own (merged at the end), so that one group's softmax runs beside the other's
// products; a larger unit gives each group 128 of its rows and every tile.
// All key tiles of all units, in order, are dealt to the CTAs (one per SM) in
// equal runs, whatever the requests' lengths; a unit cut between CTAs leaves
// partial sums in the workspace, which combine_kernel adds in order.
//
// What bounds it: with few rows the bytes of the keys (1 x 8 nodes, 32 query
// and 8 kv heads of 128, 131071 keys in bf16: 537 MB in 99 us, 5.4 TB/s; 48
// requests x 5 nodes, 870 MB: 155-168 us); with 256 rows per unit a call's fixed
// cost of some 50 us and 2.4 us per tile (12 x 64 nodes, 64 query heads: 118
// GFLOP, 177 with the remainders, in 181 us); in e4m3 the conversion, the scale
// bytes and the hand-over of tiles between the roles, 2.2 us per tile (20 x 27
// nodes, 400 MB: 218 us, 1.8 TB/s).  One bf16 per weight took 148, 203 and 161
// us where two took 159, 207 and 187 (48 x 5, 20 x 27, 12 x 64).
//
// Per CTA: warp 1 issues the products, warps 4-7 and 8-11 are the softmax
// groups.  bf16: warps 0 and 3 load K and V tiles by TMA (one box per page
// piece), warp 2 prepares the tiles past the context.  e4m3: warp 0 loads,
// warps 2 and 3 fetch the scale bytes, warps 12-19 prepare every tile: they make
// it bf16 (exact: payload times a power of two) in its slot, since a row of 128
// payload bytes lands where that row's second half of bf16 goes, and one warp
// reads and writes the row; a row of 64 lands behind the slot's tile.  Preparing
// clears what must not reach a product from the tiles past the context (slots
// past the end, and non-finite values of drafted nodes, which are added back
// to the rows that see them).

constexpr int kTile = 128;      // keys per tile, rows per query tile
constexpr int kSoftWarps = 8;
constexpr int kUnitRows = 2 * kTile;
constexpr int kBadRing = 16;
constexpr uint32_t kAtTmemCols = 512;
// O is rescaled when the scores' maximum passes the weights' offset, which is
// then put 2^8 above it: a weight is never more than 1, so that O overflows no
// earlier than the values do.
constexpr float kLazyLog2 = 8.f;

template <int kD, bool kFp8>
struct AttnShape {
  // Warps: 0 loads, 1 products, 4-11 softmax; e4m3: 2 and 3 fetch scale bytes,
  // 12-19 prepare; bf16: 2 prepares, 3 loads V (0 loads K).
  static constexpr int kThreads = kFp8 ? 640 : 384;
  static constexpr int kPrepWarp0 = kFp8 ? 12 : 2, kPrepWarps = kFp8 ? 8 : 1;
  static constexpr int kHalves = kD / 64;  // 128-byte column blocks of a bf16 row
  static constexpr uint32_t kTileBytes = kTile * kD * 2;
  // An e4m3 tile lands kRawAt bytes into its slot, in rows of kD bytes.
  static constexpr uint32_t kRawAt = kFp8 ? kTile * 128 : 0;
  static constexpr uint32_t kSlotBytes = kFp8 ? kRawAt + (kD == 128 ? kTile * 128 : kTile * kD) : kTileBytes;
  static_assert(kSlotBytes >= kTileBytes && kSlotBytes % 1024 == 0, "a slot holds a tile");
  static constexpr int kSlots = kD == 128 ? 5 : (kFp8 ? 7 : 8);
  static constexpr int kRaw = kFp8 ? kSlots : 1;    // (1 where unused)
  static constexpr int kTail = kFp8 ? 1 : kSlots;
  static constexpr size_t kTilesBytes = 2 * kTileBytes + size_t(kSlots) * kSlotBytes;
  // After the tiles (two of Q, the ring of K and V).
  struct Control {
    uint64_t full_bar[kSlots], empty_bar[kSlots];
    // bf16: a V tile past the context lands on tail_full and is handed on by
    // the preparing warp on prep_bar, instead of full_bar
    uint64_t tail_full[kTail], prep_bar[kTail];
    // e4m3: a tile and its scale bytes land on these, and full_bar says that it
    // is bf16
    uint64_t raw_full[kRaw], raw_scaled[kRaw];
    uint64_t s_full[2], p_full[2], q_full, o_full, ml_full, done_bar;
    int64_t sched[4];     // the run: request, offset in it, length; whether units are whole
    float2 ml[2][kTile];  // the groups' maxima and sums, lane by lane
    uint32_t tmem_base;
    int abort_flag;
    int bad_seg[kBadRing];
    uint8_t raw_scale[kRaw][kFp8 ? kTile : 4];
  };
  static constexpr size_t kSmem = kTilesBytes + sizeof(Control);
  static_assert(kSmem <= 227 * 1024, "shared memory of one CTA");
};

// What one CTA does with one unit: key tiles [tile0, tile0 + tiles) of it.
struct Segment {
  int b;
  int h;           // kv head
  int node0;       // first row of q of the request
  int ctx, len;    // tokens before the nodes, and with them
  int row0, rows;  // this unit's rows of the request's nodes * group
  int tile0, tiles;
  bool whole;       // the unit's only segment
  int part;         // else: workspace slot of this CTA (0 its first, 1 its last)
};

struct AttnDims {
  int group;
  int room;  // positions a block table row holds
};

struct RequestShape {
  int node0, nodes;
  int ctx, len, tiles;
  int row_units;
  int last_rows;  // of its last row unit; the others have kUnitRows
  bool bad;
};

__device__ __forceinline__ RequestShape request_shape(const AttnArgs& a, const AttnDims& d, int64_t b) {
  RequestShape r;
  int64_t n0 = a.node_start[b], n1 = a.node_start[b + 1];
  r.bad = bad_nodes(a, b);
  if (n0 < 0 || n1 > a.n_nodes || n1 < n0) n0 = n1 = 0;
  r.node0 = static_cast<int>(n0);
  r.nodes = static_cast<int>(n1 - n0);
  r.ctx = a.pages.context_len[b];
  if (r.ctx < 0) {
    r.bad = true;
    r.ctx = 0;
  }
  const int64_t len = int64_t(r.ctx) + r.nodes;
  r.bad = r.bad || (len > d.room && r.nodes > 0);
  r.len = len > d.room ? d.room : static_cast<int>(len);
  r.tiles = (r.len + kTile - 1) / kTile;
  const int rows = r.nodes * d.group;
  r.row_units = (rows + kUnitRows - 1) / kUnitRows;
  r.last_rows = rows - (r.row_units - 1) * kUnitRows;
  return r;
}

// What the deal counts.  A unit costs start_cost for its start and end (as
// measured with head_dim 128 and one bf16 per weight: 9 us, or 8 bf16 key tiles
// of 128 rows, or 3 of the slower e4m3 ones; not measured for 64) and each of its key tiles 1, or 2 with both query tiles; the sum over
// all units is dealt in equal runs.  48 requests of 450 to 8190 keys in bf16
// took 190 us with a start cost of 3, 173 with 5, 167 with 7, 168 with 9; the
// e4m3 trees 208 with 3, 211 with 5, 215 with 7.  Where no request has more
// than kWholeTiles tiles, a unit counts 1 and is never cut: a second CTA would
// save less than combining costs.
constexpr int kWholeTiles = 4;
__host__ __device__ constexpr int start_cost_of(bool fp8) { return fp8 ? 3 : 8; }

struct Deal {
  bool whole;
  int start_cost;
  // of a unit with `rows` rows of a request with `tiles` tiles
  __device__ __forceinline__ int per_tile(int rows) const { return rows > kTile ? 2 : 1; }
  __device__ __forceinline__ int64_t unit(int tiles, int rows) const {
    return whole ? 1 : start_cost + int64_t(tiles) * per_tile(rows);
  }
  __device__ __forceinline__ int64_t head(const RequestShape& r) const {
    return r.row_units == 0 ? 0
                            : (r.row_units - 1) * unit(r.tiles, kUnitRows) + unit(r.tiles, r.last_rows);
  }
  __device__ __forceinline__ int64_t request(const RequestShape& r, int heads) const {
    return r.tiles == 0 ? 0 : head(r) * heads;
  }
  // The first tile that starts at cost x of the unit or later.
  __device__ __forceinline__ int tile_at(int64_t x, int tiles, int rows) const {
    if (x <= 0 || (!whole && x <= start_cost)) return 0;
    if (whole) return tiles;
    const int per = per_tile(rows);
    const int64_t n = (x - start_cost + per - 1) >> (per - 1);  // per is 1 or 2
    return n < tiles ? static_cast<int>(n) : tiles;
  }
  // How many CTAs share `total`, and where CTA c's run starts.
  __device__ __forceinline__ int64_t runs(int64_t total, int64_t ctas) const {
    const int64_t most = whole ? total : (total + start_cost) / (start_cost + 1);
    return most < ctas ? most : ctas;
  }
  __device__ __forceinline__ static int64_t run_start(int64_t total, int64_t runs, int64_t c) {
    return c >= runs ? total : total * c / runs;
  }
  // Whose run cost x is in.
  __device__ __forceinline__ static int64_t run_of(int64_t total, int64_t runs, int64_t x) {
    return ((x + 1) * runs - 1) / total;
  }
};

// A warp's view of the whole batch: the deal, its total, and for one cost
// `find` the request it falls in and the offset there.
struct Batch {
  Deal deal;
  int64_t total;
  bool bad;
};
__device__ __forceinline__ Batch batch_of(const AttnArgs& a, const AttnDims& d) {
  const int lane = threadIdx.x & 31;
  const int start_cost = start_cost_of(a.cache.dtype == FCT_E4M3);
  int most = 0;
  int64_t cost[2] = {0, 0};
  bool bad = false;
#pragma unroll 2
  for (int64_t b = lane; b < a.pages.batch; b += 32) {
    const RequestShape r = request_shape(a, d, b);
    bad |= r.bad;
    if (r.nodes > 0) most = max(most, r.tiles);
    cost[0] += Deal{false, start_cost}.request(r, a.cache.n_heads);
    cost[1] += Deal{true, start_cost}.request(r, a.cache.n_heads);
  }
#pragma unroll
  for (int k = 16; k >= 1; k >>= 1) {
    most = max(most, __shfl_xor_sync(0xffffffffu, most, k));
    cost[0] += __shfl_xor_sync(0xffffffffu, cost[0], k);
    cost[1] += __shfl_xor_sync(0xffffffffu, cost[1], k);
  }
  const bool whole = most <= kWholeTiles;
  return Batch{Deal{whole, start_cost}, cost[whole ? 1 : 0], __any_sync(0xffffffffu, bad) != 0};
}
// f(before, cost, b, shape) for the request of every lane, 32 at a time,
// until f says (to the whole warp) that it has what it looked for.
template <typename F>
__device__ __forceinline__ void scan_requests(const AttnArgs& a, const AttnDims& d, const Deal& deal, F f) {
  const int lane = threadIdx.x & 31;
  int64_t before = 0;
  for (int64_t b0 = 0; b0 < a.pages.batch; b0 += 32) {
    const int64_t b = b0 + lane;
    RequestShape r{};
    int64_t w = 0;
    if (b < a.pages.batch) {
      r = request_shape(a, d, b);
      w = deal.request(r, a.cache.n_heads);
    }
    int64_t incl = w;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const int64_t o = __shfl_up_sync(0xffffffffu, incl, k);
      if (lane >= k) incl += o;
    }
    if (f(before + incl - w, w, b, r)) return;
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
}

// Walks the segments of a CTA's run; every role of the CTA walks the same.
struct SegmentWalk {
  const AttnArgs& a;
  const AttnDims& d;
  Deal deal;
  int b;
  int64_t off, left;  // cost into request b, and of the run's rest
  RequestShape r;     // of request b
  __device__ __forceinline__ SegmentWalk(const AttnArgs& a_, const AttnDims& d_, Deal deal_, int64_t b_,
                                         int64_t off_, int64_t left_)
      : a(a_), d(d_), deal(deal_), b(static_cast<int>(b_)), off(off_), left(left_) {
    if (left > 0) r = request_shape(a, d, b);
  }
  __device__ __forceinline__ bool next(Segment& s) {
    while (left > 0) {
      const int64_t w = deal.request(r, a.cache.n_heads);
      if (off >= w) {
        off = 0;
        if (++b >= a.pages.batch) return false;
        r = request_shape(a, d, b);
        continue;
      }
      const int64_t head = deal.head(r), full = deal.unit(r.tiles, kUnitRows);
      s.h = static_cast<int>(off / head);
      const int64_t in_head = off - s.h * head;
      const int u = static_cast<int>(min(in_head / full, int64_t(r.row_units - 1)));
      const int64_t x0 = in_head - u * full;
      s.rows = u == r.row_units - 1 ? r.last_rows : kUnitRows;
      const int64_t cost = deal.unit(r.tiles, s.rows);
      const int64_t x1 = min(cost, x0 + left);
      off += x1 - x0;
      left -= x1 - x0;
      s.b = b;
      s.node0 = r.node0;
      s.ctx = r.ctx;
      s.len = r.len;
      s.row0 = u * kUnitRows;
      s.tile0 = deal.tile_at(x0, r.tiles, s.rows);
      s.tiles = (x1 == cost ? r.tiles : deal.tile_at(x1, r.tiles, s.rows)) - s.tile0;
      s.whole = s.tiles == r.tiles;
      s.part = s.tile0 > 0 ? 0 : 1;
      if (s.tiles > 0) return true;
    }
    return false;
  }
};

__device__ __forceinline__ void tc_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void async_fence() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
// The barrier's phase completes when every product issued before has.
__device__ __forceinline__ void umma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   smem_addr(bar))
               : "memory");
}
// Upper half of a tile's shared-memory descriptor: 8-row atoms of 1024 bytes
// (128-byte swizzle), version 1.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);

// D = A B^T (+ D): A and B from shared memory, or A from tensor memory.  The
// descriptors come as their lower halves.
template <uint32_t kIdesc>
__device__ __forceinline__ void umma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(kIdesc), "r"(acc), "n"(kDescHi)
      : "memory");
}
template <uint32_t kIdesc>
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a_tmem, uint32_t b, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 db, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d),
      "r"(a_tmem), "r"(b), "r"(kIdesc), "r"(acc), "n"(kDescHi)
      : "memory");
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t is;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}"
               : "=r"(is));
  return is != 0;
}
// x, known to be the same in all lanes.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

// Instruction descriptor: fp32 accumulator, bf16 operands, M = 128, N; bit 16
// marks an MN-major B.
__host__ __device__ constexpr uint32_t attn_idesc(int n, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(b_mn) << 16) | (uint32_t(n >> 3) << 17) |
         (uint32_t(kTile >> 4) << 24);
}
// Lower half of a tile's descriptor: its address and, for an MN-major tile (V:
// rows are keys), the distance to the next 64 columns, one kTile x 128-byte
// block.
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, bool mn) {
  return ((saddr & 0x3FFFFu) >> 4) | ((mn ? uint32_t(kTile * 128) >> 4 : 1u) << 16);
}

#define FCT_R32(r)                                                                              \
  "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),            \
      "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),    \
      "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), \
      "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), \
      "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
#define FCT_RW32(r)                                                                             \
  "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),            \
      "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]),    \
      "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]),              \
      "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]),              \
      "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
#define FCT_U32(r)                                                                              \
  "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),        \
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),          \
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),        \
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),        \
      "r"(r[29]), "r"(r[30]), "r"(r[31])

// 32 columns of tensor memory, one lane per thread of the warp.  The wait has
// the registers as operands, so that no use of them comes before it.
__device__ __forceinline__ void tm_ld(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : FCT_R32(r)
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" : FCT_RW32(r)::"memory");
}
__device__ __forceinline__ void tm_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(r[0]), "r"(r[1]),
      "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tm_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
      "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tm_st(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::FCT_U32(r),
      "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tm_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Whether a phase has completed; the thread may be suspended for some
// microseconds before the answer is no, so that waiting warps leave the issue
// slots to the others.
__device__ __forceinline__ bool mbar_try_long(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 q, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity), "r"(20000u)
      : "memory");
  return done != 0;
}
// mbar_wait without a function call.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, volatile int* abort,
                                           bool heed_abort = true) {
  const uint32_t at = smem_addr(bar);
  if (mbar_try_long(at, parity)) return true;
  const long long t0 = clock64();
  do {
    if (heed_abort && *abort) return false;
    if (mbar_try_long(at, parity)) return true;
  } while (clock64() - t0 <= kWaitLimitCycles);
  *abort = 1;
  return false;
}
// A warp waits for a phase and agrees on the outcome.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return __all_sync(0xffffffffu, wait_phase(bar, parity, abort));
}
// A warp's arrival, after what all its lanes have done.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// A box of a 4-D tensor map (head_dim, slot, head, page).
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int x, int slot, int head,
                                        int page, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(slot), "r"(head), "r"(page),
      "r"(smem_addr(bar))
      : "memory");
}

// 32 bits of a node's mask from bit s on (s >= 0).
__device__ __forceinline__ uint32_t mask_bits(const int64_t* words, int64_t n_words, int s) {
  const int i = s >> 6, sh = s & 63;
  const uint64_t lo = i < n_words ? static_cast<uint64_t>(words[i]) : 0;
  const uint64_t hi = sh && i + 1 < n_words ? static_cast<uint64_t>(words[i + 1]) << (64 - sh) : 0;
  return static_cast<uint32_t>((lo >> sh) | hi);
}

// Which of the 32 keys from position p0 on node i of the segment sees.
__device__ __forceinline__ uint32_t visible32(const AttnArgs& a, const Segment& s, int node, int p0) {
  const int first = p0 - s.ctx;  // node index of the first key, or < 0
  uint32_t m;
  if (first + 32 <= 0) {
    m = 0xffffffffu;
  } else {
    const int from = max(first, 0);
    if (a.mask == nullptr) {
      const int n = node - from + 1;
      m = n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
    } else {
      m = mask_bits(a.mask + int64_t(s.node0 + node) * a.mask_words, a.mask_words, from);
    }
    if (first < 0) m = (m << -first) | ((1u << -first) - 1u);
  }
  const int held = s.len - p0;
  if (held < 32) m &= held <= 0 ? 0u : (1u << held) - 1u;
  return m;
}

// A bf16 pair without its infinities and NaNs; whether it had any.
__device__ __forceinline__ bool drop_non_finite(uint32_t& x) {
  const bool lo = (x & 0x7f80u) == 0x7f80u, hi = (x & 0x7f800000u) == 0x7f800000u;
  if (lo) x &= 0xffff0000u;
  if (hi) x &= 0x0000ffffu;
  return lo || hi;
}

// The pool's page and slot of a position; the page may be outside the pool
// (the table is the caller's).
__device__ __forceinline__ int page_of(const AttnArgs& a, const Segment& s, int pos, int* slot) {
  const int p = pos / a.cache.page_size;
  *slot = pos - p * a.cache.page_size;
  return a.pages.table[s.b * a.pages.ld + p];
}

// Order in which a segment's K and V tiles are used (and loaded): K runs
// `lead` tiles ahead of V.  f(is_v, tile) for each.
// (One loop with one call: the roles' bodies are long, and all of them share
// the instruction cache.)
template <typename F>
__device__ __forceinline__ void for_items(int tiles, int lead, F f) {
  const int ahead = min(lead, tiles), paired = 2 * (tiles - ahead);
#pragma unroll 1
  for (int n = 0; n < 2 * tiles; ++n) {
    const int m = n - ahead;
    const bool is_v = m >= 0 && (m >= paired || !(m & 1));
    const int j = m < 0 ? n : m >= paired ? m - paired / 2 : (m >> 1) + (is_v ? 0 : ahead);
    if (!f(is_v, j)) return;
  }
}

// Two e4m3 (bytes 1 and 3 of w, the others 0) to bf16, times 2^-120.
__device__ __forceinline__ uint32_t e4m3_bits(uint32_t w) {
  return ((w >> 4) & 0x07f007f0u) | (w & 0x80008000u);
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}

// One key tile of a softmax warp: `chunks` (1, 2 or 4) chunks of 32 keys from
// chunk0 on are its share, of the rows of its 32 lanes.  S's columns become
// P's (per chunk 16 of the weights in bf16 and 16 of what the rounding left);
// the chunks of other warps, which hold the same rows, become zero.  One chunk
// is held at a time (S is read twice where there are more), in loops that stay
// small: the roles of a CTA share one instruction cache.
template <int kD>
__device__ __forceinline__ void soft_tile(const AttnArgs& a, const Segment& seg, uint32_t tm_s,
                                          uint32_t tm_o, int chunk0, int chunks, int node, bool live,
                                          int p0, bool tail, bool first, float sl2, float& m, float& l) {
  uint32_t x[32];
  auto load = [&](int i) {
    tm_ld(tm_s + 32 * (chunk0 + i), x);
    if (tail) {
      const uint32_t vis = live ? visible32(a, seg, node, p0 + 32 * i) : 0u;
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 32; ++k) x[k] = (vis >> k) & 1u ? x[k] : 0xff800000u;
    }
  };
  float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
  for (int i = 0; i < chunks; ++i) {
    load(i);
#pragma unroll
    for (int k = 0; k < 32; k += 2)
      tops[(k / 2) % 4] = max3(tops[(k / 2) % 4], __uint_as_float(x[k]), __uint_as_float(x[k + 1]));
  }
  const float top = fmaxf(max3(tops[0], tops[1], tops[2]), tops[3]) * sl2;
  const bool grow = top > m;
  if (__any_sync(0xffffffffu, grow)) {
    const float f = grow ? ex2(m - (top + kLazyLog2)) : 1.f;
    if (grow) m = top + kLazyLog2;
    l *= f;
    if (!first) {
#pragma unroll 1
      for (int c = 0; c < kD; c += 32) {
        uint32_t o[32];
        tm_ld(tm_o + uint32_t(c), o);
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
        tm_st(tm_o + uint32_t(c), o);
      }
    }
  }
  const float off = m == -INFINITY ? 0.f : -m;
  const float2 s2 = make_float2(sl2, sl2), o2 = make_float2(off, off);
  float2 sum0 = make_float2(0.f, 0.f), sum1 = make_float2(0.f, 0.f);
  auto weights = [&](uint32_t at) {
    // 16 keys at a time, so that few registers are held
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t p[8], rest[8];
#pragma unroll
      for (int k = 0; k < 16; k += 2) {
        float2 e = __ffma2_rn(make_float2(__uint_as_float(x[16 * h + k]), __uint_as_float(x[16 * h + k + 1])),
                              s2, o2);
        e.x = ex2(e.x);
        e.y = ex2(e.y);
        if (k % 4 == 0)
          sum0 = __fadd2_rn(sum0, e);
        else
          sum1 = __fadd2_rn(sum1, e);
        p[k / 2] = pack_bf16x2(e.x, e.y);
        const float2 r = __ffma2_rn(make_float2(__uint_as_float(p[k / 2] << 16),
                                                __uint_as_float(p[k / 2] & 0xffff0000u)),
                                    make_float2(-1.f, -1.f), e);
        rest[k / 2] = pack_bf16x2(r.x, r.y);
      }
      tm_st8(at + 8 * h, p);
      tm_st8(at + 16 + 8 * h, rest);
    }
  };
#pragma unroll 1
  for (int i = chunks - 1; i >= 0; --i) {
    if (i != chunks - 1) load(i);  // (the last is still held)
    weights(tm_s + 32 * (chunk0 + i));
  }
  if (chunks < 4) {
    const uint32_t zero[16] = {};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if ((c & -chunks) != chunk0) {
        tm_st16(tm_s + 32 * c, zero);
        tm_st16(tm_s + 32 * c + 16, zero);
      }
    }
  }
  l += (sum0.x + sum0.y) + (sum1.x + sum1.y);
  tm_st_wait();
}

template <int kD, bool kFp8>
__global__ void __launch_bounds__(AttnShape<kD, kFp8>::kThreads, 1)
    attention_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                     const __grid_constant__ AttnArgs a, const __grid_constant__ AttnDims d,
                     int box_rows, int part_rows) {
  using Sh = AttnShape<kD, kFp8>;
  extern __shared__ __align__(1024) uint8_t attn_smem[];
  auto& ctl = *reinterpret_cast<typename Sh::Control*>(attn_smem + Sh::kTilesBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t smem0 = smem_addr(attn_smem);
  // The tiles' swizzle needs 1024-byte alignment, which a kernel without
  // static shared memory has; were it not so, nothing could be computed.
  if (smem0 % 1024 != 0) {
    if (threadIdx.x == 0 && a.dev_status) atomicOr(a.dev_status, FCT_DEV_WAIT_TIMEOUT);
    return;
  }
  const uint32_t slot0 = smem0 + 2 * Sh::kTileBytes;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (threadIdx.x == 0) {
    for (int i = 0; i < Sh::kSlots; ++i) {
      mbar_init(&ctl.full_bar[i], kFp8 ? Sh::kPrepWarps : 1);
      mbar_init(&ctl.empty_bar[i], 1);
    }
    for (int i = 0; i < Sh::kTail; ++i) {
      mbar_init(&ctl.tail_full[i], 1);
      mbar_init(&ctl.prep_bar[i], Sh::kPrepWarps);
    }
    for (int i = 0; i < Sh::kRaw; ++i) {
      mbar_init(&ctl.raw_full[i], 1);
      mbar_init(&ctl.raw_scaled[i], 1);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(&ctl.s_full[w], 1);
      mbar_init(&ctl.p_full[w], kSoftWarps / 2);
    }
    mbar_init(&ctl.q_full, kSoftWarps);
    mbar_init(&ctl.o_full, 1);
    mbar_init(&ctl.ml_full, kSoftWarps);
    mbar_init(&ctl.done_bar, 1);
    ctl.abort_flag = 0;
    for (int i = 0; i < kBadRing; ++i) ctl.bad_seg[i] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(&ctl.tmem_base)),
                 "r"(kAtTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }

  int32_t status = 0;
  if (warp == 2) {
    // the deal: this CTA's run, as the request and the offset in it where it starts
    const Batch batch = batch_of(a, d);
    if (batch.bad && blockIdx.x == 0 && lane == 0) status |= FCT_DEV_INDEX_OUT_OF_RANGE;
    const int64_t runs = batch.deal.runs(batch.total, gridDim.x);
    const int64_t run0 = Deal::run_start(batch.total, runs, blockIdx.x);
    const int64_t run1 = Deal::run_start(batch.total, runs, blockIdx.x + 1);
    if (lane == 0) {
      ctl.sched[2] = run1 - run0;
      ctl.sched[3] = batch.deal.whole;
    }
    if (run1 > run0)
      scan_requests(a, d, batch.deal, [&](int64_t before, int64_t cost, int64_t b, const RequestShape&) {
        const bool here = cost > 0 && before <= run0 && run0 < before + cost;
        if (here) {
          ctl.sched[0] = b;
          ctl.sched[1] = run0 - before;
        }
        return __any_sync(0xffffffffu, here) != 0;
      });
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = ctl.tmem_base;
  SegmentWalk walk(a, d, Deal{ctl.sched[3] != 0, start_cost_of(kFp8)}, ctl.sched[0], ctl.sched[1], ctl.sched[2]);
  Segment seg;
  auto lead_of = [](const Segment& s) { return s.rows > kTile ? 1 : 2; };
  // whether a key tile (index in the unit) reaches past the context
  auto is_tail = [](const Segment& s, int tile) { return (tile + 1) * kTile > s.ctx; };

  // ---- loads: a warp sends K tiles, V tiles or both, its lanes a tile's boxes
  auto load_tiles = [&](bool do_k, bool do_v) {
    constexpr int kBoxCols = kFp8 ? 1 : Sh::kHalves;
    uint64_t* full = kFp8 ? ctl.raw_full : ctl.full_bar;
    const int boxes = kTile / box_rows * kBoxCols;
    const uint32_t box_bytes = uint32_t(box_rows) * (kFp8 ? kD : 128);
    const int page_size = a.cache.page_size;
    uint32_t item = 0;
    // per slot: the barrier of its last fill (1: tail_full), and each
    // barrier's next parity, both warps' fills counted
    uint32_t last_tail = 0, full_phase = 0, tail_phase = 0;
    bool ok = true;
    const int piece = lane / kBoxCols, half = lane % kBoxCols;
    while (ok && walk.next(seg)) {
      // The lane's piece of tile `next`: its place in the block table, and its
      // page, asked for a tile ahead of its use.  A tile's page is kept for V,
      // which is sent at most two tiles after K.
      const int32_t* table = a.pages.table + seg.b * a.pages.ld;
      int pos = seg.tile0 * kTile + piece * box_rows;
      int in_table = pos / page_size, in_page = pos - in_table * page_size;
      int next = 0, asked_page = 0, asked_at = 0;
      int pages[4] = {0, 0, 0, 0}, slots[4] = {0, 0, 0, 0};
      auto ask = [&]() {
        asked_at = in_page;
        asked_page = 0;
        if (next < seg.tiles && lane < boxes && pos < seg.len) asked_page = table[in_table];
        ++next;
        pos += kTile;
        in_page += kTile % page_size;
        in_table += kTile / page_size;
        if (in_page >= page_size) {
          in_page -= page_size;
          ++in_table;
        }
      };
      ask();
      for_items(seg.tiles, lead_of(seg), [&](bool is_v, int j) {
        const uint32_t slot = item % Sh::kSlots, phase = (item / Sh::kSlots) & 1u;
        ++item;
        const bool prep = !kFp8 && is_v && is_tail(seg, seg.tile0 + j);
        last_tail = (last_tail & ~(1u << slot)) | (uint32_t(prep) << slot);
        (prep ? tail_phase : full_phase) ^= 1u << slot;
        if (!is_v) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if ((j & 3) == i) {
              pages[i] = asked_page;
              slots[i] = asked_at;
            }
          ask();
        }
        if (!(is_v ? do_v : do_k)) return true;
        if (!warp_wait(&ctl.empty_bar[slot], phase ^ 1u, &ctl.abort_flag)) {
          ok = false;
          return false;
        }
        uint64_t* bar = prep ? &ctl.tail_full[slot] : &full[slot];
        const int rows = min(seg.len - (seg.tile0 + j) * kTile, kTile);
        if (lane == 0)
          mbar_arrive_expect_tx(bar, uint32_t((rows + box_rows - 1) / box_rows) * kBoxCols * box_bytes);
        __syncwarp();
        if (lane < boxes && piece * box_rows < rows) {
          int page = 0, at = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if ((j & 3) == i) {
              page = pages[i];
              at = slots[i];
            }
          if (page < 0 || page >= a.cache.num_pages) status |= FCT_DEV_INDEX_OUT_OF_RANGE;
          const uint32_t dst = slot0 + slot * Sh::kSlotBytes + Sh::kRawAt +
                               (kFp8 ? uint32_t(piece) * box_bytes
                                     : uint32_t(half) * (kTile * 128) + uint32_t(piece) * box_bytes);
          tma_box(dst, is_v ? &map_v : &map_k, half * 64, at, seg.h, page, bar);
        }
        return true;
      });
    }
    // the last fills have landed before the CTA ends (bounded, even after an
    // abort)
    for (uint32_t slot = 0; slot < uint32_t(Sh::kSlots) && slot < item; ++slot) {
      const bool tail = (last_tail >> slot) & 1u;
      wait_phase(tail ? &ctl.tail_full[slot] : &full[slot],
                 (((tail ? tail_phase : full_phase) >> slot) & 1u) ^ 1u, &ctl.abort_flag, false);
    }
  };

  // Goes through converted places once more, rows row0, row0 + step, ... of the
  // key tile at p0 in slot dst, 16-byte pieces `piece` (+ 4): puts NaN where the
  // payload is e4m3's, and 0 for what is not finite of drafted values (`clear`).
  // Whether there were any of the latter.
  auto mend_tile = [&](bool is_v, int p0, int row0, int step, int piece, uint32_t dst, bool clear) {
    bool dropped = false;
#pragma unroll 1
    for (int row = row0; row < kTile && p0 + row < seg.len; row += step) {
      int at;
      const int64_t page = page_of(a, seg, p0 + row, &at);
      if (page < 0 || page >= a.cache.num_pages) continue;
      const uint8_t* src = static_cast<const uint8_t*>(is_v ? a.cache.v : a.cache.k) +
                           page * a.cache.page_stride + at * a.cache.slot_stride + seg.h * a.cache.head_stride;
      const bool drop = clear && p0 + row >= seg.ctx;
#pragma unroll 1
      for (int i = 0; i < Sh::kHalves * 16; ++i) {
        const int c = piece * 16 + i % 16;  // of a 64-column block
        const uint32_t place = dst + uint32_t(i / 16) * (kTile * 128) + uint32_t(row) * 128 +
                               uint32_t(((c / 8) ^ (row & 7)) * 16 + (c % 8) * 2);
        const bool nan = (src[(i / 16) * 64 + c] & 0x7f) == 0x7f;
        uint16_t x;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(place));
        if (!nan && !(drop && (x & 0x7f80) == 0x7f80)) continue;
        dropped |= drop;
        asm volatile("st.shared.u16 [%0], %1;" ::"r"(place), "h"(static_cast<uint16_t>(drop ? 0 : 0x7fc0))
                     : "memory");
      }
    }
    return dropped;
  };

  auto prepare = [&]() {
    // ---- tiles prepared
    constexpr int kPrepThreads = Sh::kPrepWarps * 32;
    const int t = (threadIdx.x - Sh::kPrepWarp0 * 32) % kPrepThreads;
    uint32_t item = 0, tail_phase = 0;
    int seg_n = 0;
    bool ok = true;
    while (ok && walk.next(seg)) {
      ++seg_n;
      for_items(seg.tiles, lead_of(seg), [&](bool is_v, int j) {
        const uint32_t it = item++;
        const uint32_t slot = it % Sh::kSlots;
        const int tile = seg.tile0 + j, p0 = tile * kTile;
        const uint32_t dst = slot0 + slot * Sh::kSlotBytes;
        if constexpr (kFp8) {
          const uint32_t phase = (it / Sh::kSlots) & 1u;
          if (!warp_wait(&ctl.raw_full[slot], phase, &ctl.abort_flag) ||
              !warp_wait(&ctl.raw_scaled[slot], phase, &ctl.abort_flag)) {
            ok = false;
            return false;
          }
          // A thread takes 16-byte pieces t % 4 (+ 4) of row t / 4 of each kRows rows:
          // eight lanes store to different banks, and every address but the
          // first is a constant away.  The next row is loaded before the present
          // one is turned; a row's four lanes have all loaded it before any of
          // them stores to it.
          constexpr int kHalves = Sh::kHalves, kRows = kPrepThreads / 4;
          const uint32_t src = dst + Sh::kRawAt + uint32_t(t / 4) * kD + uint32_t(t % 4) * 16;
          const uint32_t out0 = dst + uint32_t(t / 4) * 128 + uint32_t((((t % 4) * 2) ^ ((t / 4) & 7)) * 16);
          const uint32_t out1 = out0 ^ 16u;
          const uint32_t scale = smem_addr(&ctl.raw_scale[slot][t / 4]);
          const bool clear = is_v && is_tail(seg, tile);
          uint32_t odd = 0;  // bit 7 of some byte: this thread's places are looked through once more
          uint32_t in[kHalves][4], byte;
          auto load = [&](int block) {
            asm volatile("ld.shared.u8 %0, [%1];" : "=r"(byte) : "r"(scale + uint32_t(kRows) * block));
#pragma unroll
            for (int h = 0; h < kHalves; ++h)
              asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(in[h][0]), "=r"(in[h][1]), "=r"(in[h][2]), "=r"(in[h][3])
                           : "r"(src + uint32_t(kRows * kD) * block + 64u * h));
          };
          load(0);
#pragma unroll 1
          for (int block = 0; block < kTile / kRows; ++block) {
            uint32_t x[kHalves][4], e = byte;
#pragma unroll
            for (int h = 0; h < kHalves; ++h)
#pragma unroll
              for (int k = 0; k < 4; ++k) x[h][k] = in[h][k];
            if (block + 1 < kTile / kRows) load(block + 1);
            __syncwarp();
            if (clear) {
              const int pos = p0 + block * kRows + t / 4;
              if (pos >= seg.len) {
                e = 127;
#pragma unroll
                for (int h = 0; h < kHalves; ++h) x[h][0] = x[h][1] = x[h][2] = x[h][3] = 0;
              } else if (pos >= seg.ctx && e >= kLargeScale) {
                odd = ~0u;
              }
            }
            // bit 7 of a byte where adding 1 changes it: 7 bits of ones, e4m3's NaN
            // (a carry into the next byte comes from such a byte only)
#pragma unroll
            for (int h = 0; h < kHalves; ++h)
#pragma unroll
              for (int k = 0; k < 4; ++k) odd |= (x[h][k] + 0x01010101u) ^ x[h][k];
            // 2^120 * 2^(e - 127) as one bf16 factor, or as two
            const bool one = e <= 134;
            const uint32_t f1 = (one ? e + 120 : 247u) * 0x00800080u;
#pragma unroll
            for (int h = 0; h < kHalves; ++h) {
              uint32_t o[8];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                o[2 * k] = mul_bf16x2(e4m3_bits(__byte_perm(x[h][k], 0, 0x1404)), f1);
                o[2 * k + 1] = mul_bf16x2(e4m3_bits(__byte_perm(x[h][k], 0, 0x3424)), f1);
              }
              if (!one) {
                const uint32_t f2 = e == 255 ? 0x7fc07fc0u : e * 0x00800080u;
#pragma unroll
                for (int k = 0; k < 8; ++k) o[k] = mul_bf16x2(o[k], f2);
              }
              const uint32_t at = uint32_t(kRows * 128) * block + uint32_t(h) * (kTile * 128);
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(out0 + at), "r"(o[0]),
                           "r"(o[1]), "r"(o[2]), "r"(o[3])
                           : "memory");
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(out1 + at), "r"(o[4]),
                           "r"(o[5]), "r"(o[6]), "r"(o[7])
                           : "memory");
            }
          }
          // (e4m3's NaN came out as 480 times the scale, a large scale's values may
          // be infinite; both are rare)
          if ((odd & 0x80808080u) && mend_tile(is_v, p0, t / 4, kRows, t % 4, dst, clear))
            ctl.bad_seg[seg_n % kBadRing] = seg_n;
          async_fence();
          warp_arrive(&ctl.full_bar[slot]);
        } else {
          if (!is_v || !is_tail(seg, tile)) return true;
          if (!warp_wait(&ctl.tail_full[slot], (tail_phase >> slot) & 1u, &ctl.abort_flag)) {
            ok = false;
            return false;
          }
          tail_phase ^= 1u << slot;
          // 16-byte pieces of the rows past the context, several under way at once
          constexpr int kPieces = kD / 8, kBatch = 8;
          const int from = max(seg.ctx - p0, 0);
          const int held = min(seg.len - p0, kTile);  // rows from here on are cleared
          uint8_t* tile_at = attn_smem + 2 * Sh::kTileBytes + slot * Sh::kSlotBytes;
          auto place = [&](int n) {
            const int row = n / kPieces, c = n % kPieces;
            return reinterpret_cast<uint4*>(tile_at + (c / 8) * (kTile * 128) + row * 128 + ((c % 8) ^ (row & 7)) * 16);
          };
          bool found = false;
          for (int n0 = from * kPieces + t; n0 < held * kPieces; n0 += kPrepThreads * kBatch) {
            uint4 v[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
              if (n0 + i * kPrepThreads < held * kPieces) v[i] = *place(n0 + i * kPrepThreads);
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
              if (n0 + i * kPrepThreads >= held * kPieces) continue;
              uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
              bool change = false;
#pragma unroll
              for (int k = 0; k < 4; ++k) change |= drop_non_finite(w[k]);
              if (change) {
                found = true;
                *place(n0 + i * kPrepThreads) = make_uint4(w[0], w[1], w[2], w[3]);
              }
            }
          }
#pragma unroll 4
          for (int n = max(from, held) * kPieces + t; n < kTile * kPieces; n += kPrepThreads)
            *place(n) = make_uint4(0, 0, 0, 0);
          if (found) ctl.bad_seg[seg_n % kBadRing] = seg_n;
          async_fence();
          warp_arrive(&ctl.prep_bar[slot]);
        }
        return true;
      });
    }
  };

  if (warp < 4) {
    if (warp == 0) {
      load_tiles(true, kFp8);
    } else if (warp == 1) {
    // ---- products: the warp goes through the tiles converged, one lane
    // issues (what the issue needs is then the same in all lanes, which keeps
    // it in uniform registers)
    constexpr uint32_t kIdS = attn_idesc(kTile, false), kIdO = attn_idesc(kD, true);
    uint32_t item = 0, seg_n = 0, full_phase = 0, prep_phase = 0;
    uint32_t p_phase = 0;
    bool ok = true;
    const bool issue = elect_one();
    auto slot_addr = [&](uint32_t it) { return uniform(slot0 + (it % Sh::kSlots) * Sh::kSlotBytes); };
    auto wait_item = [&](uint32_t it) {
      const uint32_t slot = it % Sh::kSlots;
      const bool got = warp_wait(&ctl.full_bar[slot], (full_phase >> slot) & 1u, &ctl.abort_flag);
      full_phase ^= 1u << slot;
      return got;
    };
    auto scores = [&](int w, int q_tile, uint32_t it, bool last) {
      const uint32_t tm_s = uniform(tmem + uint32_t(w) * kTile);
      const uint32_t qd = uniform(desc_lo(smem0 + uint32_t(q_tile) * Sh::kTileBytes, false));
      const uint32_t kd = desc_lo(slot_addr(it), false);
      tc_after();
      if (issue) {
#pragma unroll
        for (int k = 0; k < kD / 16; ++k) {
          const uint32_t step = uint32_t((k / 4) * (kTile * 128) + (k % 4) * 32) >> 4;
          umma_ss<kIdS>(tm_s, qd + step, kd + step, k > 0);
        }
        umma_commit(&ctl.s_full[w]);
        if (last) umma_commit(&ctl.empty_bar[it % Sh::kSlots]);
      }
      __syncwarp();
    };
    auto values = [&](int w, uint32_t it, bool first, bool last) {
      const uint32_t tm_s = uniform(tmem + uint32_t(w) * kTile);
      const uint32_t tm_o = uniform(tmem + 2 * kTile + uint32_t(w) * kD);
      const uint32_t vd = desc_lo(slot_addr(it), true);
      tc_after();
      if (issue) {
        // a chunk of 32 keys: two steps of weights, two of remainders
#pragma unroll
        for (int k = 0; k < 2 * kTile / 16; ++k)
          umma_ts<kIdO>(tm_o, tm_s + k * 8, vd + (((k / 4) * 2 + k % 2) * 16 * 128 >> 4), !first || k > 0);
        if (last) umma_commit(&ctl.empty_bar[it % Sh::kSlots]);
      }
      __syncwarp();
    };
    auto wait_p = [&](int w) {
      const bool got = warp_wait(&ctl.p_full[w], (p_phase >> w) & 1u, &ctl.abort_flag);
      p_phase ^= 1u << w;
      return got;
    };
    auto wait_v = [&](uint32_t it, int tile) {
      if (kFp8 || !is_tail(seg, tile)) return wait_item(it);
      const uint32_t slot = it % Sh::kSlots;
      const bool got = warp_wait(&ctl.prep_bar[slot], (prep_phase >> slot) & 1u, &ctl.abort_flag);
      prep_phase ^= 1u << slot;
      return got;
    };
    while (ok && walk.next(seg)) {
      const bool two = seg.rows > kTile;
      if (!warp_wait(&ctl.q_full, seg_n & 1u, &ctl.abort_flag)) break;
      ++seg_n;
      uint32_t k_item = 0;
#pragma unroll 1
      for (int w = 0; ok && w < (two ? 2 : min(2, seg.tiles)); ++w) {
        if (!two || w == 0) {
          k_item = item++;
          ok = wait_item(k_item);
        }
        if (ok) scores(w, two ? w : 0, k_item, !two || w == 1);
      }
      const int lead = lead_of(seg), last = two ? 1 : 0;
#pragma unroll 1
      for (int j = 0; ok && j < seg.tiles; ++j) {
        const uint32_t v_item = item++;
        const bool more = j + lead < seg.tiles;
        if (more) k_item = item++;
        ok = wait_v(v_item, seg.tile0 + j);
#pragma unroll 1
        for (int u = 0; ok && u <= last; ++u) {
          const int w = two ? u : j & 1;
          ok = wait_p(w);
          if (!ok) break;
          values(w, v_item, j < lead, u == last);
          if (more) {
            if (u == 0) ok = wait_item(k_item);
            if (ok) scores(w, two ? u : 0, k_item, u == last);
          }
        }
      }
      if (ok && issue) umma_commit(&ctl.o_full);
      __syncwarp();
    }
    if (issue) umma_commit(&ctl.done_bar);  // every product issued has completed
    __syncwarp();
    } else if constexpr (kFp8) {
    // ---- scale bytes of the raw tiles, four keys per lane; warps 2 and 3 take
    // the items in turn and fetch the next one's bytes before they hand on
    // this one's
    uint32_t item = 0, held_item = 0;
    uint32_t held = 0;  // four bytes
    bool ok = true, holds = false;
    auto hand_on = [&]() {
      const uint32_t slot = held_item % Sh::kSlots, phase = (held_item / Sh::kSlots) & 1u;
      ok = warp_wait(&ctl.empty_bar[slot], phase ^ 1u, &ctl.abort_flag);
      if (!ok) return;
      *reinterpret_cast<uint32_t*>(&ctl.raw_scale[slot][4 * lane]) = held;
      warp_arrive(&ctl.raw_scaled[slot]);
    };
    while (ok && walk.next(seg)) {
      for_items(seg.tiles, lead_of(seg), [&](bool is_v, int j) {
        const uint32_t it = item++;
        if ((it & 1u) != uint32_t(warp & 1)) return true;
        const int p0 = (seg.tile0 + j) * kTile + 4 * lane;
        const uint8_t* scales = is_v ? a.cache.v_scale : a.cache.k_scale;
        uint32_t bytes = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (p0 + i < seg.len) {
            int at;
            const int64_t page = page_of(a, seg, p0 + i, &at);
            if (page >= 0 && page < a.cache.num_pages)
              bytes |= uint32_t(scales[page * a.cache.scale_page_stride + at * a.cache.scale_slot_stride +
                                       seg.h * a.cache.scale_head_stride])
                       << (8 * i);
          }
        }
        if (holds) hand_on();
        held = bytes;
        held_item = it;
        holds = true;
        return ok;
      });
    }
    if (ok && holds) hand_on();
    } else if (warp == 2) {
      prepare();
    } else {
      load_tiles(false, true);
    }
  } else if (warp < 12) {
    // ---- softmax groups A (warps 4-7) and B (8-11).  A lane of tensor memory
    // is a row; with at most 64 (32) rows the query tile holds them twice (four
    // times), and the warps of each copy take a half (quarter) of a tile's
    // keys, with maxima, sums and outputs of their own.
    const int w = warp >= 8 ? 1 : 0;
    const int r = threadIdx.x & (kTile - 1);       // lane of tensor memory
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    const uint32_t tm_s = tmem + uint32_t(w) * kTile + lanes;
    const uint32_t tm_o = tmem + 2 * kTile + lanes;
    // The factor of the scores is positive, so that -inf (masked) stays -inf: a
    // negative scale negates the query rows, a scale of 0 makes them 0.
    const bool no_scale = a.scale == 0.f;
    const float sl2 = no_scale ? kLog2e : fabsf(a.scale) * kLog2e;
    const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;
    // bf16 pairs times 0: NaN where they are not finite
    auto times_zero = [](uint32_t x) {
      return ((x & 0x7f80u) == 0x7f80u ? 0x7fc0u : 0u) | ((x & 0x7f800000u) == 0x7f800000u ? 0x7fc00000u : 0u);
    };
    const bool vec_q = reinterpret_cast<uintptr_t>(a.q) % 16 == 0 && a.ld_qn % 8 == 0 && a.ld_qh % 8 == 0;
    const bool vec_o = reinterpret_cast<uintptr_t>(a.out) % 16 == 0 && a.ld_on % 8 == 0 && a.ld_oh % 8 == 0;
    uint32_t s_n = 0, ml_n = 0;
    int seg_n = 0;
    bool ok = true;
    // all softmax warps meet (false: a wait ran out)
    auto meet = [&]() {
      warp_arrive(&ctl.ml_full);
      return warp_wait(&ctl.ml_full, ml_n++ & 1u, &ctl.abort_flag);
    };
    while (ok && walk.next(seg)) {
      ++seg_n;
      const bool two = seg.rows > kTile;
      // rows per copy: 32, 64, or all 128 lanes
      const int span = two || seg.rows > 64 ? kTile : seg.rows > 32 ? 64 : 32;
      const int row = (two ? w * kTile : 0) + (r & (span - 1));   // of the unit
      const bool live = row < seg.rows;
      const bool warp_live = (row & ~31) < seg.rows;
      const int node = live ? (seg.row0 + row) / d.group : 0;
      const int head = seg.h * d.group + (live ? (seg.row0 + row) % d.group : 0);
      // the query tile, in the products' swizzle; with one tile its columns
      // are split over the groups
      if (live) {
        const uint16_t* src = static_cast<const uint16_t*>(a.q) + int64_t(seg.node0 + node) * a.ld_qn +
                              int64_t(head) * a.ld_qh;
        const uint32_t dst = smem0 + (two ? uint32_t(w) * Sh::kTileBytes : 0u) + uint32_t(r) * 128;
        // half of a row at a time, all its loads under way at once
        constexpr int kHalf = kD / 16;
#pragma unroll 1
        for (int c0 = two ? 0 : w * kHalf; c0 < (two ? kD / 8 : (w + 1) * kHalf); c0 += kHalf) {
          uint4 x[kHalf];
          if (vec_q) {
#pragma unroll
            for (int c = 0; c < kHalf; ++c) x[c] = *reinterpret_cast<const uint4*>(src + (c0 + c) * 8);
          } else {
#pragma unroll
            for (int c = 0; c < kHalf; ++c) {
              uint32_t y[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                y[k] = uint32_t(src[(c0 + c) * 8 + 2 * k]) | (uint32_t(src[(c0 + c) * 8 + 2 * k + 1]) << 16);
              x[c] = make_uint4(y[0], y[1], y[2], y[3]);
            }
          }
          if (no_scale) {
#pragma unroll
            for (int c = 0; c < kHalf; ++c)
              x[c] = make_uint4(times_zero(x[c].x), times_zero(x[c].y), times_zero(x[c].z), times_zero(x[c].w));
          }
#pragma unroll
          for (int c = 0; c < kHalf; ++c)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                             dst + uint32_t((c0 + c) / 8) * (kTile * 128) +
                             uint32_t((((c0 + c) % 8) ^ (r & 7)) * 16)),
                         "r"(x[c].x ^ flip), "r"(x[c].y ^ flip), "r"(x[c].z ^ flip), "r"(x[c].w ^ flip)
                         : "memory");
        }
      }
      async_fence();
      tc_before();
      warp_arrive(&ctl.q_full);

      float m = -INFINITY, l = 0.f;   // the weights' exponent offset and their sum
      bool first = true;
      const int chunk0 = span == kTile ? 0 : span == 64 ? (warp & 2) : (warp & 3);
      for (int j = two ? 0 : w; j < seg.tiles; j += two ? 1 : 2) {
        if (!warp_wait(&ctl.s_full[w], s_n & 1u, &ctl.abort_flag)) {
          ok = false;
          break;
        }
        ++s_n;
        tc_after();
        if (warp_live) {
          const int p0 = (seg.tile0 + j) * kTile + 32 * chunk0;
          const bool tail = is_tail(seg, seg.tile0 + j);
          soft_tile<kD>(a, seg, tm_s, tm_o + uint32_t(w) * kD, chunk0, span / 32, node, live, p0, tail,
                        first, sl2, m, l);
        }
        first = false;
        tc_before();
        warp_arrive(&ctl.p_full[w]);
      }
      if (!ok || !warp_wait(&ctl.o_full, (seg_n - 1) & 1u, &ctl.abort_flag)) break;
      tc_after();
      const bool fix = *reinterpret_cast<volatile int*>(&ctl.bad_seg[seg_n % kBadRing]) == seg_n;
      float* const slot = seg.whole ? nullptr
                                    : static_cast<float*>(a.workspace) +
                                          (int64_t(blockIdx.x) * 2 + seg.part) * part_rows * (kD + 2);
      // a row's maximum and sum, and n of its columns from c on, to where they go
      auto put_stats = [&](int row_, float M, float L) {
        const int i = seg.row0 + row_;
        if (slot)
          reinterpret_cast<float2*>(slot + int64_t(part_rows) * kD)[row_] = make_float2(M, L);
        else if (a.lse)
          a.lse[int64_t(seg.node0 + i / d.group) * a.n_q_heads + seg.h * d.group + i % d.group] =
              L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
      };
      auto put = [&](int row_, int c, auto& o, float L) {
        constexpr int kN = int(sizeof(o) / sizeof(float));
        const int i = seg.row0 + row_, node_ = i / d.group, head_ = seg.h * d.group + i % d.group;
        if (fix) {
          // non-finite values of drafted nodes that this row sees
          const int end = min((seg.tile0 + seg.tiles) * kTile, seg.len);
          for (int pos = max(seg.ctx, seg.tile0 * kTile); pos < end; ++pos) {
            if (!(visible32(a, seg, node_, pos) & 1u)) continue;
            int at;
            const int64_t page = page_of(a, seg, pos, &at);
            if (page < 0 || page >= a.cache.num_pages) continue;
            const int64_t v_at = page * a.cache.page_stride + at * a.cache.slot_stride +
                                 seg.h * a.cache.head_stride + c;
            auto add = [&](int k, float y) {
              if (!(fabsf(y) < INFINITY)) o[k] += y;
            };
            if constexpr (kFp8) {
              const float scale =
                  scale_of(a.cache.v_scale[page * a.cache.scale_page_stride + at * a.cache.scale_slot_stride +
                                           seg.h * a.cache.scale_head_stride]);
              const uint8_t* v = static_cast<const uint8_t*>(a.cache.v) + v_at;
#pragma unroll
              for (int k = 0; k < kN; k += 4) {
                const float4 y = e4m3_floats(*reinterpret_cast<const uint32_t*>(v + k));
                add(k, y.x * scale);
                add(k + 1, y.y * scale);
                add(k + 2, y.z * scale);
                add(k + 3, y.w * scale);
              }
            } else {
              const bf16_t* v = static_cast<const bf16_t*>(a.cache.v) + v_at;
#pragma unroll
              for (int k = 0; k < kN; ++k) add(k, Elem<bf16_t>::load1(v + k));
            }
          }
        }
        if (slot) {
#pragma unroll
          for (int k = 0; k < kN; k += 4)
            *reinterpret_cast<float4*>(slot + int64_t(row_) * kD + c + k) =
                make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
          return;
        }
        const float inv = 1.f / L;
#pragma unroll
        for (int k = 0; k < kN; ++k) o[k] = L == 0.f ? 0.f : o[k] * inv;
        uint16_t* dst = static_cast<uint16_t*>(a.out) + int64_t(seg.node0 + node_) * a.ld_on +
                        int64_t(head_) * a.ld_oh + c;
        if (vec_o) {
          if constexpr (kN % 8 == 0) {
#pragma unroll
            for (int k = 0; k < kN; k += 8)
              *reinterpret_cast<uint4*>(dst + k) =
                  make_uint4(pack_bf16x2(o[k], o[k + 1]), pack_bf16x2(o[k + 2], o[k + 3]),
                             pack_bf16x2(o[k + 4], o[k + 5]), pack_bf16x2(o[k + 6], o[k + 7]));
          } else {
            *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
          }
        } else {
#pragma unroll
          for (int k = 0; k < kN; ++k) dst[k] = static_cast<uint16_t>(pack_bf16x2(o[k], 0.f));
        }
      };
      if (two) {
        if (live) put_stats(row, m, l);
        if (warp_live) {
#pragma unroll 1
          for (int c = 0; c < kD; c += 32) {
            uint32_t x[32];
            float o[32];
            __syncwarp();
            tm_ld(tm_o + uint32_t(w * kD + c), x);
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __uint_as_float(x[k]);
            if (live) put(row, c, o, l);
          }
        }
        continue;
      }
      // One query tile: a row's sums are spread over both groups and its copies.
      // (The next segment's write of ml follows every thread's read of this
      // one's: it waits for products that wait for all threads' query rows.)
      ctl.ml[w][r] = make_float2(m, l);
      if (!meet()) break;
      const bool both = seg.tiles > 1;
      auto row_sums = [&](int first_lane, float& M, float& L) {
        M = -INFINITY;
        for (int c = first_lane; c < kTile; c += span)
          M = max3(M, ctl.ml[0][c].x, both ? ctl.ml[1][c].x : -INFINITY);
        const float base = M == -INFINITY ? 0.f : M;
        L = 0.f;
        for (int c = first_lane; c < kTile; c += span) {
          L += ctl.ml[0][c].y * ex2(ctl.ml[0][c].x - base);
          if (both) L += ctl.ml[1][c].y * ex2(ctl.ml[1][c].x - base);
        }
      };
      float M, L;
      row_sums(r & (span - 1), M, L);
      const float base = M == -INFINITY ? 0.f : M;
      const float wa = ex2(ctl.ml[0][r].x - base), wb = both ? ex2(ctl.ml[1][r].x - base) : 0.f;
      if (live && w == 0 && r == row) put_stats(row, M, L);
      // each group merges half of the columns of both; copies meet in the query
      // tiles' place (all products of this segment are done), 16-byte pieces
      // of a row at their place exclusive-or the row
      const uint32_t xch = smem0 + uint32_t(r) * (kD * 4);
      if (warp_live) {
#pragma unroll 1
        for (int c = w * (kD / 2); c < (w + 1) * (kD / 2); c += 32) {
          uint32_t x[32];
          float o[32];
          __syncwarp();
          tm_ld(tm_o + uint32_t(c), x);
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = __uint_as_float(x[k]) * wa;
          if (both) {
            tm_ld(tm_o + uint32_t(kD + c), x);
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = fmaf(__uint_as_float(x[k]), wb, o[k]);
          }
          if (span == kTile) {
            if (live) put(row, c, o, L);
          } else {
#pragma unroll
            for (int k = 0; k < 32; k += 4)
              asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(
                               xch + uint32_t((((c + k) / 4) ^ (r & (kD / 4 - 1))) * 16)),
                           "f"(o[k]), "f"(o[k + 1]), "f"(o[k + 2]), "f"(o[k + 3])
                           : "memory");
          }
        }
      }
      if (span < kTile) {
        if (!meet()) break;
        constexpr int kPieces = kD / 4;  // of a row; a warp takes 32 at a time
        for (int i = (warp - 4) * 32 + lane; i < seg.rows * kPieces; i += kSoftWarps * 32) {
          const int row_ = i / kPieces, piece = i % kPieces;
          float o[4] = {0.f, 0.f, 0.f, 0.f};
          for (int c = row_; c < kTile; c += span) {
            float x[4];
            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3])
                         : "r"(smem0 + uint32_t(c) * (kD * 4) +
                               uint32_t((piece ^ (c & (kPieces - 1))) * 16)));
#pragma unroll
            for (int k = 0; k < 4; ++k) o[k] += x[k];
          }
          if (!slot) row_sums(row_, M, L);
          put(row_, piece * 4, o, L);
        }
        if (!meet()) break;  // before the next query rows take the place
      }
    }
  } else {
    if constexpr (kFp8) prepare();
  }
  tc_before();
  __syncthreads();
  if (warp == 1) {
    if (lane == 0) wait_phase(&ctl.done_bar, 0, &ctl.abort_flag, false);
    __syncwarp();
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kAtTmemCols)
                 : "memory");
  }
  if (threadIdx.x == 0 && ctl.abort_flag) status |= FCT_DEV_WAIT_TIMEOUT;
  if (status && a.dev_status) atomicOr(a.dev_status, status);
}

// Adds the partial sums of units that were cut between CTAs, the pieces in the
// order of the keys, one row to a warp.  A unit is cut where runs meet, so
// blockIdx.x stands for the start of run blockIdx.x + 1: the meeting points
// inside one unit share its rows, and the kCombineBlocks blocks of each share
// that share.  Few bytes: what bounds it is the latency of a block's start, of
// working out its unit and of the loads of a piece.  8, 16 and 32 blocks of 8
// warps per meeting point, each warp working its unit out, took 1 x 8 nodes
// over 131071 keys 101, 108 and 126 us in all; 2 blocks of 16 warps and one
// warp to work it out 97 (12 x 64 nodes of 64 query heads: 164 -> 156).
constexpr int kCombineWarps = 16, kCombineBlocks = 2;

template <int kD>
__global__ void __launch_bounds__(kCombineWarps * 32)
    combine_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ AttnDims d, int ctas,
                   int part_rows) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // Which unit is cut here depends on the arguments only.  One warp works it out
  // for the block: it is 64-bit divisions mostly, and those of 16 warps took
  // longer than the rows.  Every thread waits for the attention kernel before
  // it reads a piece or leaves.
  __shared__ struct {
    int64_t total, runs, c0, c1, s, cost, h, node0, first[32];
    int rows, u, tiles;
  } cut;
  constexpr int kPer = kD / 32;
  const int64_t c = int64_t(blockIdx.x) + 1;
  const float* ws = static_cast<const float*>(a.workspace);
  const int64_t slot = int64_t(part_rows) * (kD + 2);
  // Where a run's piece of the unit lies: -1 if it has none, -2 if it has all of
  // the tiles.  The same for every row.
  // (units are only cut where they are not dealt whole)
  const Deal cut_deal{false, start_cost_of(a.cache.dtype == FCT_E4M3)};
  auto piece_at = [&](int64_t ci) -> int64_t {
    if (ci > cut.c1) return -1;
    const int64_t x1 = Deal::run_start(cut.total, cut.runs, ci + 1) - cut.s;
    const int t0 = cut_deal.tile_at(Deal::run_start(cut.total, cut.runs, ci) - cut.s, cut.tiles, cut.rows);
    const int t1 = x1 >= cut.cost ? cut.tiles : cut_deal.tile_at(x1, cut.tiles, cut.rows);
    if (t0 == 0 && t1 == cut.tiles) return -2;
    return t0 < t1 ? (ci * 2 + (t0 > 0 ? 0 : 1)) * slot : -1;
  };
  if (warp == 0) {
    const Batch batch = batch_of(a, d);
    const Deal& deal = batch.deal;
    const int64_t runs = deal.runs(batch.total, ctas);
    const int64_t at = Deal::run_start(batch.total, runs, c);
    int64_t before = 0, b = -1;
    if (!deal.whole && c < runs)
      scan_requests(a, d, deal, [&](int64_t before_, int64_t cost, int64_t b_, const RequestShape&) {
        const unsigned here = __ballot_sync(0xffffffffu, cost > 0 && before_ <= at && at < before_ + cost);
        if (!here) return false;
        const int src = __ffs(here) - 1;
        before = __shfl_sync(0xffffffffu, before_, src);
        b = __shfl_sync(0xffffffffu, b_, src);
        return true;
      });
    int rows = 0;  // 0: the runs meet between units, or there is no run
    if (b >= 0) {
      const RequestShape r = request_shape(a, d, b);
      const int64_t head_cost = deal.head(r), full = deal.unit(r.tiles, kUnitRows);
      const int64_t h = (at - before) / head_cost, in_head = (at - before) - h * head_cost;
      const int u = static_cast<int>(min(in_head / full, int64_t(r.row_units - 1)));
      const int64_t s = before + h * head_cost + u * full;
      if (at != s) {
        rows = u == r.row_units - 1 ? r.last_rows : kUnitRows;
        const int64_t cost = deal.unit(r.tiles, rows);
        if (lane == 0) {
          cut.total = batch.total;
          cut.runs = runs;
          cut.c0 = Deal::run_of(batch.total, runs, s);
          cut.c1 = Deal::run_of(batch.total, runs, s + cost - 1);
          cut.s = s;
          cut.cost = cost;
          cut.h = h;
          cut.node0 = r.node0;
          cut.u = u;
          cut.tiles = r.tiles;
        }
      }
    }
    if (lane == 0) cut.rows = rows;
    __syncwarp();
    if (rows > 0) cut.first[lane] = piece_at(cut.c0 + lane);
  }
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int rows = cut.rows, u = cut.u;
  if (rows == 0) return;
  const int64_t c0 = cut.c0, c1 = cut.c1, h = cut.h;
  // a piece's maximum and sum of row `at`
  auto stats = [&](int64_t p, int64_t at) {
    return p >= 0 && at < rows ? reinterpret_cast<const float2*>(ws + p + int64_t(part_rows) * kD)[at]
                               : make_float2(-INFINITY, 0.f);
  };
  const int64_t first = cut.first[lane];
  // the meeting points inside the unit are the starts of runs c0 + 1 .. c1
  const int64_t step = (c1 - c0) * kCombineBlocks * kCombineWarps;
  const int64_t at0 = ((c - c0 - 1) * kCombineBlocks + blockIdx.y) * kCombineWarps + warp;
  float2 ahead = stats(first, at0);
  for (int64_t at = at0; at < rows; at += step) {
    float M = -INFINITY, L = 0.f, o[kPer] = {};
    const float2 present = ahead;
    ahead = stats(first, at + step);
    for (int64_t base = c0; base <= c1; base += 32) {
      const int64_t p = base == c0 ? first : piece_at(base + lane);
      const float2 x = base == c0 ? present : stats(p, at);
      if (__any_sync(0xffffffffu, p == -2)) return;
      float top = x.x;
#pragma unroll
      for (int k = 16; k >= 1; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
      const float mn = fmaxf(M, top), off = mn == -INFINITY ? 0.f : mn;
      const float f = ex2(M - off), g = ex2(x.x - off);
      L = L * f + warp_sum(x.y * g);
      M = mn;
#pragma unroll
      for (int k = 0; k < kPer; ++k) o[k] *= f;
      const int n = c1 - base < 31 ? static_cast<int>(c1 - base) + 1 : 32;
#pragma unroll 8
      for (int i = 0; i < n; ++i) {
        const int64_t pi = __shfl_sync(0xffffffffu, p, i);
        const float gi = __shfl_sync(0xffffffffu, g, i);
        // (a NaN or infinity in a piece that counts for nothing stays out)
        if (pi >= 0 && gi != 0.f) {
          const float* src = ws + pi + at * kD + lane * kPer;
#pragma unroll
          for (int k = 0; k < kPer; ++k) o[k] = fmaf(gi, src[k], o[k]);
        }
      }
    }
    const int i = u * kUnitRows + static_cast<int>(at);
    const int64_t node = cut.node0 + i / d.group, head = h * d.group + i % d.group;
    bf16_t* dst = static_cast<bf16_t*>(a.out) + node * a.ld_on + head * a.ld_oh + lane * kPer;
#pragma unroll
    for (int k = 0; k < kPer; ++k) Elem<bf16_t>::store1(dst + k, L == 0.f ? 0.f : o[k] / L);
    if (a.lse && lane == 0)
      a.lse[node * a.n_q_heads + head] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
  }
}

PFN_cuTensorMapEncodeTiled_v12000 attn_encode_fn() {
  static std::once_flag once;
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    else
      cudaGetLastError();
  });
  return fn;
}

// Tensor map of a pool: (head_dim, slot, head, page), boxes of box_rows slots
// of one head and page; bf16 in 64-column blocks with 128-byte swizzle, e4m3
// whole rows as they are.
bool cache_map(CUtensorMap* map, const fct_kv_cache& c, void* base, int box_rows) {
  auto encode = attn_encode_fn();
  if (encode == nullptr) return false;
  const bool fp8 = c.dtype == FCT_E4M3;
  const cuuint64_t e = fp8 ? 1 : 2;
  const cuuint64_t dims[4] = {cuuint64_t(c.head_dim), cuuint64_t(c.page_size), cuuint64_t(c.n_heads),
                              cuuint64_t(c.num_pages)};
  const cuuint64_t strides[3] = {cuuint64_t(c.slot_stride) * e, cuuint64_t(c.head_stride) * e,
                                 cuuint64_t(c.page_stride) * e};
  const cuuint32_t box[4] = {cuuint32_t(fp8 ? c.head_dim : 64), cuuint32_t(box_rows), 1, 1};
  const cuuint32_t elem[4] = {1, 1, 1, 1};
  return encode(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base,
                dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                fp8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
                c.head_dim * int(e) >= 256 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                                           : CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Whether the tensor-core kernel takes this cache: a head_dim it is built
// for, pages of whole 8-token rows (a TMA box fills whole swizzle atoms), and
// what a tensor map needs (16-byte base and strides, 40-bit strides, 32-bit
// sizes).
bool tensor_core_layout(const fct_kv_cache& c) {
  if (c.head_dim != 64 && c.head_dim != 128) return false;
  if (c.page_size % 8 != 0 || c.num_pages > INT32_MAX) return false;
  const int64_t e = c.dtype == FCT_E4M3 ? 1 : 2;
  for (const void* p : {c.k, c.v})
    if (reinterpret_cast<uintptr_t>(p) % 16 != 0) return false;
  for (int64_t s : {c.slot_stride, c.head_stride, c.page_stride})
    if ((s * e) % 16 != 0 || s * e >= (int64_t(1) << 40) || s <= 0) return false;
  return true;
}

// Rows of a workspace slot: the most a unit has, in fours (16-byte rows).
int part_rows_of(int64_t n_nodes, int group) {
  const int64_t rows = (n_nodes * group + 3) / 4 * 4;
  return static_cast<int>(rows < kUnitRows ? rows : kUnitRows);
}

template <int kD, bool kFp8>
cudaError_t launch_tensor(const AttnArgs& a, int sms, int device, cudaStream_t st) {
  using Sh = AttnShape<kD, kFp8>;
  static std::once_flag once[64];
  static cudaError_t ready[64];
  if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
  auto kernel = attention_kernel<kD, kFp8>;
  std::call_once(once[device], [&] {
    ready[device] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(Sh::kSmem));
  });
  if (ready[device] != cudaSuccess) return ready[device];
  int box_rows = kTile;
  while (a.cache.page_size % box_rows != 0) box_rows /= 2;
  CUtensorMap mk, mv;
  if (!cache_map(&mk, a.cache, a.cache.k, box_rows) || !cache_map(&mv, a.cache, a.cache.v, box_rows))
    return cudaErrorInvalidValue;
  const AttnDims d{a.n_q_heads / a.cache.n_heads, static_cast<int>(a.pages.max_pages * a.cache.page_size)};
  const int part_rows = part_rows_of(a.n_nodes, d.group);
  kernel<<<static_cast<unsigned>(sms), Sh::kThreads, Sh::kSmem, st>>>(mk, mv, a, d, box_rows, part_rows);
  cudaError_t e = cudaGetLastError();
  // units of so few tiles are never cut
  if (e != cudaSuccess || d.room <= kWholeTiles * kTile) return e;
  if (sms < 2) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(sms - 1), kCombineBlocks);
  cfg.blockDim = dim3(kCombineWarps * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, combine_kernel<kD>, a, d, sms, part_rows);
}

}  // namespace

size_t attn_workspace_bytes(int64_t n_nodes, int n_q_heads, int n_heads, int head_dim, int sms) {
  if (head_dim != 64 && head_dim != 128) return 0;
  return size_t(sms) * 2 * size_t(part_rows_of(n_nodes, n_q_heads / n_heads)) * (head_dim + 2) * 4;
}

cudaError_t launch_attention(const AttnArgs& a, int sms, int device, cudaStream_t st) {
  if (!tensor_core_layout(a.cache)) return launch_general(a, st);
  const bool fp8 = a.cache.dtype == FCT_E4M3;
  if (a.cache.head_dim == 128)
    return fp8 ? launch_tensor<128, true>(a, sms, device, st) : launch_tensor<128, false>(a, sms, device, st);
  return fp8 ? launch_tensor<64, true>(a, sms, device, st) : launch_tensor<64, false>(a, sms, device, st);
}

}  // namespace fct
