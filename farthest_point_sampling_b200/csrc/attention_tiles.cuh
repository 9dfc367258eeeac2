// What the attention kernels share: the tile list, the key tiles a query tile
// sees and the visibility of one row.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "attention.h"
#include "common.cuh"
#include "tcgen05.cuh"

namespace fpstok {

constexpr int kTile = 128;  // rows of a query or key tile: one TMEM lane each

// One tile of an event: its rows are t * kTile .. of the event's queries (or
// keys, in the key list).
struct TileItem {
  int q0, nq, k0, nk;  // the event's first query row, queries, first key row, keys
  int t;
  int pad[3];
};

// A block's walk over (tile, head) items, heads first, `step` items at a time
// without a division.
struct ItemWalk {
  int tile, h, step_tiles, step_heads, heads, n_tiles;
  __device__ __forceinline__ ItemWalk(int heads_, int n_tiles_) : heads(heads_), n_tiles(n_tiles_) {
    tile = blockIdx.x / heads;
    h = blockIdx.x - tile * heads;
    step_tiles = gridDim.x / heads;
    step_heads = gridDim.x - step_tiles * heads;
  }
  __device__ __forceinline__ bool more() const { return tile < n_tiles; }
  __device__ __forceinline__ void advance() {
    tile += step_tiles;
    h += step_heads;
    if (h >= heads) {
      h -= heads;
      ++tile;
    }
  }
};

// The same items taken in turn by whichever block is free, by a whole warp:
// the first by block index, the others from a counter that starts at 0.  The
// next claim and its list entry are on their way while one is worked on.
struct ItemClaims {
  int* counter;
  const TileItem* items;
  int heads, total, claimed;
  TileItem entry;
  __device__ __forceinline__ ItemClaims(int* counter_, const TileItem* items_, int heads_, int n_tiles)
      : counter(counter_), items(items_), heads(heads_), total(n_tiles * heads_), claimed(blockIdx.x) {
    fetch();
  }
  __device__ __forceinline__ void fetch() { entry = items[claimed < total ? claimed / heads : 0]; }
  // The next item and its head; false when none is left.
  __device__ __forceinline__ bool take(TileItem* e, int* h) {
    if (claimed >= total) return false;
    *e = entry;
    *h = claimed % heads;
    int c = 0;
    if ((threadIdx.x & 31) == 0) c = atomicAdd(counter, 1);
    claimed = __shfl_sync(0xffffffffu, c, 0) + gridDim.x;
    fetch();
    return true;
  }
};

// Tiles of both lists: sum of ceil(n_b / kTile) <= n / kTile + B.
__host__ __device__ inline int64_t max_tiles(int64_t n, int B) { return n / kTile + B; }

// Sinks that the query at position p of nk keys sees: keys 0 .. n - 1.
__device__ __forceinline__ int sinks_of(const AttnMask& m, int p) {
  return m.causal ? min(m.sinks, p + 1) : m.sinks;
}

// Key tiles of kSize keys that some query at positions p0 .. p1 sees: first
// `before` tiles over the sinks [0, s), then tiles from key `first` (a
// multiple of 16) up to `end`.  A tile holds the keys from start(j) on,
// extent(j) of them.
template <int kSize>
struct KeyTiles {
  int before, first, end, s, count;
  __device__ __forceinline__ int start(int j) const { return j < before ? j * kSize : first + (j - before) * kSize; }
  __device__ __forceinline__ int extent(int j) const { return min(kSize, (j < before ? s : end) - start(j)); }
};
template <int kSize>
__device__ __forceinline__ KeyTiles<kSize> key_tiles(const AttnMask& m, int p0, int p1, int nk) {
  KeyTiles<kSize> k;
  k.s = max(min(sinks_of(m, p1), nk), 0);
  k.end = min(nk, p1 + m.right + 1);
  k.first = max(0, p0 - m.left) & ~15;
  if (k.end <= k.first) {  // no window: the sinks alone
    k.first = 0;
    k.end = k.s;
  } else if (k.s > 0 && k.s + kSize > k.first) {  // sinks that reach the window's tiles, or nearly: one run of tiles
    k.first = 0;
    k.end = max(k.end, k.s);
  }
  k.before = k.first > 0 ? (k.s + kSize - 1) / kSize : 0;
  k.count = k.before + (k.end - k.first + kSize - 1) / kSize;
  return k;
}

// The keys that some query of a whole event sees, counted through: the sinks,
// then the window's.
struct FewSpan {
  int s, lo, hi;
  __device__ __forceinline__ int count() const { return s + max(hi - lo, 0); }
  __device__ __forceinline__ int key(int v) const { return v < s ? v : lo + (v - s); }
};
__device__ __forceinline__ FewSpan few_span(const AttnMask& m, int nq, int nk) {
  FewSpan f;
  f.s = max(min(sinks_of(m, nk - 1), nk), 0);
  f.lo = max(max(0, nk - nq - m.left), f.s);
  f.hi = min(nk, nk + m.right);
  return f;
}

// The same for one query, at position p.
__device__ __forceinline__ FewSpan row_span(const AttnMask& m, int p, int nk) {
  FewSpan f;
  f.s = max(min(sinks_of(m, p), nk), 0);
  f.lo = max(max(0, p - m.left), f.s);
  f.hi = min(nk, p + m.right + 1);
  return f;
}
// Queries that see so few keys take their D from attention_backward_rows.cu.
constexpr int kFewKeys = 16;
__device__ __forceinline__ bool few_keys(const AttnMask& m, int p, int nk) {
  return row_span(m, p, nk).count() <= kFewKeys;
}
// Whether an event may have such queries: but for few keys or a narrow window
// they stand before the first key, or are the first ones under a causal mask.
__device__ __forceinline__ bool may_see_few(const AttnMask& m, int nq, int nk) {
  return m.causal || nk <= kFewKeys || m.left < kFewKeys || nq > nk;
}

// Positions of the queries that see key j, as [lo, hi].
struct ColumnSpan {
  int lo, hi;
};
__device__ __forceinline__ ColumnSpan column_span(const AttnMask& m, int j) {
  ColumnSpan c;
  c.lo = j - m.right;
  c.hi = j + m.left;
  if (j < m.sinks) {
    c.hi = kFar;
    if (!m.causal) c.lo = -kFar;
  }
  return c;
}

// Queries [lo, hi) of the nq that see some key of the `rows` keys from `at` on:
// the first key's lower and the last key's upper bound; a tile with a sink in
// it is seen to the end.
__device__ __forceinline__ void queries_of(const AttnMask& m, int at, int rows, int shift, int nq, int* lo, int* hi) {
  const ColumnSpan first = column_span(m, at), last = column_span(m, at + rows - 1);
  *lo = min(max(first.lo - shift, 0), nq);
  *hi = min(max(max(first.hi, last.hi) - shift + 1, 0), nq);
}

// Bits lo .. hi - 1 of a word, bounds clipped to 0 .. 32.
__device__ __forceinline__ uint32_t bits(int lo, int hi) {
  lo = max(lo, 0);
  hi = min(hi, 32);
  return hi <= lo ? 0u : (0xffffffffu >> (32 - hi)) & (0xffffffffu << lo);
}

// The keys k .. k + 31 against the queries at positions pa .. pb: whether some
// pair sees one another, and whether every pair does.
__device__ __forceinline__ bool some_seen(const AttnMask& m, int pa, int pb, int k) {
  return (k + 31 >= pa - m.left && k <= pb + m.right) || k < sinks_of(m, pb);
}
__device__ __forceinline__ bool all_seen(const AttnMask& m, int pa, int pb, int k) {
  return (k >= pb - m.left && k + 31 <= pa + m.right) || k + 31 < sinks_of(m, pa);
}
// Those of the keys k .. k + 31 that the query at position p sees.
__device__ __forceinline__ uint32_t seen_keys(const AttnMask& m, int p, int k) {
  return bits(p - m.left - k, p + m.right + 1 - k) | bits(0, sinks_of(m, p) - k);
}

template <typename T>
__device__ __forceinline__ uint32_t pack16(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack16<__nv_bfloat16>(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack16<__half>(float lo, float hi) {
  __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// a * b + c of two values at once.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(d)
      : "l"(pack2(a.x, a.y)), "l"(pack2(b.x, b.y)), "l"(pack2(c.x, c.y)));
  return make_float2(lo2(d), hi2(d));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  const uint64_t d = add2(pack2(a.x, a.y), pack2(b.x, b.y));
  return make_float2(lo2(d), hi2(d));
}

__device__ __forceinline__ float log2_approx(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// The largest power of two c <= 1 / M, M^2 being the product of an event's
// largest |dO_i|^2 and |V_j|^2: M < 2^((x + 1) / 2) with x = floor(log2 M^2).
__device__ __forceinline__ float range_scale(float dout2, float v2) {
  const float m2 = dout2 * v2;  // from 2^-96 to 2^78 for float16 values
  if (!(m2 > 0.f)) return 1.f;
  const int e = (((__float_as_int(m2) >> 23) - 127) + 2) >> 1;
  return __int_as_float((127 - e) << 23);
}

// One row's kCols float32 accumulator columns from TMEM to memory, times f,
// rounded: whole 32-byte sectors per thread where rows start on them, else 16
// bytes (sectors took the forward over 4096 events of up to 128 tokens, 12 heads
// of 64, from 682 to 642 us, the backward over 2048 from 1281 to 1100).  Rows past the tile's read TMEM like the others (a warp reads as
// one) and store nothing; columns from D on are not part of the row.
template <typename T, int kCols>
__device__ __forceinline__ void store_row(uint32_t acc, bool live, float f, T* to, int cols, bool sectors) {
#pragma unroll
  for (int c = 0; c < kCols; c += 32) {
    uint32_t o[32];
    tmem_ld32(acc + c, o);
    tmem_wait_ld32(o);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint64_t v = mul2(pack2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1])), pack2(f, f));
      o[i] = pack16<T>(lo2(v), hi2(v));
    }
    if (!live) continue;
    if (sectors) {
#pragma unroll
      for (int i = 0; i < 16; i += 8)
        if (c + 2 * i < cols)
          asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to + c + 2 * i), "r"(o[i]),
                       "r"(o[i + 1]), "r"(o[i + 2]), "r"(o[i + 3]), "r"(o[i + 4]), "r"(o[i + 5]), "r"(o[i + 6]),
                       "r"(o[i + 7])
                       : "memory");
    } else {
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        if (c + 2 * i < cols)
          *reinterpret_cast<uint4*>(to + c + 2 * i) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
    }
  }
}

template <typename T>
__device__ __forceinline__ float2 unpack16(uint32_t v);
template <>
__device__ __forceinline__ float2 unpack16<__nv_bfloat16>(uint32_t v) {
  return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&v));
}
template <>
__device__ __forceinline__ float2 unpack16<__half>(uint32_t v) {
  return __half22float2(*reinterpret_cast<__half2*>(&v));
}

// d += a b^T for 16 rows of a and 8 of b, 16 values of the sum.
template <typename T>
__device__ __forceinline__ void mma16(float* d, const uint32_t* a, const uint32_t* b) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// Products run over 64 rows of a tile at a time.  Past the rows a tile
// takes (`extent`) the weights are 0, and what follows is rows of the same
// event up to its last (`left` rows from the tile's first), then those of
// another event or of nothing, which must not reach this one: they are set to
// 0, by `threads` threads.  Returns whether there are any to set.
__device__ __forceinline__ bool rows_to_clear(int extent, int left) { return left < ((extent + 63) & ~63); }
template <int kPanels, int kTileRows = kTile>
__device__ __forceinline__ void clear_rows(uint8_t* tile, int extent, int left, int thread, int threads) {
  const int rows = ((extent + 63) & ~63) - left;
#pragma unroll 1
  for (int e = thread; e < rows * 8 * kPanels; e += threads) {
    const int r = left + e / (8 * kPanels), c = e % (8 * kPanels);
    *reinterpret_cast<uint4*>(tile + (c >> 3) * (kTileRows * 128) + r * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
  }
}

// `values` 16-bit values (a multiple of 8) of `rows` rows to 0, by one warp.
template <typename T>
__device__ __forceinline__ void clear_strided(T* base, int rows, int64_t stride, int values) {
#pragma unroll 1
  for (int r = 0; r < rows; ++r)
#pragma unroll 1
    for (int c = (threadIdx.x & 31) * 8; c < values; c += 256)
      *reinterpret_cast<uint4*>(base + r * stride + c) = make_uint4(0, 0, 0, 0);
}

// Whether the offsets tell which rows lie behind the last event.
__device__ __forceinline__ bool rows_known(const WsHeader* hdr) { return hdr->status != kDevBadOffsets; }

// Rows [first, n) of a [n, row_values] 16-bit tensor to 0, over the whole grid.
__device__ __forceinline__ void zero_rows(void* base, int64_t first, int64_t n, int64_t row_values) {
  if (first < 0 || first >= n) return;
  uint4* p = reinterpret_cast<uint4*>(static_cast<char*>(base) + first * row_values * 2);
  const int64_t total = (n - first) * row_values / 8;
#pragma unroll 1
  for (int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; e < total; e += (int64_t)gridDim.x * blockDim.x)
    p[e] = make_uint4(0, 0, 0, 0);
}

// A forward's rows of no event, [first, n): out to 0 and lse to -inf, as
// FPS_TAIL_* says.
__device__ __forceinline__ void clear_tail(int which, void* out, float* lse, int64_t first, int64_t n, int heads, int D) {
  if (which & FPS_TAIL_OUT) zero_rows(out, first, n, (int64_t)heads * D);
  if (!(which & FPS_TAIL_LSE) || !lse || first < 0 || first >= n) return;
#pragma unroll 1
  for (int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; e < (n - first) * heads; e += (int64_t)gridDim.x * blockDim.x)
    lse[e / (n - first) * n + first + e % (n - first)] = -INFINITY;
}

}  // namespace fpstok
