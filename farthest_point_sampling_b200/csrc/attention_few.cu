// Attention of packed events for events with few query rows: a summary query
// per event, tokens generated one at a time, or tiny events.
//
// An event whose queries times the heads of a group are at most 16 fills one
// 16-row matrix tile per key head (row = query * group + head), so keys and
// values are read once for the whole group.  Such a call is bound by reading
// K and V: what counts is that every SM has copies in flight, not the products
// (mma.sync with M = 16; a 128-row tcgen05 tile would be seven eighths empty).
//
// The keys the event sees are cut into chunks of C, one block per chunk and
// key head: four warps take 16 keys each of a 64-key tile, copied to shared
// memory by cp.async some tiles ahead, and keep a running maximum, sum and
// output of their own; the block joins its warps' and, where the event has one
// chunk, writes the result.  Otherwise it leaves (m, l, O) in the workspace and
// a second kernel joins the chunks, in order.  One query for each of 8 events
// of 50000 to 200000 tokens, 12 query and 4 key heads of 64: 206 us, 5.0 TB/s.
#include <type_traits>

#include "attention_few.h"
#include "attention_plan.h"
#include "attention_tiles.cuh"
#include "common.cuh"
#include "internal.h"

namespace fpstok {

namespace {

constexpr int kFewThreads = 128;
constexpr int kFewTile = 64;  // keys of one stage: 16 per warp

template <int DP>
struct FewShape {
  static constexpr int kRow = DP * 2 + 16;  // bytes of a row in shared memory: 16 more, so that 8 rows of a column
                                            // of 16-byte chunks fall on different banks
  static constexpr int kStages = DP == 64 ? 4 : 3;
  static constexpr int kBlocks = DP == 64 ? 3 : 2;  // on an SM, by shared memory
  static constexpr int kTileBytes = kFewTile * kRow;
  static constexpr size_t kSmem = kFewRows * kRow + kStages * 2 * kTileBytes;
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool real) {
  const int n = real ? 16 : 0;  // 0: the 16 bytes become zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}
__device__ __forceinline__ void ldmatrix(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_trans(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
struct FewArgs {
  const void *q, *k, *v;
  int64_t q_token, q_head, k_token, k_head, v_token, v_head;
  int64_t n_q;
  int heads, kv_heads, group, D;
  int chunk;  // keys of one
  AttnMask mask;
  float scale, scale_log2;
  void* out;
  float* lse;
  const TileItem* units;
  const JoinItem* joins;
  float* part_o;    // [slot][key head][16][DP]
  float2* part_ml;  // [slot][key head][16]
  const int64_t* q_offsets;
  int B, zero_tail;
  WsHeader* hdr;
};

template <typename T, int DP>
__global__ void __launch_bounds__(kFewThreads, FewShape<DP>::kBlocks) k_attn_few(const FewArgs a) {
  using Sh = FewShape<DP>;
  extern __shared__ __align__(16) uint8_t s_raw[];
  const uint32_t s_q = smem_u32(s_raw), s_kv = s_q + kFewRows * Sh::kRow;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // the columns past D of every row stay zero: copies never touch them
  for (int e = tid; e < (int)(Sh::kSmem / 16); e += kFewThreads)
    reinterpret_cast<uint4*>(s_raw)[e] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int n_units = a.hdr->n_items[kFewUnits];
  const int row_chunks = a.D / 8;
  ItemWalk walk(a.kv_heads, n_units);
  for (; walk.more(); walk.advance()) {
    const TileItem u = a.units[walk.tile];
    const int g = walk.h, rows = u.nq * a.group, n_chunks = u.pad[0], slot = u.pad[1];
    const FewSpan span = few_span(a.mask, u.nq, u.nk);
    const int v0 = u.t * a.chunk, v1 = min(v0 + a.chunk, span.count());
    const int tiles = (v1 - v0 + kFewTile - 1) / kFewTile;
    const T* kb = static_cast<const T*>(a.k) + u.k0 * a.k_token + g * a.k_head;
    const T* vb = static_cast<const T*>(a.v) + u.k0 * a.v_token + g * a.v_head;
    const auto load = [&](int t) {
      const uint32_t to = s_kv + (t % Sh::kStages) * 2 * Sh::kTileBytes;
      const int c = tid % (DP / 8);
      if (c < row_chunks)
#pragma unroll
      for (int r = tid / (DP / 8); r < kFewTile; r += kFewThreads / (DP / 8)) {
        const int at = v0 + t * kFewTile + r;
        const bool real = at < v1;
        const int64_t j = real ? span.key(at) : 0;
        const uint32_t dst = to + r * Sh::kRow + c * 16;
        copy16(dst, kb + j * a.k_token + c * 8, real);
        copy16(dst + Sh::kTileBytes, vb + j * a.v_token + c * 8, real);
      }
    };
    for (int e = tid; e < kFewRows * row_chunks; e += kFewThreads) {
      const int r = e / row_chunks, c = e - r * row_chunks;
      const bool real = r < rows;
      const int64_t i = real ? r / a.group : 0, h = g * a.group + (real ? r - i * a.group : 0);
      copy16(s_q + r * Sh::kRow + c * 16, static_cast<const T*>(a.q) + (u.q0 + i) * a.q_token + h * a.q_head + c * 8, real);
    }
#pragma unroll
    for (int t = 0; t < Sh::kStages - 1; ++t) {
      if (t < tiles) load(t);
      copy_commit();
    }
    float o[DP / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int d = 0; d < DP / 8; ++d) o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.f;
    uint32_t qf[DP / 16][4];
    for (int t = 0; t < tiles; ++t) {
      copy_wait<Sh::kStages - 2>();
      __syncthreads();  // tile t is there for all, and all are done with the tile before it
      if (t + Sh::kStages - 1 < tiles) load(t + Sh::kStages - 1);
      copy_commit();
      if (t == 0) {
#pragma unroll
        for (int k = 0; k < DP / 16; ++k)
          ldmatrix(qf[k], s_q + (lane & 15) * Sh::kRow + k * 32 + (lane >> 4) * 16);
      }
      const int first = v0 + t * kFewTile + warp * 16;  // this warp's 16 keys
      if (first >= v1) continue;
      const uint32_t kt = s_kv + (t % Sh::kStages) * 2 * Sh::kTileBytes + warp * 16 * Sh::kRow;
      float s[2][4] = {};
#pragma unroll
      for (int k = 0; k < DP / 16; ++k) {
        uint32_t b[4];
        ldmatrix(b, kt + ((lane & 7) + (lane >> 4) * 8) * Sh::kRow + k * 32 + ((lane >> 3) & 1) * 16);
        mma16<T>(s[0], qf[k], b);
        mma16<T>(s[1], qf[k], b + 2);
      }
      // row lane / 4 (+ 8), keys (lane % 4) * 2 + {0, 1} of each 8
      if (first + 16 > v1 || u.nq > 1) {
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int at = first + x * 8 + (lane & 3) * 2 + (y & 1);
            const int p = ((lane >> 2) + (y >> 1) * 8) / a.group + u.nk - u.nq;
            const int j = span.key(at);
            const bool seen = (j >= p - a.mask.left && j <= p + a.mask.right) || j < sinks_of(a.mask, p);
            if (at >= v1 || !seen) s[x][y] = -INFINITY;
          }
      }
      uint32_t pf[4];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        float top = fmaxf(fmaxf(s[0][2 * y], s[0][2 * y + 1]), fmaxf(s[1][2 * y], s[1][2 * y + 1]));
        top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
        top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
        if (__any_sync(kFull, top > m[y])) {
          const float now = fmaxf(m[y], top);
          const float f = m[y] == -INFINITY ? 0.f : exp2_approx((m[y] - now) * a.scale_log2);
          m[y] = now;
          l[y] *= f;
#pragma unroll
          for (int d = 0; d < DP / 8; ++d) {
            o[d][2 * y] *= f;
            o[d][2 * y + 1] *= f;
          }
        }
        const float base = m[y] == -INFINITY ? 0.f : m[y] * a.scale_log2;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float e0 = exp2_approx(fmaf(s[x][2 * y], a.scale_log2, -base));
          const float e1 = exp2_approx(fmaf(s[x][2 * y + 1], a.scale_log2, -base));
          l[y] += e0 + e1;
          pf[x * 2 + y] = pack16<T>(e0, e1);
        }
      }
#pragma unroll
      for (int d = 0; d < DP / 16; ++d) {
        uint32_t b[4];
        ldmatrix_trans(b, kt + Sh::kTileBytes + (lane & 15) * Sh::kRow + d * 32 + (lane >> 4) * 16);
        mma16<T>(o[2 * d], pf, b);
        mma16<T>(o[2 * d + 1], pf, b + 2);
      }
    }
    copy_wait<0>();
    __syncthreads();  // the tiles are free: the warps' results take their place
    float* w_o = reinterpret_cast<float*>(s_raw + kFewRows * Sh::kRow);  // [warp][16][DP]
    float2* w_ml = reinterpret_cast<float2*>(w_o + 4 * kFewRows * DP);   // [warp][16]
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int r = (lane >> 2) + y * 8;
      float sum = l[y];
      sum += __shfl_xor_sync(kFull, sum, 1);
      sum += __shfl_xor_sync(kFull, sum, 2);
      if ((lane & 3) == 0) w_ml[warp * kFewRows + r] = make_float2(m[y], sum);
#pragma unroll
      for (int d = 0; d < DP / 8; ++d)
        *reinterpret_cast<float2*>(w_o + (warp * kFewRows + r) * DP + d * 8 + (lane & 3) * 2) =
            make_float2(o[d][2 * y], o[d][2 * y + 1]);
    }
    __syncthreads();
    for (int e = tid; e < rows * (DP / 4); e += kFewThreads) {
      const int r = e / (DP / 4), c = (e - r * (DP / 4)) * 4;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < 4; ++w) top = fmaxf(top, w_ml[w * kFewRows + r].x);
      float sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float2 ml = w_ml[w * kFewRows + r];
        // nothing seen: what its output holds is not a number to add.  Scores that
        // are all NaN leave the maximum at -inf too, and a sum of NaN, which goes on.
        if (ml.x == -INFINITY && ml.y == 0.f) continue;
        const float f = exp2_approx((ml.x - top) * a.scale_log2);
        const float4 x = *reinterpret_cast<const float4*>(w_o + (w * kFewRows + r) * DP + c);
        sum = fmaf(ml.y, f, sum);
        acc.x = fmaf(x.x, f, acc.x);
        acc.y = fmaf(x.y, f, acc.y);
        acc.z = fmaf(x.z, f, acc.z);
        acc.w = fmaf(x.w, f, acc.w);
      }
      const int64_t i = u.q0 + r / a.group;
      const int h = g * a.group + r % a.group;
      if (n_chunks > 1) {
        const int64_t at = (int64_t)(slot + u.t) * a.kv_heads + g;
        *reinterpret_cast<float4*>(a.part_o + (at * kFewRows + r) * DP + c) = acc;
        if (c == 0) a.part_ml[at * kFewRows + r] = make_float2(top, sum);
      } else {
        if (c < a.D) {
          const float inv = sum == 0.f ? 0.f : 1.f / sum;
          *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + (i * a.heads + h) * a.D + c) =
              make_uint2(pack16<T>(acc.x * inv, acc.y * inv), pack16<T>(acc.z * inv, acc.w * inv));
        }
        if (c == 0 && a.lse) a.lse[h * a.n_q + i] = sum == 0.f ? -INFINITY : fmaf(top, a.scale, log2_approx(sum) * kLn2);
      }
    }
    __syncthreads();
    // the next item's copies write over these floats; its columns past D must read as zeros again
    if (a.D < DP)
      for (int e = tid; e < (int)((4 * kFewRows * DP * 4 + 4 * kFewRows * 8) / 16); e += kFewThreads)
        reinterpret_cast<uint4*>(w_o)[e] = make_uint4(0, 0, 0, 0);
    __syncthreads();
  }
  if (a.zero_tail && rows_known(a.hdr))
    clear_tail(a.zero_tail, a.out, a.lse, a.B > 0 ? a.q_offsets[a.B] : 0, a.n_q, a.heads, a.D);
}

// Joins the chunks of one event and head: sum_c 2^(m_c - M) (l_c, O_c); a
// chunk that saw nothing has l = 0 and O = 0, one that saw only NaN has a l of
// NaN, which 0 times it stays.  The threads of a column take every eighth (or
// fourth) chunk, and their sums are added in order.
template <typename T, int DP>
__global__ void __launch_bounds__(kFewThreads) k_attn_join(const FewArgs a) {
  constexpr int kColumns = DP / 4, kParts = kFewThreads / kColumns;
  __shared__ float4 s_acc[kParts][kColumns];
  __shared__ float s_sum[kParts], s_top[kFewThreads / 32];
  const int tid = threadIdx.x, c = tid % kColumns, part = tid / kColumns;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  ItemWalk walk(a.heads, a.hdr->n_items[kFewJoins]);
  for (; walk.more(); walk.advance()) {
    const JoinItem e = a.joins[walk.tile];
    const int h = walk.h, g = h / a.group;
    for (int i = 0; i < e.nq; ++i) {
      const int r = i * a.group + h - g * a.group;
      const auto at = [&](int k) { return ((int64_t)(e.slot + k) * a.kv_heads + g) * kFewRows + r; };
      float top = -INFINITY;
      for (int k = tid; k < e.chunks; k += kFewThreads) top = fmaxf(top, a.part_ml[at(k)].x);
#pragma unroll
      for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
      if ((tid & 31) == 0) s_top[tid >> 5] = top;
      __syncthreads();
      top = fmaxf(fmaxf(s_top[0], s_top[1]), fmaxf(s_top[2], s_top[3]));
      float sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int k = part; k < e.chunks; k += kParts) {
        const float2 ml = a.part_ml[at(k)];
        const float4 x = *reinterpret_cast<const float4*>(a.part_o + at(k) * DP + c * 4);
        const float f = ml.x == -INFINITY ? 0.f : exp2_approx((ml.x - top) * a.scale_log2);
        sum = fmaf(ml.y, f, sum);
        acc.x = fmaf(x.x, f, acc.x);
        acc.y = fmaf(x.y, f, acc.y);
        acc.z = fmaf(x.z, f, acc.z);
        acc.w = fmaf(x.w, f, acc.w);
      }
      s_acc[part][c] = acc;
      if (c == 0) s_sum[part] = sum;
      __syncthreads();
      if (part == 0) {
        sum = s_sum[0];
#pragma unroll
        for (int p = 1; p < kParts; ++p) {
          const float4 x = s_acc[p][c];
          sum += s_sum[p];
          acc.x += x.x;
          acc.y += x.y;
          acc.z += x.z;
          acc.w += x.w;
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        if (c * 4 < a.D)
          *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + ((int64_t)(e.q0 + i) * a.heads + h) * a.D + c * 4) =
              make_uint2(pack16<T>(acc.x * inv, acc.y * inv), pack16<T>(acc.z * inv, acc.w * inv));
        if (c == 0 && a.lse)
          a.lse[h * a.n_q + e.q0 + i] = sum == 0.f ? -INFINITY : fmaf(top, a.scale, log2_approx(sum) * kLn2);
      }
      __syncthreads();
    }
  }
}

template <typename K>
cudaError_t start(K kernel, const FewArgs& a, int64_t blocks, size_t smem, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(blocks < 1 ? 1 : blocks));
  cfg.blockDim = dim3(kFewThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  count_launch();
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <typename T, int DP>
cudaError_t run(const AttnCall& c, const FewArgs& a, cudaStream_t s) {
  using Sh = FewShape<DP>;
  static_assert(4 * kFewRows * DP * 4 + 4 * kFewRows * 8 <= Sh::kStages * 2 * Sh::kTileBytes, "results over the tiles");
  cudaError_t e = allow_shared_memory(reinterpret_cast<const void*>(k_attn_few<T, DP>), (int)Sh::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t sms = device_info().sm_count;
  const int64_t units = (c.n_kv / a.chunk + c.B) * c.kv_heads, joins = (c.n_kv / a.chunk) * c.heads;
  if ((e = start(k_attn_few<T, DP>, a, units < sms * Sh::kBlocks ? units : sms * Sh::kBlocks, Sh::kSmem, s)) != cudaSuccess)
    return e;
  // an event of one chunk needs no joining, and fewer keys than two chunks hold no other
  if (c.n_kv <= a.chunk) return cudaSuccess;
  return start(k_attn_join<T, DP>, a, joins < sms * 4 ? joins : sms * 4, 0, s);
}

}  // namespace

int few_chunk(int64_t n_kv, int kv_heads) {
  // enough chunks for four rounds of three blocks on each of 148 SMs, none
  // below 256 keys; sizes a workspace, so it does not ask which device it is
  const int64_t items = 148 * 12;
  int64_t c = (n_kv * kv_heads + items - 1) / items;
  c = (c + kFewTile - 1) / kFewTile * kFewTile;
  return (int)(c < 256 ? 256 : c);
}

size_t few_partial_floats(int64_t n_kv, int kv_heads, int D, int chunk) {
  // an event of several chunks has fewer than 2 n / C of them
  return (size_t)(2 * (n_kv / chunk) + 1) * kv_heads * kFewRows * ((D <= 64 ? 64 : 128) + 2);
}

cudaError_t launch_attention_few(const AttnCall& c, const FewPlan& plan, WsHeader* hdr, cudaStream_t s) {
  FewArgs a;
  a.q = c.q;
  a.k = c.k;
  a.v = c.v;
  a.q_token = c.q_token;
  a.q_head = c.q_head;
  a.k_token = c.k_token;
  a.k_head = c.k_head;
  a.v_token = c.v_token;
  a.v_head = c.v_head;
  a.n_q = c.n_q;
  a.heads = c.heads;
  a.kv_heads = c.kv_heads;
  a.group = c.group;
  a.D = c.D;
  a.chunk = plan.chunk;
  a.mask = c.mask;
  a.scale = c.scale;
  a.scale_log2 = c.scale * kLog2e;
  a.out = c.out;
  a.lse = c.lse;
  a.units = plan.units;
  a.joins = plan.joins;
  const int64_t slots = (2 * (c.n_kv / plan.chunk) + 1) * c.kv_heads * kFewRows;
  a.part_ml = reinterpret_cast<float2*>(plan.partial);
  a.part_o = plan.partial + 2 * slots;
  a.q_offsets = c.q_offsets;
  a.B = c.B;
  a.zero_tail = c.zero_tail;
  a.hdr = hdr;
  if (c.dtype == FPS_DTYPE_BF16) return c.D <= 64 ? run<__nv_bfloat16, 64>(c, a, s) : run<__nv_bfloat16, 128>(c, a, s);
  return c.D <= 64 ? run<__half, 64>(c, a, s) : run<__half, 128>(c, a, s);
}

}  // namespace fpstok
