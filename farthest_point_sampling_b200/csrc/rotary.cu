// Rotary positions over several coordinate axes (graphnet PR #923, "What is
// added": a 4D rotary embedding beside the tokenizer; the axes are the
// coordinates of a token).
//
// Pair p of a head belongs to axis a(p) and turns by theta = pos[t, a(p)] *
// w_p:  y1 = x1 cos - x2 sin,  y2 = x2 cos + x1 sin; the inverse (which is
// also the gradient, the rotation being orthogonal) turns by -theta.
//
// Angles: the table holds turns per unit, f = w / 2 pi, as a float pair
// (hi, lo).  pos * f is formed as hi product + its exact rounding error + lo
// product, whole turns are dropped from the hi product exactly, and
// sincospi takes what is left.  The angle's error then stays near 2^-24
// turns for positions of any size a detector gives (times of 1e4 ns and up
// at 1 rad per ns), where a float32 product would lose three digits.
//
// What bounds it: memory.  A block takes a few tokens, forms each token's
// sines and cosines once in shared memory and applies them to all of the
// token's heads with 16-byte loads and stores.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"
#include "rotary.h"

namespace fpstok {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTile = 16;     // tokens of one block
// (token, head) rows that a thread has on the way, every load before the first
// store.  Float32 rows, two at once: 256 events (30,691 tokens x 10 heads x 72)
// 43 -> 41 us.  16-bit rows, one at once in at least six blocks an SM: 446,880
// tokens x 24 heads x 64 take 495 us; two at once 599, four 933, because a
// block then reads from as many more places at a time.
template <typename T>
constexpr int kRowsOf = sizeof(T) == 4 ? 2 : 1;
template <typename T>
constexpr int kBlocksOf = sizeof(T) == 4 ? 1 : 6;

template <typename T>
__device__ __forceinline__ float to_float(T v);
template <>
__device__ __forceinline__ float to_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_float<__half>(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }

// V values moved together: 16 bytes, or one value where rows are not 16-byte
// aligned or pairs do not fill whole vectors.
template <typename T, int V>
struct alignas(V * sizeof(T)) Vec {
  T v[V];
};

struct Shape {
  int64_t T;
  int H, D, R;           // R pairs
  int64_t x_token, x_head, y_token, y_head;
  const float* positions;
  int64_t position_stride;
  float sign;
  int tile;
  int copy_rest;         // 0 when y is x: what does not turn is in place already
};

// One unit of a head: V pairs as two vectors p and p + R (halves layout), one
// vector of V / 2 pairs (interleaved layout; two values for V = 1), or one
// vector of the part that does not turn.
template <typename T, int V, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, kBlocksOf<T>) k_rotary(const T* x, T* y, const Shape s,
                                                     const __grid_constant__ fps_rotary_table table) {
  constexpr int kRowsAtOnce = kRowsOf<T>;
  extern __shared__ float2 s_cs[];  // [tile][R] (cos, sin)
  const int64_t t0 = (int64_t)blockIdx.x * s.tile;
  const int nt = (int)min((int64_t)s.tile, s.T - t0);
  for (int e = threadIdx.x; e < nt * s.R; e += kThreads) {
    const int t = e / s.R, p = e - t * s.R;
    const float pos = s.positions[(t0 + t) * s.position_stride + table.axis[p]];
    const float hi = pos * table.turns_hi[p];
    const float lo = fmaf(pos, table.turns_lo[p], fmaf(pos, table.turns_hi[p], -hi));
    const float turn = (hi - rintf(hi)) + lo;
    float sn, cs;
    sincospif(2.f * turn, &sn, &cs);
    s_cs[e] = make_float2(cs, s.sign * sn);
  }
  __syncthreads();
  constexpr int kPairVec = kInterleaved ? (V > 1 ? V / 2 : 1) : V;  // pairs of one unit
  const int turn_units = s.R / kPairVec;
  const int units = turn_units + (s.copy_rest ? (s.D - 2 * s.R) / V : 0);
  // thread -> (row group, unit); rows are (token, head) pairs, heads first.
  // A head has at most kThreads units (D <= FPS_MAX_ROTARY_DIM = kThreads).
  const int groups = kThreads / units;
  const int step_t = groups / s.H, step_h = groups - step_t * s.H;
  const int g = threadIdx.x / units, u = threadIdx.x - g * units;
  if (g >= groups) return;
  int t = g / s.H, h = g - t * s.H;
  const bool turns = u < turn_units;
  // vectors of a row that this thread moves: the pair's halves, or one
  const bool two = turns && !(kInterleaved && V > 1);
  const int i1 = !turns                    ? 2 * s.R + (u - turn_units) * V
                 : kInterleaved && V == 1 ? 2 * u
                                          : u * V;
  const int i2 = kInterleaved ? i1 + 1 : i1 + s.R;
  while (t < nt) {
    Vec<T, V> a[kRowsAtOnce], b[kRowsAtOnce];
    int tt[kRowsAtOnce], hh[kRowsAtOnce];
#pragma unroll
    for (int k = 0; k < kRowsAtOnce; ++k) {
      tt[k] = t;
      hh[k] = h;
      if (t < nt) {
        const T* xr = x + (t0 + t) * s.x_token + h * s.x_head;
        a[k] = *reinterpret_cast<const Vec<T, V>*>(xr + i1);
        if (two) b[k] = *reinterpret_cast<const Vec<T, V>*>(xr + i2);
      }
      t += step_t;
      h += step_h;
      if (h >= s.H) {
        h -= s.H;
        ++t;
      }
    }
#pragma unroll
    for (int k = 0; k < kRowsAtOnce; ++k) {
      if (tt[k] >= nt) continue;
      T* yr = y + (t0 + tt[k]) * s.y_token + hh[k] * s.y_head;
      const float2* cs = s_cs + tt[k] * s.R;
      if (turns) {
        if constexpr (kInterleaved && V > 1) {
#pragma unroll
          for (int q = 0; q < V / 2; ++q) {
            const float2 c = cs[u * (V / 2) + q];
            const float a1 = to_float(a[k].v[2 * q]), a2 = to_float(a[k].v[2 * q + 1]);
            a[k].v[2 * q] = from_float<T>(fmaf(a1, c.x, -(a2 * c.y)));
            a[k].v[2 * q + 1] = from_float<T>(fmaf(a2, c.x, a1 * c.y));
          }
        } else {
#pragma unroll
          for (int q = 0; q < V; ++q) {
            const float2 c = cs[u * V + q];
            const float a1 = to_float(a[k].v[q]), a2 = to_float(b[k].v[q]);
            a[k].v[q] = from_float<T>(fmaf(a1, c.x, -(a2 * c.y)));
            b[k].v[q] = from_float<T>(fmaf(a2, c.x, a1 * c.y));
          }
          *reinterpret_cast<Vec<T, V>*>(yr + i2) = b[k];
        }
      }
      *reinterpret_cast<Vec<T, V>*>(yr + i1) = a[k];
    }
  }
}

template <typename T, int V, bool kInterleaved>
cudaError_t launch(const RotaryCall& c, const fps_rotary_table& table, cudaStream_t s) {
  Shape sh;
  sh.T = c.T;
  sh.H = c.H;
  sh.D = c.D;
  sh.R = table.pairs;
  sh.x_token = c.x_token;
  sh.x_head = c.x_head;
  sh.y_token = c.y_token;
  sh.y_head = c.y_head;
  sh.positions = c.positions;
  sh.position_stride = c.position_stride;
  sh.sign = c.inverse ? -1.f : 1.f;
  sh.copy_rest = c.x != c.y;
  // enough blocks for four on every SM before a block takes more than one token
  const int64_t spread = (int64_t)device_info().sm_count * 4;
  if (spread <= 0) return cudaErrorNoDevice;
  int64_t tile = (c.T + spread - 1) / spread;
  sh.tile = (int)(tile < 1 ? 1 : tile > kMaxTile ? kMaxTile : tile);
  const unsigned blocks = (unsigned)((c.T + sh.tile - 1) / sh.tile);
  count_launch();
  k_rotary<T, V, kInterleaved><<<blocks, kThreads, (size_t)sh.tile * sh.R * sizeof(float2), s>>>(
      static_cast<const T*>(c.x), static_cast<T*>(c.y), sh, table);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_type(const RotaryCall& c, const fps_rotary_table& table, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const int R = table.pairs;
  // 16-byte units need every row 16-byte aligned and the turning part, its
  // halves and the rest in whole units
  const bool rows = (reinterpret_cast<uintptr_t>(c.x) | reinterpret_cast<uintptr_t>(c.y)) % 16 == 0 &&
                    (c.x_token | c.x_head | c.y_token | c.y_head) % V == 0 && c.D % V == 0;
  if (table.interleaved)
    return rows && (2 * R) % V == 0 ? launch<T, V, true>(c, table, s) : launch<T, 1, true>(c, table, s);
  return rows && R % V == 0 ? launch<T, V, false>(c, table, s) : launch<T, 1, false>(c, table, s);
}

}  // namespace

cudaError_t launch_rotary(const RotaryCall& c, const fps_rotary_table& table, cudaStream_t s) {
  switch (c.dtype) {
    case FPS_DTYPE_BF16: return launch_type<__nv_bfloat16>(c, table, s);
    case FPS_DTYPE_F16: return launch_type<__half>(c, table, s);
    default: return launch_type<float>(c, table, s);
  }
}

}  // namespace fpstok
