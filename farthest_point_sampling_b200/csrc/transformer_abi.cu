// C ABI of the packed-token transformer operators (declared in
// include/fpstok.h): argument checks and launches.
#include <atomic>
#include <cmath>

#include "../../include/fpstok.h"
#include "attention.h"
#include "internal.h"
#include "rotary.h"

namespace fpstok {

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int from_cuda(cudaError_t e) { return e == cudaSuccess ? FPS_OK : FPS_ERR_CUDA; }
constexpr int64_t kMaxRows = kFar;  // positions, their differences and a window more fit 32 bits
constexpr int64_t kMaxStride = (int64_t)1 << 38;  // elements; a TMA stride is below 2^40 bytes

constexpr int kWaitPolls = 100000;  // 2 s
std::atomic<int> g_wait_polls{kWaitPolls}, g_wait_skip{0};

// Rows of `width` bytes, n of each of `heads`; strides in bytes, 0 or more.
struct Rows {
  const void* base;
  int64_t n, heads, token, head, width;
  int64_t at() const { return (int64_t)reinterpret_cast<uintptr_t>(base); }
  // bytes from the first to the end of the last
  int64_t reach() const { return n == 0 ? 0 : (n - 1) * token + (heads - 1) * head + width; }
};
Rows rows_of(const void* base, int64_t n, int64_t heads, int64_t token, int64_t head, int64_t values, int64_t size) {
  // strides that nothing uses may be anything; none reaches beyond 2^60 bytes
  const auto bytes = [&](int64_t stride, int64_t count) {
    const int64_t most = ((int64_t)1 << 60) / count;
    return stride > most / size ? most : stride * size;
  };
  return {base, n, heads, n > 1 ? bytes(token, n) : 0, heads > 1 ? bytes(head, heads) : 0, values * size};
}
bool apart(const Rows& a, const Rows& b) { return a.at() + a.reach() <= b.at() || b.at() + b.reach() <= a.at(); }

// Whether a row of a set meets one of the same set moved by `by` bytes; the row
// itself does not count.
bool rows_meet(const Rows& r, int64_t by) {
  for (int64_t h = 1 - r.heads; h < r.heads; ++h) {
    const int64_t at = by + h * r.head;
    // the two nearest rows of this head
    const int64_t t0 = r.token > 0 ? (at > 0 ? -((at + r.token - 1) / r.token) : -at / r.token) : 0;
    for (int64_t t = t0; t <= t0 + 1; ++t) {
      const int64_t from = at + t * r.token;
      if (t > -r.n && t < r.n && from > -r.width && from < r.width && !(by == 0 && h == 0 && t == 0)) return true;
    }
  }
  return false;
}
bool rows_meet(const Rows& r) {
  const bool heads_in_rows = r.head >= r.width && r.token >= (r.heads - 1) * r.head + r.width;
  const bool rows_in_heads = r.token >= r.width && r.head >= (r.n - 1) * r.token + r.width;
  return !heads_in_rows && !rows_in_heads && rows_meet(r, 0);
}

// Whether a row meets `bytes` at `base`.
bool block_meets(const void* base, int64_t bytes, const Rows& r) {
  const Rows block = {base, 1, 1, 0, 0, bytes};
  if (bytes == 0 || r.n == 0 || apart(block, r)) return false;
  for (int64_t h = 0; h < r.heads; ++h) {
    const int64_t at = r.at() + h * r.head - block.at();  // row 0 of this head; the first that ends behind the block's start
    const int64_t t = r.token > 0 && at + r.width <= 0 ? -(at + r.width) / r.token + 1 : 0;
    const int64_t from = at + t * r.token;
    if (t < r.n && from < bytes && from + r.width > 0) return true;
  }
  return false;
}

// Sizes only: enough to compute a workspace.
int check_attention_sizes(const fps_attention_args* a) {
  if (!a) return FPS_ERR_ARG;
  if (a->dtype != FPS_DTYPE_BF16 && a->dtype != FPS_DTYPE_F16) return FPS_ERR_ARG;
  if (a->heads < 1 || a->kv_heads < 1 || a->heads % a->kv_heads || a->head_dim < 8 || a->head_dim % 8)
    return FPS_ERR_ARG;
  if ((a->causal != 0 && a->causal != 1) || a->window < -1 || a->sinks < 0) return FPS_ERR_ARG;
  if (a->n_q < 0 || a->n_kv < 0 || a->events < 0 || a->max_tokens < 0) return FPS_ERR_ARG;
  if (a->head_dim > FPS_MAX_ATTENTION_DIM || a->heads > 65535 || a->n_q >= kMaxRows || a->n_kv >= kMaxRows)
    return FPS_ERR_TOO_LARGE;
  // work items (tiles of at least 64 rows, times heads) are counted in 32 bits
  const int64_t rows = a->n_q > a->n_kv ? a->n_q : a->n_kv;
  if ((rows / 32 + 2 * (int64_t)a->events) * a->heads >= ((int64_t)1 << 31)) return FPS_ERR_TOO_LARGE;
  return FPS_OK;
}

bool row_strides_ok(int64_t token, int64_t head) {
  return token > 0 && head > 0 && token % 8 == 0 && head % 8 == 0 && token < kMaxStride && head < kMaxStride;
}

int make_sizes(const fps_attention_args* a, AttnCall* c) {
  const int rc = check_attention_sizes(a);
  if (rc) return rc;
  *c = AttnCall{};
  c->dtype = a->dtype;
  c->n_q = a->n_q;
  c->n_kv = a->n_kv;
  c->heads = a->heads;
  c->kv_heads = a->kv_heads;
  c->group = a->heads / a->kv_heads;
  c->D = a->head_dim;
  c->B = a->events;
  // positions stay below kMaxRows = kFar: a wider window sees everything
  c->mask.causal = a->causal;
  c->mask.left = a->window < 0 || a->window >= kMaxRows ? kFar : (int)a->window;
  c->mask.right = a->causal ? 0 : c->mask.left;
  c->mask.sinks = c->mask.left == kFar ? 0 : (int)(a->sinks >= kMaxRows ? kMaxRows : a->sinks);
  c->max_tokens = a->max_tokens;
  return FPS_OK;
}

int make_call(const fps_attention_args* a, AttnCall* c) {
  const int rc = make_sizes(a, c);
  if (rc) return rc;
  if (!(a->scale > 0.f) || !std::isfinite(a->scale)) return FPS_ERR_ARG;
  if (a->events > 0 && (!a->q_offsets || !a->kv_offsets)) return FPS_ERR_ARG;
  if (a->n_q > 0 && (!a->q || !aligned(a->q, 16) || !row_strides_ok(a->q_token_stride, a->q_head_stride)))
    return FPS_ERR_ARG;
  if (a->n_kv > 0 && (!a->k || !a->v || !aligned(a->k, 16) || !aligned(a->v, 16) ||
                      !row_strides_ok(a->k_token_stride, a->k_head_stride) ||
                      !row_strides_ok(a->v_token_stride, a->v_head_stride)))
    return FPS_ERR_ARG;
  c->q = a->q;
  c->k = a->k;
  c->v = a->v;
  c->q_token = a->q_token_stride;
  c->q_head = a->q_head_stride;
  c->k_token = a->k_token_stride;
  c->k_head = a->k_head_stride;
  c->v_token = a->v_token_stride;
  c->v_head = a->v_head_stride;
  c->q_offsets = a->q_offsets;
  c->kv_offsets = a->kv_offsets;
  c->scale = a->scale;
  c->zero_tail = a->zero_tail;
  c->test = {g_wait_polls.load(std::memory_order_relaxed), g_wait_skip.load(std::memory_order_relaxed)};
  return FPS_OK;
}

// Whether `bytes` that the call writes meet what it reads.
bool meets_input(const AttnCall& c, const void* base, int64_t bytes) {
  return block_meets(base, bytes, rows_of(c.q, c.n_q, c.heads, c.q_token, c.q_head, c.D, 2)) ||
         block_meets(base, bytes, rows_of(c.k, c.n_kv, c.kv_heads, c.k_token, c.k_head, c.D, 2)) ||
         block_meets(base, bytes, rows_of(c.v, c.n_kv, c.kv_heads, c.v_token, c.v_head, c.D, 2));
}

}  // namespace

}  // namespace fpstok

using namespace fpstok;

extern "C" {

int fps_rotary_table_init(fps_rotary_table* table, const int* axis_dims, int axes, double base,
                          const double* axis_scale, int interleaved) {
  if (!table || !axis_dims || axes < 1 || !(base > 0.0) || !std::isfinite(base)) return FPS_ERR_ARG;
  if (axes > FPS_MAX_ROTARY_AXES) return FPS_ERR_TOO_LARGE;
  int64_t dims = 0;
  for (int a = 0; a < axes; ++a) {
    if (axis_dims[a] < 0 || axis_dims[a] % 2) return FPS_ERR_ARG;
    if (axis_scale && !std::isfinite(axis_scale[a])) return FPS_ERR_ARG;
    dims += axis_dims[a];
  }
  if (dims == 0) return FPS_ERR_ARG;
  if (dims > FPS_MAX_ROTARY_DIM) return FPS_ERR_TOO_LARGE;
  fps_rotary_table t = {};
  t.axes = axes;
  t.interleaved = interleaved != 0;
  const double turns_per_radian = 0.15915494309189533577;  // 1 / 2 pi
  for (int a = 0; a < axes; ++a) {
    const int n = axis_dims[a] / 2;
    for (int i = 0; i < n; ++i) {
      const double w = (axis_scale ? axis_scale[a] : 1.0) * std::pow(base, -(double)i / n) * turns_per_radian;
      if (!(std::fabs(w) < 1e30)) return FPS_ERR_ARG;  // the float pair would overflow
      t.turns_hi[t.pairs] = (float)w;
      t.turns_lo[t.pairs] = (float)(w - (double)t.turns_hi[t.pairs]);
      t.axis[t.pairs] = (unsigned char)a;
      ++t.pairs;
    }
  }
  *table = t;
  return FPS_OK;
}

int fps_rotary(const void* x, void* y, int dtype, int64_t T, int H, int D, int64_t x_token_stride,
               int64_t x_head_stride, int64_t y_token_stride, int64_t y_head_stride, const float* positions,
               int64_t position_stride, const fps_rotary_table* table, int inverse, fps_stream_t stream) {
  if (dtype != FPS_DTYPE_F32 && dtype != FPS_DTYPE_BF16 && dtype != FPS_DTYPE_F16) return FPS_ERR_ARG;
  if (!table || T < 0 || H < 1 || D < 2) return FPS_ERR_ARG;
  if (table->pairs < 1 || table->pairs > FPS_MAX_ROTARY_DIM / 2 || table->axes < 1 ||
      table->axes > FPS_MAX_ROTARY_AXES || 2 * table->pairs > D)
    return FPS_ERR_ARG;
  for (int p = 0; p < table->pairs; ++p)
    if (table->axis[p] >= table->axes) return FPS_ERR_ARG;
  if (D > FPS_MAX_ROTARY_DIM || T >= kMaxRows || H > 65535) return FPS_ERR_TOO_LARGE;
  if (T == 0) return FPS_OK;
  const size_t size = dtype == FPS_DTYPE_F32 ? 4 : 2;
  if (!x || !y || !positions || !aligned(x, size) || !aligned(y, size) || !aligned(positions, 4)) return FPS_ERR_ARG;
  if (position_stride < table->axes || x_token_stride < 0 || x_head_stride < 0) return FPS_ERR_ARG;
  if ((T > 1 && y_token_stride < D) || (H > 1 && y_head_stride < D)) return FPS_ERR_ARG;
  if (x == y && (x_token_stride != y_token_stride || x_head_stride != y_head_stride)) return FPS_ERR_ARG;
  const Rows from = rows_of(x, T, H, x_token_stride, x_head_stride, D, size);
  const Rows to = rows_of(y, T, H, y_token_stride, y_head_stride, D, size);
  if (rows_meet(to)) return FPS_ERR_ARG;
  // x and y among one another with the same strides, such as other heads of the
  // same rows; with other strides only clear of one another
  if (x != y && !apart(from, to) &&
      (from.token != to.token || from.head != to.head || rows_meet(to, from.at() - to.at())))
    return FPS_ERR_ARG;
  RotaryCall c = {x,           y, dtype, T, H, D, x_token_stride, x_head_stride, y_token_stride, y_head_stride,
                  positions, position_stride, inverse != 0};
  return from_cuda(launch_rotary(c, *table, reinterpret_cast<cudaStream_t>(stream)));
}

size_t fps_attention_workspace_bytes(const fps_attention_args* args, int backward) {
  AttnCall c;
  if (make_sizes(args, &c)) return 0;
  return backward ? attention_backward_bytes(c) : attention_forward_bytes(c);
}

int fps_attention(const fps_attention_args* args, void* out, float* lse, void* workspace, size_t workspace_bytes,
                  fps_stream_t stream) {
  AttnCall c;
  const int rc = make_call(args, &c);
  if (rc) return rc;
  if (c.n_q > 0 && (!out || !aligned(out, 16) || !aligned(lse, 4))) return FPS_ERR_ARG;
  const size_t need = fps_attention_workspace_bytes(args, 0);
  if (!workspace || workspace_bytes < need || !aligned(workspace, 256)) return FPS_ERR_WORKSPACE;
  if (meets_input(c, out, c.n_q * c.heads * c.D * 2)) return FPS_ERR_ARG;
  c.out = out;
  c.lse = lse;
  return from_cuda(launch_attention_forward(c, workspace, reinterpret_cast<cudaStream_t>(stream)));
}

int fps_attention_backward(const fps_attention_args* args, const void* out, const float* lse, const void* dout,
                           int64_t dout_token_stride, int64_t dout_head_stride, void* dq, void* dk, void* dv,
                           void* workspace, size_t workspace_bytes, fps_stream_t stream) {
  AttnCall c;
  const int rc = make_call(args, &c);
  if (rc) return rc;
  if (c.n_q > 0 && (!out || !lse || !dout || !dq || !aligned(out, 16) || !aligned(lse, 4) || !aligned(dout, 16) ||
                    !aligned(dq, 16) || !row_strides_ok(dout_token_stride, dout_head_stride)))
    return FPS_ERR_ARG;
  if (c.n_kv > 0 && (!dk || !dv || !aligned(dk, 16) || !aligned(dv, 16))) return FPS_ERR_ARG;
  const size_t need = fps_attention_workspace_bytes(args, 1);
  if (!workspace || workspace_bytes < need || !aligned(workspace, 256)) return FPS_ERR_WORKSPACE;
  const int64_t q_bytes = c.n_q * c.heads * c.D * 2, kv_bytes = c.n_kv * c.kv_heads * c.D * 2;
  const Rows of_out = rows_of(out, 1, 1, 0, 0, q_bytes, 1), of_dq = rows_of(dq, 1, 1, 0, 0, q_bytes, 1);
  const Rows of_dk = rows_of(dk, 1, 1, 0, 0, kv_bytes, 1);
  const Rows of_dout = rows_of(dout, c.n_q, c.heads, dout_token_stride, dout_head_stride, c.D, 2);
  for (int i = 0; i < 3; ++i) {
    const void* base = i == 0 ? dq : i == 1 ? dk : dv;
    const int64_t bytes = i == 0 ? q_bytes : kv_bytes;
    if (meets_input(c, base, bytes) || block_meets(base, bytes, of_out) || block_meets(base, bytes, of_dout) ||
        (i > 0 && block_meets(base, bytes, of_dq)) || (i > 1 && block_meets(base, bytes, of_dk)))
      return FPS_ERR_ARG;
  }
  c.out = const_cast<void*>(out);
  c.lse = const_cast<float*>(lse);
  c.dout = dout;
  c.do_token = dout_token_stride;
  c.do_head = dout_head_stride;
  c.dq = dq;
  c.dk = dk;
  c.dv = dv;
  return from_cuda(launch_attention_backward(c, workspace, reinterpret_cast<cudaStream_t>(stream)));
}

void fps_set_attention_test(int poll_limit, int skip) {
  g_wait_polls = poll_limit > 0 ? poll_limit : kWaitPolls;
  g_wait_skip = skip;
}

}  // extern "C"
