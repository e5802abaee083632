// generation_api.cu -- host side of the generation entry points of
// include/attn.h: rotation plans, argument validation and launches for the
// rotary positions, the paged cache and the one-token attention.
#include <cuda_runtime.h>
#include <math.h>
#include <stddef.h>
#include <stdint.h>
#include <string.h>

#include "generation_internal.h"

namespace attn {
namespace {

constexpr double kPi = 3.14159265358979323846;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// A strided tensor's dimensions outside the innermost one, and its reach.
struct Dims {
  int n = 0;
  int64_t size[3], stride[3];
  void add(int64_t sz, int64_t st) {
    size[n] = sz;
    stride[n] = st;
    ++n;
  }
};

// Elements from the first to behind the last; 0 when it does not fit.
int64_t reach(const Dims& d, int64_t inner) {
  // 2^50 elements are beyond any device, and keep the sums from wrapping
  const int64_t most = (int64_t)1 << 50;
  int64_t r = inner;
  for (int i = 0; i < d.n; ++i) {
    if (d.stride[i] < 0) return 0;
    if (d.size[i] > 1 && d.stride[i] > most / (d.size[i] - 1)) return 0;
    r += (d.size[i] - 1) * d.stride[i];
    if (r > most) return 0;
  }
  return r;
}

// Whether no two elements share an address: taken by stride, each dimension
// steps over all that the smaller ones reach.
bool distinct(Dims d, int64_t inner) {
  int64_t r = inner;
  for (int k = 0; k < d.n; ++k) {
    int at = -1;
    for (int i = 0; i < d.n; ++i)
      if (d.size[i] > 1 && (at < 0 || d.stride[i] < d.stride[at])) at = i;
    if (at < 0) return true;
    if (d.stride[at] < r) return false;
    r += (d.size[at] - 1) * d.stride[at];
    d.size[at] = 1;
  }
  return true;
}

bool same_place(const void* a, const Dims& x, const void* b, const Dims& y) {
  if (a != b) return false;
  for (int i = 0; i < x.n; ++i)
    if (x.size[i] > 1 && x.stride[i] != y.stride[i]) return false;
  return true;
}

// Byte ranges [p, p + n).
bool overlaps(const void* a, uint64_t na, const void* b, uint64_t nb) {
  if (a == nullptr || b == nullptr) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

// Whether the rows {token, head} of y share no element with those of x:
// ranges that do not meet, or parts of one buffer that lie side by side in
// every token (equal token strides).  nx, ny: their reach; bf16.
bool rows_apart(const void* x, const Dims& dx, int64_t nx, const void* y, const Dims& dy,
                int64_t ny, int64_t inner) {
  if (!overlaps(x, 2 * (uint64_t)nx, y, 2 * (uint64_t)ny)) return true;
  const int64_t ts = dx.stride[0];
  if (dx.size[0] <= 1 || ts <= 0 || dy.stride[0] != ts) return false;
  const int64_t rx = inner + (dx.size[1] - 1) * dx.stride[1];
  const int64_t ry = inner + (dy.size[1] - 1) * dy.stride[1];
  const int64_t d = (int64_t)(reinterpret_cast<intptr_t>(y) - reinterpret_cast<intptr_t>(x)) / 2;
  const int64_t at = ((d % ts) + ts) % ts;  // of y's row in x's token
  return at >= rx && at + ry <= ts;
}

// Whether rows can move in accesses of so many bytes: base and row starts.
bool vec_rows(const void* p, const Dims& d, int elem = 2, int bytes = 16) {
  if (!aligned(p, (size_t)bytes)) return false;
  for (int i = 0; i < d.n; ++i)
    if (d.size[i] > 1 && (d.stride[i] * elem) % bytes != 0) return false;
  return true;
}

// The widest access, in elements, of rows of D elements of which plan turns
// the first: two of them hold whole pairs.  Halves that pair must both start
// where an access does; neighbours may stop turning anywhere.
int row_width(int D, const attn_rope_plan* plan) {
  const int whole = plan != nullptr && plan->layout == ATTN_ROPE_HALF ? plan->rot_dim : 0;
  int w = 8;
  while (w > 1 && (D % (2 * w) != 0 || whole % (2 * w) != 0)) w /= 2;
  return w;
}
int row_width(int w, const void* p, const Dims& d) {
  while (w > 1 && !vec_rows(p, d, 2, 2 * w)) w /= 2;
  return w;
}

bool plan_ok(const attn_rope_plan* p) {
  return p != nullptr && p->version == 1u && p->rot_dim >= 2 && p->rot_dim % 2 == 0 &&
         p->rot_dim <= ATTN_ROPE_MAX_DIM &&
         (p->layout == ATTN_ROPE_HALF || p->layout == ATTN_ROPE_INTERLEAVED) &&
         isfinite(p->mscale);
}

attn_status run_rope(const void* x, const int64_t* xs, void* out, const int64_t* os, int B, int H,
                     int S, int D, const int32_t* positions, int64_t pos_stride, int32_t offset,
                     const attn_rope_plan* plan, float sign, attn_stream_t stream) {
  if (x == nullptr || out == nullptr || xs == nullptr || os == nullptr) return ATTN_ERR_INVALID_ARG;
  if (B <= 0 || H <= 0 || S <= 0 || D <= 0 || D % 2 != 0) return ATTN_ERR_INVALID_ARG;
  if (!plan_ok(plan) || plan->rot_dim > D) return ATTN_ERR_INVALID_ARG;
  if (D > 1024) return ATTN_ERR_UNSUPPORTED;
  if ((int64_t)B * S > INT32_MAX) return ATTN_ERR_INVALID_ARG;
  if (!aligned(x, 2) || !aligned(out, 2)) return ATTN_ERR_INVALID_ARG;
  if (positions != nullptr && (!aligned(positions, 4) || pos_stride < 0))
    return ATTN_ERR_INVALID_ARG;
  Dims dx, dy;
  const int64_t sizes[3] = {B, H, S};
  for (int i = 0; i < 3; ++i) {
    dx.add(sizes[i], xs[i]);
    dy.add(sizes[i], os[i]);
  }
  const int64_t nx = reach(dx, D), ny = reach(dy, D);
  if (nx == 0 || ny == 0 || !distinct(dy, D)) return ATTN_ERR_INVALID_ARG;
  if (overlaps(x, 2 * (uint64_t)nx, out, 2 * (uint64_t)ny) && !same_place(x, dx, out, dy))
    return ATTN_ERR_INVALID_ARG;
  if (positions != nullptr) {
    Dims dp;
    dp.add(B, pos_stride);
    const int64_t np = reach(dp, S);
    if (np == 0 || overlaps(positions, 4 * (uint64_t)np, out, 2 * (uint64_t)ny))
      return ATTN_ERR_INVALID_ARG;
  }
  RopeArgs a;
  memset(&a, 0, sizeof(a));
  a.x = static_cast<const __nv_bfloat16*>(x);
  a.out = static_cast<__nv_bfloat16*>(out);
  for (int i = 0; i < 3; ++i) {
    a.xs[i] = xs[i];
    a.os[i] = os[i];
  }
  a.B = B;
  a.H = H;
  a.S = S;
  a.D = D;
  a.positions = positions;
  a.pos_stride = pos_stride;
  a.offset = offset;
  a.sign = sign;
  a.plan = *plan;
  const int width = row_width(row_width(row_width(D, plan), x, dx), out, dy);
  return launch_rope(a, width, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? ATTN_OK
             : ATTN_ERR_CUDA;
}

// Checks of a cache description; the reach of its keys and values in bytes.
attn_status check_cache(const attn_cache_desc* c, uint64_t* k_bytes, uint64_t* v_bytes) {
  if (c == nullptr || c->version != 1u) return ATTN_ERR_INVALID_ARG;
  if (c->dtype != ATTN_CACHE_BF16 && c->dtype != ATTN_CACHE_E4M3) return ATTN_ERR_INVALID_ARG;
  if (c->num_pages <= 0 || c->page_size <= 0 || c->H_kv <= 0 || c->D <= 0)
    return ATTN_ERR_INVALID_ARG;
  if (c->page_size > (1 << 30)) return ATTN_ERR_INVALID_ARG;
  if (c->k == nullptr || c->v == nullptr) return ATTN_ERR_INVALID_ARG;
  if (c->D != 64 && c->D != 128) return ATTN_ERR_UNSUPPORTED;
  const int elem = c->dtype == ATTN_CACHE_BF16 ? 2 : 1;
  if (elem == 2 && (c->k_scale != nullptr || c->v_scale != nullptr)) return ATTN_ERR_INVALID_ARG;
  if (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4)) return ATTN_ERR_INVALID_ARG;
  for (int which = 0; which < 2; ++which) {
    const int64_t* s = which ? c->v_strides : c->k_strides;
    Dims d;
    d.add(c->num_pages, s[0]);
    d.add(c->H_kv, s[1]);
    d.add(c->page_size, s[2]);
    const int64_t n = reach(d, c->D);
    if (n == 0 || !distinct(d, c->D) || !vec_rows(which ? c->v : c->k, d, elem))
      return ATTN_ERR_INVALID_ARG;
    *(which ? v_bytes : k_bytes) = (uint64_t)n * elem;
  }
  return ATTN_OK;
}

}  // namespace
}  // namespace attn

using namespace attn;

extern "C" {

attn_status attn_rope_plan_init(const attn_rope_config* c, attn_rope_plan* plan) {
  if (c == nullptr || plan == nullptr || c->version != 1u) return ATTN_ERR_INVALID_ARG;
  const int rot = c->rot_dim;
  if (rot < 2 || rot % 2 != 0 || rot > ATTN_ROPE_MAX_DIM) return ATTN_ERR_INVALID_ARG;
  if (c->layout != ATTN_ROPE_HALF && c->layout != ATTN_ROPE_INTERLEAVED)
    return ATTN_ERR_INVALID_ARG;
  const int sc = c->scaling;
  if (sc < ATTN_ROPE_SCALE_NONE || sc > ATTN_ROPE_SCALE_CUSTOM) return ATTN_ERR_INVALID_ARG;
  double base = c->base == 0.0 ? 10000.0 : c->base;
  const double factor = c->factor;
  const double fast = c->beta_fast == 0.0 ? 32.0 : c->beta_fast;
  const double slow = c->beta_slow == 0.0 ? 1.0 : c->beta_slow;
  const double low = c->low_factor == 0.0 ? 1.0 : c->low_factor;
  const double high = c->high_factor == 0.0 ? 4.0 : c->high_factor;
  if (sc != ATTN_ROPE_SCALE_CUSTOM && !(isfinite(base) && base > 1.0)) return ATTN_ERR_INVALID_ARG;
  if (sc >= ATTN_ROPE_SCALE_LINEAR && sc <= ATTN_ROPE_SCALE_BANDS &&
      !(isfinite(factor) && factor >= 1.0))
    return ATTN_ERR_INVALID_ARG;
  if (sc == ATTN_ROPE_SCALE_NTK && rot <= 2) return ATTN_ERR_INVALID_ARG;
  if ((sc == ATTN_ROPE_SCALE_YARN || sc == ATTN_ROPE_SCALE_BANDS) &&
      !(isfinite(c->original_len) && c->original_len > 0.0))
    return ATTN_ERR_INVALID_ARG;
  if (sc == ATTN_ROPE_SCALE_YARN &&
      !(isfinite(fast) && isfinite(slow) && slow > 0.0 && fast > slow))
    return ATTN_ERR_INVALID_ARG;
  if (sc == ATTN_ROPE_SCALE_BANDS &&
      !(isfinite(low) && isfinite(high) && low > 0.0 && high > low))
    return ATTN_ERR_INVALID_ARG;
  if (sc == ATTN_ROPE_SCALE_CUSTOM && c->inv_freq == nullptr) return ATTN_ERR_INVALID_ARG;
  if (!(isfinite(c->mscale) && c->mscale >= 0.0)) return ATTN_ERR_INVALID_ARG;
  double m = c->mscale;
  if (m == 0.0) m = sc == ATTN_ROPE_SCALE_YARN ? 0.1 * log(factor) + 1.0 : 1.0;
  if (!isfinite((float)m)) return ATTN_ERR_INVALID_ARG;
  if (sc == ATTN_ROPE_SCALE_NTK) {
    base *= pow(factor, (double)rot / (rot - 2));
    if (!isfinite(base)) return ATTN_ERR_INVALID_ARG;
  }
  double lo = 0.0, hi = 0.0;
  if (sc == ATTN_ROPE_SCALE_YARN) {
    lo = floor(rot * log(c->original_len / (fast * 2.0 * kPi)) / (2.0 * log(base)));
    hi = ceil(rot * log(c->original_len / (slow * 2.0 * kPi)) / (2.0 * log(base)));
    lo = lo < 0.0 ? 0.0 : lo;
    hi = hi > rot - 1 ? rot - 1 : hi;
  }
  const double width = hi - lo < 0.001 ? 0.001 : hi - lo;
  attn_rope_plan out;
  memset(&out, 0, sizeof(out));
  out.version = 1u;
  out.rot_dim = rot;
  out.layout = c->layout;
  out.mscale = (float)m;
  for (int i = 0; i < rot / 2; ++i) {
    double f = sc == ATTN_ROPE_SCALE_CUSTOM ? c->inv_freq[i] : pow(base, -2.0 * i / rot);
    if (!isfinite(f)) return ATTN_ERR_INVALID_ARG;
    if (sc == ATTN_ROPE_SCALE_LINEAR) {
      f /= factor;
    } else if (sc == ATTN_ROPE_SCALE_YARN) {
      double r = (i - lo) / width;
      r = r < 0.0 ? 0.0 : r > 1.0 ? 1.0 : r;
      f = f * (1.0 - r) + f / factor * r;
    } else if (sc == ATTN_ROPE_SCALE_BANDS) {
      double s = (c->original_len * f / (2.0 * kPi) - low) / (high - low);
      s = s < 0.0 ? 0.0 : s > 1.0 ? 1.0 : s;
      f = f / factor * (1.0 - s) + f * s;
    }
    // turns modulo one, of the magnitude: a double below one times 2^64
    // fits 64 bits
    const double t = fabs(f) / (2.0 * kPi);
    const uint64_t u = (uint64_t)ldexp(t - floor(t), 64);
    out.turns[i] = f < 0.0 ? (uint64_t)0 - u : u;
  }
  *plan = out;
  return ATTN_OK;
}

attn_status attn_rope(const void* x, const int64_t* x_strides, void* out,
                      const int64_t* out_strides, int B, int H, int S, int D,
                      const int32_t* positions, int64_t pos_batch_stride, int32_t offset,
                      const attn_rope_plan* plan, attn_stream_t stream) {
  return run_rope(x, x_strides, out, out_strides, B, H, S, D, positions, pos_batch_stride, offset,
                  plan, 1.0f, stream);
}

attn_status attn_rope_bwd(const void* dout, const int64_t* dout_strides, void* dx,
                          const int64_t* dx_strides, int B, int H, int S, int D,
                          const int32_t* positions, int64_t pos_batch_stride, int32_t offset,
                          const attn_rope_plan* plan, attn_stream_t stream) {
  return run_rope(dout, dout_strides, dx, dx_strides, B, H, S, D, positions, pos_batch_stride,
                  offset, plan, -1.0f, stream);
}

attn_status attn_cache_slots(const int32_t* ctx_lens, const int32_t* new_lens, int B,
                             int page_size, int num_pages, int32_t* block_table,
                             int64_t table_stride, int max_pages, const int32_t* free_pages,
                             int free_cap, const int32_t* n_free, int32_t* seq_lens,
                             int32_t* cu_new, int32_t* token_req, int32_t* positions,
                             int64_t* slots, int32_t* n_free_out, int max_tokens,
                             attn_stream_t stream) {
  if (ctx_lens == nullptr || new_lens == nullptr || block_table == nullptr ||
      seq_lens == nullptr || cu_new == nullptr || token_req == nullptr || positions == nullptr ||
      slots == nullptr)
    return ATTN_ERR_INVALID_ARG;
  if (B <= 0 || page_size <= 0 || num_pages <= 0 || max_pages <= 0 || max_tokens <= 0 ||
      max_tokens > (1 << 30))
    return ATTN_ERR_INVALID_ARG;
  if (B > ATTN_SLOTS_MAX_BATCH) return ATTN_ERR_UNSUPPORTED;
  if ((int64_t)max_pages * page_size > (1 << 30)) return ATTN_ERR_INVALID_ARG;
  if (table_stride < max_pages && B > 1) return ATTN_ERR_INVALID_ARG;
  if (free_pages != nullptr) {
    if (n_free == nullptr || n_free_out == nullptr || free_cap < 0) return ATTN_ERR_INVALID_ARG;
  } else if (n_free != nullptr || n_free_out != nullptr || free_cap != 0) {
    return ATTN_ERR_INVALID_ARG;
  }
  Dims dt;
  dt.add(B, B > 1 ? table_stride : 0);
  const int64_t nt = reach(dt, max_pages);
  if (nt == 0) return ATTN_ERR_INVALID_ARG;
  // inputs, then outputs: an output overlaps neither an input nor another
  // output but for the two pairs that are the same array
  struct Part {
    const void* p;
    uint64_t bytes;
    const void* same;  // the one input an output may be
  };
  const uint64_t T = (uint64_t)max_tokens, nb = (uint64_t)B;
  const Part in[4] = {{ctx_lens, 4 * nb, nullptr},
                      {new_lens, 4 * nb, nullptr},
                      {free_pages, 4 * (uint64_t)free_cap, nullptr},
                      {n_free, 4, nullptr}};
  const Part out[7] = {{block_table, 4 * (uint64_t)nt, nullptr},
                       {seq_lens, 4 * nb, ctx_lens},
                       {cu_new, 4 * (nb + 1), nullptr},
                       {token_req, 4 * T, nullptr},
                       {positions, 4 * T, nullptr},
                       {slots, 8 * T, nullptr},
                       {n_free_out, 4, n_free}};
  for (int i = 0; i < 4; ++i)
    if (!aligned(in[i].p, 4)) return ATTN_ERR_INVALID_ARG;
  for (int i = 0; i < 7; ++i) {
    if (!aligned(out[i].p, out[i].p == slots ? 8 : 4)) return ATTN_ERR_INVALID_ARG;
    for (int j = 0; j < 4; ++j)
      if (overlaps(out[i].p, out[i].bytes, in[j].p, in[j].bytes) &&
          !(out[i].p == in[j].p && out[i].same == in[j].p))
        return ATTN_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlaps(out[i].p, out[i].bytes, out[j].p, out[j].bytes)) return ATTN_ERR_INVALID_ARG;
  }
  SlotArgs a;
  memset(&a, 0, sizeof(a));
  attn_status st = device_status_word(&a.status);
  if (st != ATTN_OK) return st;
  a.ctx_lens = ctx_lens;
  a.new_lens = new_lens;
  a.B = B;
  a.page_size = page_size;
  a.num_pages = num_pages;
  a.table = block_table;
  a.table_stride = table_stride;
  a.max_pages = max_pages;
  a.free_pages = free_pages;
  a.free_cap = free_cap;
  a.n_free = n_free;
  a.seq_lens = seq_lens;
  a.cu_new = cu_new;
  a.token_req = token_req;
  a.positions = positions;
  a.slots = slots;
  a.n_free_out = n_free_out;
  a.max_tokens = max_tokens;
  return launch_slots(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? ATTN_OK
                                                                                 : ATTN_ERR_CUDA;
}

attn_status attn_cache_append(const void* q, const int64_t* q_strides, const void* k,
                              const int64_t* k_strides, const void* v, const int64_t* v_strides,
                              void* q_out, const int64_t* q_out_strides, int T, int H,
                              const int32_t* positions, const int64_t* slots,
                              const attn_rope_plan* plan, const attn_cache_desc* cache,
                              attn_stream_t stream) {
  if (k == nullptr || v == nullptr || k_strides == nullptr || v_strides == nullptr ||
      slots == nullptr)
    return ATTN_ERR_INVALID_ARG;
  if ((q != nullptr) != (q_out != nullptr)) return ATTN_ERR_INVALID_ARG;
  if (q != nullptr && (q_strides == nullptr || q_out_strides == nullptr || H <= 0))
    return ATTN_ERR_INVALID_ARG;
  if (T <= 0 || T > (1 << 24)) return ATTN_ERR_INVALID_ARG;
  uint64_t kb = 0, vb = 0;
  attn_status st = check_cache(cache, &kb, &vb);
  if (st != ATTN_OK) return st;
  const int D = cache->D, H_kv = cache->H_kv;
  if (H_kv > 65535 || (q != nullptr && H > 65535)) return ATTN_ERR_INVALID_ARG;
  if (plan != nullptr) {
    if (!plan_ok(plan) || plan->rot_dim > D) return ATTN_ERR_INVALID_ARG;
    if (positions == nullptr || !aligned(positions, 4)) return ATTN_ERR_INVALID_ARG;
  } else if (positions != nullptr) {
    return ATTN_ERR_INVALID_ARG;
  }
  if (!aligned(slots, 8) || cache->k == cache->v) return ATTN_ERR_INVALID_ARG;
  Dims dq, dk, dv, dqo;
  int width = row_width(D, plan);
  dk.add(T, k_strides[0]);
  dk.add(H_kv, k_strides[1]);
  dv.add(T, v_strides[0]);
  dv.add(H_kv, v_strides[1]);
  const int64_t nk = reach(dk, D), nv = reach(dv, D);
  int64_t nq = 0, nqo = 0;
  if (nk == 0 || nv == 0 || !aligned(k, 2) || !aligned(v, 2)) return ATTN_ERR_INVALID_ARG;
  width = row_width(row_width(width, k, dk), v, dv);
  if (q != nullptr) {
    dq.add(T, q_strides[0]);
    dq.add(H, q_strides[1]);
    dqo.add(T, q_out_strides[0]);
    dqo.add(H, q_out_strides[1]);
    nq = reach(dq, D);
    nqo = reach(dqo, D);
    if (nq == 0 || nqo == 0 || !distinct(dqo, D) || !aligned(q, 2) || !aligned(q_out, 2))
      return ATTN_ERR_INVALID_ARG;
    width = row_width(row_width(width, q, dq), q_out, dqo);
  }
  // the cache overlaps no input; q_out is q as a whole or shares nothing
  // with it, and shares nothing with k and v, though all may be parts of one
  // projection's output
  const void* const cp[2] = {cache->k, cache->v};
  const uint64_t cb[2] = {kb, vb};
  const uint64_t t4 = 4 * (uint64_t)T, h4 = 4 * (uint64_t)H_kv;
  const float* const sc[2] = {cache->k_scale, cache->v_scale};
  for (int i = 0; i < 2; ++i) {
    if (overlaps(cp[0], cb[0], sc[i], h4) || overlaps(cp[1], cb[1], sc[i], h4) ||
        overlaps(q_out, 2 * (uint64_t)nqo, sc[i], h4))
      return ATTN_ERR_INVALID_ARG;
    if (overlaps(cp[i], cb[i], k, 2 * (uint64_t)nk) || overlaps(cp[i], cb[i], v, 2 * (uint64_t)nv) ||
        overlaps(cp[i], cb[i], slots, 2 * t4) || overlaps(cp[i], cb[i], positions, t4) ||
        overlaps(cp[i], cb[i], q, 2 * (uint64_t)nq) ||
        overlaps(cp[i], cb[i], q_out, 2 * (uint64_t)nqo))
      return ATTN_ERR_INVALID_ARG;
  }
  if (q != nullptr && ((!same_place(q, dq, q_out, dqo) &&
                        !rows_apart(q, dq, nq, q_out, dqo, nqo, D)) ||
                       !rows_apart(k, dk, nk, q_out, dqo, nqo, D) ||
                       !rows_apart(v, dv, nv, q_out, dqo, nqo, D)))
    return ATTN_ERR_INVALID_ARG;
  if (q != nullptr && (overlaps(q_out, 2 * (uint64_t)nqo, slots, 2 * t4) ||
                       overlaps(q_out, 2 * (uint64_t)nqo, positions, t4)))
    return ATTN_ERR_INVALID_ARG;

  AppendArgs a;
  memset(&a, 0, sizeof(a));
  st = device_status_word(&a.status);
  if (st != ATTN_OK) return st;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.q_out = static_cast<__nv_bfloat16*>(q_out);
  a.kc = cache->k;
  a.vc = cache->v;
  for (int i = 0; i < 2; ++i) {
    a.qs[i] = q != nullptr ? q_strides[i] : 0;
    a.qos[i] = q != nullptr ? q_out_strides[i] : 0;
    a.ks[i] = k_strides[i];
    a.vs[i] = v_strides[i];
  }
  for (int i = 0; i < 3; ++i) {
    a.kcs[i] = cache->k_strides[i];
    a.vcs[i] = cache->v_strides[i];
  }
  a.T = T;
  a.H = q != nullptr ? H : 0;
  a.H_kv = H_kv;
  a.D = D;
  a.num_pages = cache->num_pages;
  a.page_size = cache->page_size;
  a.positions = positions;
  a.slots = slots;
  a.k_scale = cache->k_scale;
  a.v_scale = cache->v_scale;
  a.rotate = plan != nullptr ? 1 : 0;
  if (plan != nullptr) a.plan = *plan;
  return launch_append(a, width, cache->dtype == ATTN_CACHE_E4M3,
                       reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? ATTN_OK
             : ATTN_ERR_CUDA;
}

size_t attn_decode_workspace_bytes(int H, int H_kv, int D) {
  if (H <= 0 || H_kv <= 0 || H % H_kv != 0 || H > 65535 || (D != 64 && D != 128)) return 0;
  return decode_workspace_bytes(H, H_kv, D);
}

attn_status attn_decode(const void* q, const int64_t* q_strides, const attn_cache_desc* cache,
                        const int32_t* block_table, int64_t table_stride, int max_pages,
                        const int32_t* seq_lens, void* out, float* lse, int B, int H, float scale,
                        const attn_mod_desc* mod, void* workspace, size_t workspace_bytes,
                        attn_stream_t stream) {
  if (q == nullptr || q_strides == nullptr || block_table == nullptr || seq_lens == nullptr ||
      out == nullptr || workspace == nullptr)
    return ATTN_ERR_INVALID_ARG;
  uint64_t kb = 0, vb = 0;
  attn_status st = check_cache(cache, &kb, &vb);
  if (st != ATTN_OK) return st;
  const int D = cache->D, H_kv = cache->H_kv;
  if (B <= 0 || B > 65536 || H <= 0 || H > 65535 || H % H_kv != 0 || max_pages <= 0)
    return ATTN_ERR_INVALID_ARG;
  if ((int64_t)max_pages * cache->page_size > (1 << 30)) return ATTN_ERR_INVALID_ARG;
  if (!(isfinite(scale) && scale > 0.f)) return ATTN_ERR_INVALID_ARG;
  attn_mod_desc m;
  memset(&m, 0, sizeof(m));
  if (mod != nullptr) {
    // the same descriptor rules as attn_fwd's, then what this call serves
    st = load_checked_mod(mod, &m);
    if (st != ATTN_OK) return st;
    if ((m.mask_flags & ~(uint32_t)(ATTN_MASK_CAUSAL | ATTN_MASK_WINDOW)) != 0u ||
        m.q_offset != 0 || m.block_mask != nullptr)
      return ATTN_ERR_UNSUPPORTED;
  }
  if (table_stride < 0 || !aligned(block_table, 4) || !aligned(seq_lens, 4))
    return ATTN_ERR_INVALID_ARG;
  Dims dt, dq;
  dt.add(B, table_stride);
  dq.add(B, q_strides[0]);
  dq.add(H, q_strides[1]);
  const int64_t nt = reach(dt, max_pages), nq = reach(dq, D);
  if (nt == 0 || nq == 0) return ATTN_ERR_INVALID_ARG;
  if (!aligned(q, 4) || (B > 1 && q_strides[0] % 2 != 0) || (H > 1 && q_strides[1] % 2 != 0))
    return ATTN_ERR_INVALID_ARG;
  if (!aligned(out, 16) || !aligned(lse, 4) || !aligned(workspace, 16))
    return ATTN_ERR_INVALID_ARG;
  if (workspace_bytes < decode_workspace_bytes(H, H_kv, D)) return ATTN_ERR_INVALID_ARG;
  // 64-key units of all requests and heads, times the grid, in 64 bits
  if ((double)B * H * ((double)max_pages * cache->page_size / 64 + 1) > 9.0e15)
    return ATTN_ERR_UNSUPPORTED;
  const uint64_t ob = 2 * (uint64_t)B * H * D, lb = 4 * (uint64_t)B * H;
  struct Part {
    const void* p;
    uint64_t bytes;
  };
  const Part outs[3] = {{out, ob}, {lse, lb}, {workspace, (uint64_t)workspace_bytes}};
  const bool slopes = (m.score_flags & ATTN_SCORE_ALIBI) != 0u;
  const bool bias = (m.score_flags & ATTN_SCORE_RELBIAS) != 0u;
  const Part ins[9] = {{q, 2 * (uint64_t)nq},
                       {cache->k, kb},
                       {cache->v, vb},
                       {block_table, 4 * (uint64_t)nt},
                       {seq_lens, 4 * (uint64_t)B},
                       {cache->k_scale, 4 * (uint64_t)H_kv},
                       {cache->v_scale, 4 * (uint64_t)H_kv},
                       {slopes ? m.alibi_slopes : nullptr, 4 * (uint64_t)H},
                       {bias ? m.rel_bias : nullptr, 4 * (uint64_t)H * (2 * (uint64_t)m.rel_max + 1)}};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < 9; ++j)
      if (overlaps(outs[i].p, outs[i].bytes, ins[j].p, ins[j].bytes)) return ATTN_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlaps(outs[i].p, outs[i].bytes, outs[j].p, outs[j].bytes)) return ATTN_ERR_INVALID_ARG;
  }

  DecodeArgs a;
  memset(&a, 0, sizeof(a));
  st = device_status_word(&a.status);
  if (st != ATTN_OK) return st;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.qs[0] = q_strides[0];
  a.qs[1] = q_strides[1];
  a.kc = cache->k;
  a.vc = cache->v;
  for (int i = 0; i < 3; ++i) {
    a.kcs[i] = cache->k_strides[i];
    a.vcs[i] = cache->v_strides[i];
  }
  a.num_pages = cache->num_pages;
  a.page_size = cache->page_size;
  a.table = block_table;
  a.table_stride = table_stride;
  a.max_pages = max_pages;
  a.seq_lens = seq_lens;
  a.k_scale = cache->k_scale;
  a.v_scale = cache->v_scale;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.B = B;
  a.H = H;
  a.H_kv = H_kv;
  a.D = D;
  a.scale = scale;
  a.window = (m.mask_flags & ATTN_MASK_WINDOW) ? m.window : 0;
  a.score_flags = m.score_flags;
  a.softcap = m.softcap;
  a.alibi_slopes = (m.score_flags & ATTN_SCORE_ALIBI) ? m.alibi_slopes : nullptr;
  a.rel_bias = (m.score_flags & ATTN_SCORE_RELBIAS) ? m.rel_bias : nullptr;
  a.rel_max = (m.score_flags & ATTN_SCORE_RELBIAS) ? m.rel_max : 0;
  a.workspace = workspace;
  wait_options(&a.wait_budget_ms, &a.debug_stall);
  return launch_decode(a, cache->dtype == ATTN_CACHE_E4M3,
                       reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? ATTN_OK
             : ATTN_ERR_CUDA;
}

}  // extern "C"
