// rope_cache_sm103.cu -- rotary positions, the slot map of a paged key/value
// cache, and the writes into it.
//
// Rotation of pair i of a row at position p:
//   a = p f_i,  (u, v) -> m (u cos a - v sin a, v cos a + u sin a),
// and its gradient the same with -a.  f_i comes as turns per position in
// units of 2^-64 (modulo one turn), so p * f_i is an integer product whose
// low 64 bits are the angle's fraction of a turn, with no rounding at any
// position (what is left is p times the plan's own error in f_i, 2^-53 of it);
// read as a signed number it lies in [-1/2, 1/2) turns.  A product in fp32
// would be off by 2^-24 p f_i radians: 0.06 at position 2^20 of the fastest
// pair.  The nearest quarter turn is taken off as an integer too, and sine and
// cosine of the rest (at most pi / 4) come from their series, to 2^-23.4.  Of
// the product's 64 bits the upper 32 are made: with all of them, and their two
// conversions, 4 heads x 100000 rows took 39.1 us, now 33.4.
//
// What bounds it: each element is read and written once (4 bytes per bf16
// element).  A block takes a few tokens and a run of heads; its threads make
// the tokens' angles together, one sincos per pair and token into shared
// memory, while their first loads are on the way, and then go over the heads,
// two multiply-adds per element.  Measured on GB300, of the 6.78 TB/s of a
// copy: 41.0 us for B 2, H 32, S 8192, D 128 (97%); the cache write of 16384
// tokens of 32 + 8 + 8 heads into e4m3 62.7 us (87%); 111 rows of 8 heads 1.9
// us, 64 tokens into bf16 2.3 us, the slot map of 64 requests 2.9 us and of 48
// prompts with 49 thousand tokens 4.2 us, which are latencies.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <stdint.h>

#include <type_traits>

#include "generation_internal.h"
#include "sm103_ptx.cuh"

namespace attn {
namespace {

__device__ __forceinline__ void record_error(DeviceStatus* st, int site, int detail) {
  if (atomicCAS(&st->code, 0, ATTN_ERR_DEVICE_CHECK) == 0) {
    st->where = site;
    st->block = blockIdx.x;
    st->detail = detail;
  }
}

// cos and sin (times m) of pair i at position p; sign = -1 turns backwards.
__device__ __forceinline__ void pair_angle(int32_t p, uint64_t turns, float m, float sign,
                                           float& c, float& s) {
  // the high word of the product modulo 2^64; what it leaves out is below
  // 2^-32 turns, 1.5e-9 radians
  const uint32_t lo = (uint32_t)turns;
  const uint32_t a = (uint32_t)p * (uint32_t)(turns >> 32) + __umulhi((uint32_t)p, lo) -
                     (p < 0 ? lo : 0u);
  const uint32_t q = (a + 0x20000000u) >> 30;  // quarter turns, nearest
  const float x = (float)(int32_t)(a - (q << 30)) * 1.4629180792671596e-09f;  // 2 pi 2^-32
  // sin x to x^9, cos x to x^8: the next terms are 2^-29 and 2^-25 at pi / 4
  const float z = x * x;
  float sn = fmaf(z, 1.0f / 362880.0f, -1.0f / 5040.0f);
  sn = fmaf(z, sn, 1.0f / 120.0f);
  sn = fmaf(z, sn, -1.0f / 6.0f);
  sn = fmaf(x * z, sn, x);
  float cs = fmaf(z, 1.0f / 40320.0f, -1.0f / 720.0f);
  cs = fmaf(z, cs, 1.0f / 24.0f);
  cs = fmaf(z, cs, -0.5f);
  cs = fmaf(z, cs, 1.0f);
  // a quarter turn makes (cos, sin) of it (-sin, cos)
  const float u = (q & 1u) ? sn : cs, v = (q & 1u) ? cs : sn;
  c = ((q + 1u) & 2u) ? -u * m : u * m;
  s = (q & 2u) ? -v * (m * sign) : v * (m * sign);
}

__device__ __forceinline__ float2 bf2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// What pairs, and whether all of an item's pairs turn or none; neighbours that
// stop turning inside an item have a variant of their own, whose test of each
// pair takes 4% (16 heads of which half turns, 43.1 us and 44.8).
enum Kind { kNeighbours, kHalves, kNeighboursPart };

// A thread's share of a row: W pairs of elements, moved as two accesses of W
// elements at a and b (W = 8: 16 bytes each, the widest that alignment and
// sizes allow: 3 x 31664 rows of 96 elements that turn 14, neighbours, 10.0 us
// and 41.5 in 2-byte accesses; 16 x 8192 rows that turn 24, halves, 9.6 in
// 8-byte ones and 29.4).  Where halves pair, u and v of
// a turned item are the two accesses; in every other item neighbours
// (2 i, 2 i + 1) of the 2 W elements form a pair.
template <int W>
struct Item {
  int a, b;    // element offsets in the row
  bool rotated;
  int turned;  // pairs that turn if any do, the first ones (W and more: all)
  int pair0;   // first pair's index in the plan
};

template <int W, int KIND>
__device__ __forceinline__ Item<W> item_at(int j, int rot) {
  Item<W> it;
  it.pair0 = j * W;
  it.rotated = 2 * W * j < rot;
  it.turned = KIND == kNeighboursPart ? rot / 2 - it.pair0 : W;
  const bool split = it.rotated && KIND == kHalves;
  it.a = split ? W * j : 2 * W * j;
  it.b = split ? W * j + rot / 2 : 2 * W * j + W;
  return it;
}

// The two accesses of an item.
template <int W>
struct Vals {
  using T = std::conditional_t<W == 8, uint4,
            std::conditional_t<W == 4, uint2, std::conditional_t<W == 2, uint32_t, uint16_t>>>;
  T a, b;
};

template <int W>
__device__ __forceinline__ void load_item(const __nv_bfloat16* row, const Item<W>& it,
                                          Vals<W>& x) {
  x.a = *reinterpret_cast<const typename Vals<W>::T*>(row + it.a);
  x.b = *reinterpret_cast<const typename Vals<W>::T*>(row + it.b);
}

__device__ __forceinline__ void unpack(uint4 x, float* y) {
  const float2 a = bf2(x.x), b = bf2(x.y), c = bf2(x.z), d = bf2(x.w);
  y[0] = a.x, y[1] = a.y, y[2] = b.x, y[3] = b.y;
  y[4] = c.x, y[5] = c.y, y[6] = d.x, y[7] = d.y;
}
__device__ __forceinline__ void unpack(uint2 x, float* y) {
  const float2 a = bf2(x.x), b = bf2(x.y);
  y[0] = a.x, y[1] = a.y, y[2] = b.x, y[3] = b.y;
}
__device__ __forceinline__ void unpack(uint32_t x, float* y) {
  const float2 a = bf2(x);
  y[0] = a.x, y[1] = a.y;
}
__device__ __forceinline__ void unpack(uint16_t x, float* y) {
  y[0] = __uint_as_float((uint32_t)x << 16);
}

// (u, v) turned by the angle of cos and sin a.
__device__ __forceinline__ void turn(float& u, float& v, float c, float s) {
  const float x = u, y = v;
  u = fmaf(x, c, -(y * s));
  v = fmaf(y, c, x * s);
}

// An item in fp32, its pairs turned if `rotated`: y[i] for the elements at
// a, y[W + i] at b.  angles: the item's first piece; step: floats between its
// pieces.
template <int W, int KIND>
__device__ __forceinline__ void rotate_item(const Item<W>& it, bool rotated, const Vals<W>& x,
                                            const float* angles, int step, float* y) {
  unpack(x.a, y);
  unpack(x.b, y + W);
  if (!rotated) return;
  if constexpr (W == 1) {
    turn(y[0], y[1], angles[0], angles[1]);
  } else {
#pragma unroll
    for (int q = 0; q < W / 2; ++q) {
      const float4 cs = *reinterpret_cast<const float4*>(angles + q * step);
      if (KIND == kHalves) {
        turn(y[2 * q], y[W + 2 * q], cs.x, cs.y);
        turn(y[2 * q + 1], y[W + 2 * q + 1], cs.z, cs.w);
      } else {
        if (KIND != kNeighboursPart || 2 * q < it.turned) turn(y[4 * q], y[4 * q + 1], cs.x, cs.y);
        if (KIND != kNeighboursPart || 2 * q + 1 < it.turned)
          turn(y[4 * q + 2], y[4 * q + 3], cs.z, cs.w);
      }
    }
  }
}

template <int W>
__device__ __forceinline__ typename Vals<W>::T pack(const float* y) {
  typename Vals<W>::T r;
  if constexpr (W == 8)
    r = make_uint4(ptx::pack_bf16x2(y[0], y[1]), ptx::pack_bf16x2(y[2], y[3]),
                   ptx::pack_bf16x2(y[4], y[5]), ptx::pack_bf16x2(y[6], y[7]));
  else if constexpr (W == 4)
    r = make_uint2(ptx::pack_bf16x2(y[0], y[1]), ptx::pack_bf16x2(y[2], y[3]));
  else if constexpr (W == 2)
    r = ptx::pack_bf16x2(y[0], y[1]);
  else
    r = __bfloat16_as_ushort(__float2bfloat16_rn(y[0]));
  return r;
}

template <int W>
__device__ __forceinline__ void store_item(__nv_bfloat16* row, const Item<W>& it,
                                           const float* y) {
  *reinterpret_cast<typename Vals<W>::T*>(row + it.a) = pack<W>(y);
  *reinterpret_cast<typename Vals<W>::T*>(row + it.b) = pack<W>(y + W);
}

__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
  uint16_t r;
  // rounds to nearest even; beyond +-448 gives +-448, NaN gives NaN
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// y / scale for storing: the product with inv = 1 / scale and one correction by
// the remainder (Markstein's division step), so that values next to a border
// of two e4m3 numbers fall on the side that the quotient does.  Numbers far
// beyond the range keep the product (an infinity has no remainder).
__device__ __forceinline__ float scaled(float y, float scale, float inv) {
  const float q = y * inv;
  const float r = fmaf(fmaf(-q, scale, y), inv, q);
  return fabsf(q) < 1024.0f ? r : q;
}

// W elements in e4m3 to p.
template <int W>
__device__ __forceinline__ void store_e4m3(uint8_t* p, const float* y) {
  if constexpr (W == 1) {
    *p = (uint8_t)pack_e4m3x2(y[0], 0.f);
  } else {
    const uint32_t lo = pack_e4m3x2(y[0], y[1]);
    if constexpr (W == 2) {
      *reinterpret_cast<uint16_t*>(p) = (uint16_t)lo;
    } else {
      const uint32_t w = lo | pack_e4m3x2(y[2], y[3]) << 16;
      if constexpr (W == 4)
        *reinterpret_cast<uint32_t*>(p) = w;
      else
        *reinterpret_cast<uint2*>(p) =
            make_uint2(w, pack_e4m3x2(y[4], y[5]) | pack_e4m3x2(y[6], y[7]) << 16);
    }
  }
}

template <int W>
__device__ __forceinline__ void store_item_e4m3(uint8_t* row, const Item<W>& it, float* y,
                                                float scale) {
  // 0 stays 0 for a scale of 0 or one whose reciprocal is beyond fp32, and every
  // number becomes 0 for an infinite one, as the quotient does
  const float inv = fminf(__fdiv_rn(1.0f, scale), FLT_MAX);
  if (inv == 0.0f) scale = 0.0f;  // the remainder times infinity would be NaN
#pragma unroll
  for (int i = 0; i < 2 * W; ++i) y[i] = scaled(y[i], scale, inv);
  store_e4m3<W>(row + it.a, y);
  store_e4m3<W>(row + it.b, y + W);
}

constexpr int kThreads = 256;
constexpr int kUnroll = 2;      // heads of a thread whose loads are in flight together
constexpr int kAngles = 2048;   // of a block: tokens x pairs

// How a block's threads share its tokens and heads: threadIdx.x the item of a
// row, .y the token, .z the head (so a warp works on few heads).  More heads
// side by side are fewer tokens and so fewer angles: with 128-element heads
// and 8 of them a thread makes one angle, where 32 tokens side by side would
// have each make eight.  Measured: 16 heads of which half turns (B 1,
// S 32768) 42.7 us with 4 side by side, 44.6 with 8, 43.3 with 2; the cache
// write of 16384 tokens 61 us with 8 and 72 with 4.  A thread of rope_kernel
// wants kUnroll heads of its own before they are put side by side (4 heads,
// S 100000: 39.4 us with 2 side by side, 51.7 with 4); and in 2-byte accesses a
// row takes so many threads that 4 heads leave few tokens (16 x 8192 rows that
// turn 66 of 128 in halves, 27.5 us with 2 and 38.2 with 4).
dim3 block_shape(int D, int width, int heads, int most) {
  const int items = D / (2 * width) < kThreads ? D / (2 * width) : kThreads;
  const int rows = kThreads / items;
  int side = 1;
  while (side * 2 <= heads && side < most && side * 2 <= rows) side *= 2;
  return dim3((unsigned)items, (unsigned)(rows / side < 64 ? rows / side : 64), (unsigned)side);
}

// cos and sin of the block's tokens, in the order that items read them: an
// item's pairs as 16-byte pieces of two, each next to the same piece of the
// neighbouring items, so that a warp's reads fall into different banks.
template <int W, int KIND>
__device__ __forceinline__ int angle_step(int tokens, int pairs) {  // between an item's pieces
  return tokens * ((KIND == kNeighboursPart ? pairs + W - 1 : pairs) / W) * 4;
}
template <int W, int KIND>
__device__ __forceinline__ int angle_at(int tokens, int pairs, int t, int i) {
  if constexpr (W == 1)
    return 2 * (t * pairs + i);
  else
    return ((i >> 1) & (W / 2 - 1)) * angle_step<W, KIND>(tokens, pairs) +
           angle_step<W, KIND>(t, pairs) + (i / W) * 4 + 2 * (i & 1);
}
// The threads of one token make its angles.
template <int W, int KIND>
__device__ __forceinline__ void make_angles(float* s_angle, const attn_rope_plan& plan, float sign,
                                            int32_t pos) {
  const int pairs = plan.rot_dim / 2;
  for (int i = threadIdx.z * blockDim.x + threadIdx.x; i < pairs; i += blockDim.x * blockDim.z) {
    float c, s;
    pair_angle(pos, plan.turns[i], plan.mscale, sign, c, s);
    *reinterpret_cast<float2*>(s_angle + angle_at<W, KIND>(blockDim.y, pairs, threadIdx.y, i)) =
        make_float2(c, s);
  }
}

// --------------------------------------------------------------- rope ----

template <int W, int KIND>
__global__ void __launch_bounds__(kThreads, W == 8 ? 4 : W == 4 ? 5 : 6)
    rope_kernel(const __grid_constant__ RopeArgs p) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  __shared__ __align__(16) float s_angle[2 * kAngles];
  const int row_items = p.D / (2 * W);  // more than the threads of a row for wide scalar rows
  const int t = threadIdx.y, side = blockDim.z;
  const int64_t row = (int64_t)blockIdx.x * blockDim.y + t;
  const int h0 = blockIdx.y * p.heads_per_block + threadIdx.z;
  const int h1 = min(p.H, (int)(blockIdx.y + 1) * p.heads_per_block);
  const bool work = row < (int64_t)p.B * p.S;
  const int b = work ? (int)((uint32_t)row / (uint32_t)p.S) : 0;
  const int s = work ? (int)((uint32_t)row - (uint32_t)b * (uint32_t)p.S) : 0;
  const __nv_bfloat16* xin = p.x + b * p.xs[0] + s * p.xs[2];
  __nv_bfloat16* out = p.out + b * p.os[0] + s * p.os[2];
  int j = threadIdx.x;
  Item<W> it = item_at<W, KIND>(j, p.plan.rot_dim);
  Vals<W> v[kUnroll];
  auto load = [&](int h) {
#pragma unroll
    for (int k = 0; k < kUnroll; ++k)
      if (h + k * side < h1) load_item<W>(xin + (h + k * side) * p.xs[1], it, v[k]);
  };
  if (work) {
    load(h0);
    make_angles<W, KIND>(s_angle, p.plan, p.sign,
                     (int32_t)((uint32_t)(p.positions ? p.positions[b * p.pos_stride + s] : s) +
                               (uint32_t)p.offset));
  }
  __syncthreads();
  if (!work) return;
  const int pairs = p.plan.rot_dim / 2, step = angle_step<W, KIND>(blockDim.y, pairs);
  for (;;) {
    const float* angles = s_angle + angle_at<W, KIND>(blockDim.y, pairs, t, it.pair0);
    for (int h = h0; h < h1; h += kUnroll * side) {
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int hh = h + k * side;
        if (hh >= h1) break;
        float y[2 * W];
        rotate_item<W, KIND>(it, it.rotated, v[k], angles, step, y);
        store_item<W>(out + hh * p.os[1], it, y);
      }
      if (h + kUnroll * side < h1) load(h + kUnroll * side);
    }
    j += blockDim.x;
    if (W > 1 || j >= row_items) break;
    it = item_at<W, KIND>(j, p.plan.rot_dim);
    load(h0);
  }
}

// ------------------------------------------------------------- append ----

// A block of few tokens takes all heads, the key and value heads first; where
// that makes too few blocks, blocks of the grid's second dimension take a run
// of query heads or a run of key and value heads each.  A row of the cache is
// at most 128 elements, so its items are always fewer than the threads.
template <int W, int KIND, bool E4M3>
__global__ void __launch_bounds__(kThreads, W == 8 ? 3 : 4)
    append_kernel(const __grid_constant__ AppendArgs p) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  __shared__ __align__(16) float s_angle[2 * kAngles];
  const int t = threadIdx.y, side = blockDim.z;
  const int64_t tok = (int64_t)blockIdx.x * blockDim.y + t;
  const bool work = tok < p.T;
  // this block's query heads [q0, q1) and kv heads [k0, k1), a thread's from z on
  const int per = p.heads_per_block, y = blockIdx.y;
  int q0 = 0, q1 = p.H, k0 = 0, k1 = p.H_kv;
  if (gridDim.y > 1) {
    const int kv_runs = (p.H_kv + per - 1) / per;
    if (y < kv_runs) {
      k0 = y * per, k1 = min(p.H_kv, k0 + per);
      q1 = 0;
    } else {
      q0 = (y - kv_runs) * per, q1 = min(p.H, q0 + per);
      k1 = 0;
    }
  }
  q0 += threadIdx.z;
  k0 += threadIdx.z;
  const int rot = p.rotate ? p.plan.rot_dim : 0;
  const Item<W> it = item_at<W, KIND>(threadIdx.x, rot);
  const __nv_bfloat16* q = p.q + tok * p.qs[0];
  const __nv_bfloat16* k = p.k + tok * p.ks[0];
  const __nv_bfloat16* v = p.v + tok * p.vs[0];
  Vals<W> xk, xv, xq[kUnroll];
  auto load_q = [&](int h) {
#pragma unroll
    for (int i = 0; i < kUnroll; ++i)
      if (h + i * side < q1) load_item<W>(q + (h + i * side) * p.qs[1], it, xq[i]);
  };
  int64_t slot = -1;
  if (work) {
    if (k0 < k1) {
      slot = p.slots[tok];
      load_item<W>(k + k0 * p.ks[1], it, xk);
      load_item<W>(v + k0 * p.vs[1], it, xv);
    }
    load_q(q0);
    if (rot > 0) make_angles<W, KIND>(s_angle, p.plan, 1.0f, p.positions[tok]);
  }
  __syncthreads();
  if (!work) return;
  const float* angles = s_angle + angle_at<W, KIND>(blockDim.y, rot / 2, t, it.pair0);
  const int step = angle_step<W, KIND>(blockDim.y, rot / 2);

  if (slot >= (int64_t)p.num_pages * p.page_size) {
    record_error(p.status, kSiteSlot, (int)tok);
    slot = -1;
  }
  if (slot >= 0) {
    // 32 bits hold the slots of all but the largest caches
    const int64_t page = (slot >> 32) == 0 ? (uint32_t)slot / (uint32_t)p.page_size
                                           : slot / p.page_size;
    const int64_t in_page = slot - page * p.page_size;
    const int64_t kat = page * p.kcs[0] + in_page * p.kcs[2];
    const int64_t vat = page * p.vcs[0] + in_page * p.vcs[2];
    for (int h = k0; h < k1; h += side) {
      float y[2 * W], z[2 * W];
      rotate_item<W, KIND>(it, it.rotated, xk, angles, step, y);
      rotate_item<W, KIND>(it, false, xv, angles, step, z);
      if (h + side < k1) {
        load_item<W>(k + (h + side) * p.ks[1], it, xk);
        load_item<W>(v + (h + side) * p.vs[1], it, xv);
      }
      if (E4M3) {
        store_item_e4m3<W>(static_cast<uint8_t*>(p.kc) + kat + h * p.kcs[1], it, y,
                             p.k_scale != nullptr ? p.k_scale[h] : 1.0f);
        store_item_e4m3<W>(static_cast<uint8_t*>(p.vc) + vat + h * p.vcs[1], it, z,
                             p.v_scale != nullptr ? p.v_scale[h] : 1.0f);
      } else {
        store_item<W>(static_cast<__nv_bfloat16*>(p.kc) + kat + h * p.kcs[1], it, y);
        store_item<W>(static_cast<__nv_bfloat16*>(p.vc) + vat + h * p.vcs[1], it, z);
      }
    }
  }
  __nv_bfloat16* out = p.q_out + tok * p.qos[0];
  for (int h = q0; h < q1; h += kUnroll * side) {
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      if (h + i * side >= q1) break;
      float y[2 * W];
      rotate_item<W, KIND>(it, it.rotated, xq[i], angles, step, y);
      store_item<W>(out + (h + i * side) * p.qos[1], it, y);
    }
    if (h + kUnroll * side < q1) load_q(h + kUnroll * side);
  }
}

// -------------------------------------------------------------- slots ----

constexpr int kSlotThreads = 1024;  // at most

// Inclusive sum over the block of (x, y); every thread gets its own prefix,
// warp_x[31] and warp_y[31] the totals.
__device__ __forceinline__ void block_scan2(int64_t& x, int64_t& y, int64_t* warp_x,
                                            int64_t* warp_y) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t ox = __shfl_up_sync(0xffffffffu, x, d);
    const int64_t oy = __shfl_up_sync(0xffffffffu, y, d);
    if (lane >= d) x += ox, y += oy;
  }
  if (lane == 31) warp_x[w] = x, warp_y[w] = y;
  __syncthreads();
  if (w == 0) {
    const bool have = lane < (int)(blockDim.x >> 5);
    int64_t a = have ? warp_x[lane] : 0, b = have ? warp_y[lane] : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t oa = __shfl_up_sync(0xffffffffu, a, d);
      const int64_t ob = __shfl_up_sync(0xffffffffu, b, d);
      if (lane >= d) a += oa, b += ob;
    }
    warp_x[lane] = a, warp_y[lane] = b;
  }
  __syncthreads();
  if (w > 0) x += warp_x[w - 1], y += warp_y[w - 1];
}

// Every CTA scans all requests into its own shared memory (tokens and pages
// before each), and then the CTAs share the tokens: each thread finds its
// token's request by bisection.  A new page's table entry is written by the
// page's first token, which is always one of the new ones; entries that are
// read are those of older pages.  So the only outputs that a CTA may still
// have to read when another writes them are the two that may be their inputs
// (in_place): then the grid is one cluster, which meets once in between.
__global__ void __launch_bounds__(kSlotThreads) slots_kernel(const __grid_constant__ SlotArgs p) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  extern __shared__ int32_t sm[];
  int32_t* s_ctx = sm;               // [B]
  int32_t* s_cu = s_ctx + p.B;       // [B] new tokens before the request
  int32_t* s_pg = s_cu + p.B;        // [B] new pages before the request
  __shared__ int64_t s_wx[32], s_wy[32];
  __shared__ int s_bad;
  const int tid = threadIdx.x;
  const int rank = (int)blockIdx.x, stride = (int)(gridDim.x * blockDim.x);
  const int P = p.page_size;
  if (tid == 0) s_bad = 0;
  __syncthreads();
  // a thread's run of requests, so that one scan over the threads is enough
  const int per = (p.B + (int)blockDim.x - 1) / (int)blockDim.x;
  const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
  const int64_t room = (int64_t)p.max_pages * P;
  int64_t toks = 0, pgs = 0;
  int bad = 0;
  for (int b = b0; b < b1; ++b) {
    const int64_t c = p.ctx_lens[b], nw = p.new_lens[b];
    s_ctx[b] = (int32_t)c;
    if (c < 0 || nw < 0 || c + nw > room) {
      bad = 1;
      s_cu[b] = s_pg[b] = 0;
      continue;
    }
    const int64_t pages = p.free_pages != nullptr ? (c + nw + P - 1) / P - (c + P - 1) / P : 0;
    s_cu[b] = (int32_t)nw;
    s_pg[b] = (int32_t)pages;
    toks += nw;
    pgs += pages;
  }
  int64_t xt = toks, xp = pgs;
  block_scan2(xt, xp, s_wx, s_wy);
  const int64_t all_toks = s_wx[31], all_pgs = s_wy[31];
  int64_t n_free = 0;
  if (p.free_pages != nullptr) {
    n_free = *p.n_free;
    if (n_free < 0 || n_free > p.free_cap || all_pgs > n_free) bad = 1;
  }
  if (all_toks > p.max_tokens) bad = 1;
  if (bad) s_bad = 1;
  __syncthreads();
  bad = s_bad;
  if (!bad) {  // the sums fit 32 bits
    int32_t ct = (int32_t)(xt - toks), cp = (int32_t)(xp - pgs);
    for (int b = b0; b < b1; ++b) {
      const int32_t nw = s_cu[b], pg = s_pg[b];
      s_cu[b] = ct;
      s_pg[b] = cp;
      ct += nw;
      cp += pg;
    }
  }
  __syncthreads();
  if (p.in_place) ptx::cluster_sync();
  if (bad && rank == 0 && tid == 0) record_error(p.status, kSiteSlotMap, (int)all_pgs);
  const int total = bad ? 0 : (int)all_toks;
  for (int b = rank * (int)blockDim.x + tid; b < p.B; b += stride) {
    const int32_t next = bad ? 0 : (b + 1 < p.B ? s_cu[b + 1] : total);
    const int32_t cu = bad ? 0 : s_cu[b];
    p.seq_lens[b] = s_ctx[b] + (next - cu);
    p.cu_new[b] = cu;
    if (b == p.B - 1) {
      p.cu_new[p.B] = total;
      if (p.n_free_out != nullptr) *p.n_free_out = (int32_t)(bad ? n_free : n_free - all_pgs);
    }
  }
  for (int64_t j = rank * (int)blockDim.x + tid; j < p.max_tokens; j += stride) {
    int32_t req = -1, pos = 0;
    int64_t slot = -1;
    if (j < total) {
      // the last request that starts at or before token j: requests that
      // add nothing start where the next one does, so this one adds token j
      int lo = 0, hi = p.B;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_cu[mid] <= (int32_t)j) lo = mid; else hi = mid;
      }
      req = lo;
      const int32_t ctx = s_ctx[lo];
      pos = ctx + (int32_t)j - s_cu[lo];
      const int col = pos / P, row = pos - col * P;
      int32_t* entry = p.table + lo * p.table_stride + col;
      int32_t page;
      const int had = (int)(((int64_t)ctx + P - 1) / P);
      if (p.free_pages != nullptr && col >= had) {
        page = p.free_pages[n_free - 1 - (s_pg[lo] + (col - had))];
        if (row == 0) *entry = page;
      } else {
        page = *entry;
      }
      if (page >= 0 && page < p.num_pages) {
        slot = (int64_t)page * P + row;
      } else {
        record_error(p.status, kSitePage, page);
      }
    }
    p.token_req[j] = req;
    p.positions[j] = pos;
    p.slots[j] = slot;
  }
}

// Grid of a kernel over rows and heads; *per: the heads of its blocks.  All of
// them, so that their tokens' angles are made once, or fewer (a multiple of
// those side by side) where that leaves too few blocks to fill the GPU: four
// waves of four a SM.
dim3 grid_over(int64_t rows, int heads, dim3 block, int sms, int* per) {
  const int side = (int)block.z;
  const int64_t bx = (rows + block.y - 1) / block.y, want = (int64_t)sms * 16;
  const int rounds = (heads + side - 1) / side;  // a thread's heads
  int64_t chunks = (want + bx - 1) / bx;
  if (chunks > rounds) chunks = rounds;
  int r = (int)((rounds + chunks - 1) / chunks);
  while ((heads + side * r - 1) / (side * r) > 65535) ++r;  // a grid's second dimension
  *per = side * r;
  return dim3((unsigned)bx, (unsigned)((heads + *per - 1) / *per));
}

cudaError_t sm_count(int* sms) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  return cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
}

}  // namespace

// f(width, kind) as types, for the width chosen and the plan's layout.
template <int W, class F>
auto with_kind(const attn_rope_plan& plan, F f) {
  using Width = std::integral_constant<int, W>;
  if (plan.layout == ATTN_ROPE_HALF) return f(Width(), std::integral_constant<int, kHalves>());
  if constexpr (W > 1)
    if (plan.rot_dim % (2 * W) != 0)
      return f(Width(), std::integral_constant<int, kNeighboursPart>());
  return f(Width(), std::integral_constant<int, kNeighbours>());
}
template <class F>
auto with_item(int width, const attn_rope_plan& plan, F f) {
  return width == 8   ? with_kind<8>(plan, f)
         : width == 4 ? with_kind<4>(plan, f)
         : width == 2 ? with_kind<2>(plan, f)
                      : with_kind<1>(plan, f);
}

cudaError_t launch_rope(const RopeArgs& a, int width, cudaStream_t stream) {
  int sms = 0;
  cudaError_t err = sm_count(&sms);
  if (err != cudaSuccess) return err;
  RopeArgs p = a;
  const dim3 block = block_shape(a.D, width, a.H / kUnroll, width > 1 ? 4 : 2);
  const dim3 grid = grid_over((int64_t)a.B * a.S, a.H, block, sms, &p.heads_per_block);
  auto kern = with_item(width, a.plan, [](auto w, auto kind) {
    return rope_kernel<decltype(w)::value, decltype(kind)::value>;
  });
  return launch_overlapped(kern, grid, block, 0, 0, stream, p);
}

cudaError_t launch_append(const AppendArgs& a, int width, bool e4m3, cudaStream_t stream) {
  int sms = 0;
  cudaError_t err = sm_count(&sms);
  if (err != cudaSuccess) return err;
  AppendArgs p = a;
  const dim3 block = block_shape(a.D, width, a.H > a.H_kv ? a.H : a.H_kv, 8);
  // all heads to a block, or runs of query heads and of kv heads apart
  dim3 grid = grid_over(a.T, a.H + a.H_kv, block, sms, &p.heads_per_block);
  if (grid.y > 1) {
    const int per = p.heads_per_block;
    grid.y = (unsigned)((a.H + per - 1) / per + (a.H_kv + per - 1) / per);
  }
  auto kern = with_item(width, a.plan, [&](auto w, auto kind) {
    constexpr int W = decltype(w)::value, K = decltype(kind)::value;
    return e4m3 ? append_kernel<W, K, true> : append_kernel<W, K, false>;
  });
  return launch_overlapped(kern, grid, block, 0, 0, stream, p);
}

cudaError_t launch_slots(const SlotArgs& a, cudaStream_t stream) {
  SlotArgs p = a;
  p.in_place = a.seq_lens == a.ctx_lens || (a.n_free_out != nullptr && a.n_free_out == a.n_free);
  const size_t smem = 3 * sizeof(int32_t) * (size_t)a.B;
  // per device and cheap, so set on every call that needs it
  if (smem > 48 * 1024) {
    cudaError_t err = cudaFuncSetAttribute(
        slots_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
        (int)(3 * sizeof(int32_t) * ATTN_SLOTS_MAX_BATCH));
    if (err != cudaSuccess) return err;
  }
  // A token a thread.  Small steps take small blocks, whose scan is shorter
  // (64 requests of one token: 256 threads); in place the grid is one cluster
  // of at most the portable size.
  const int most = a.B > a.max_tokens ? a.B : a.max_tokens;
  const int threads = most <= 2048 ? 256 : kSlotThreads;
  int ctas = (most + threads - 1) / threads;
  if (p.in_place) {
    int c = 1;
    while (c < 8 && c < ctas) c *= 2;
    ctas = c;
  } else {
    int sms = 0;
    cudaError_t err = sm_count(&sms);
    if (err != cudaSuccess) return err;
    if (ctas > sms) ctas = sms;
  }
  return launch_overlapped(slots_kernel, dim3((unsigned)ctas), dim3((unsigned)threads), smem,
                           p.in_place ? (unsigned)ctas : 0u, stream, p);
}

}  // namespace attn
