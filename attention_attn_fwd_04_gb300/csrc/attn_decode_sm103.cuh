// attn_decode_sm103.cuh -- attention of one new token per request over a
// paged key/value cache (compiled once per cache type: attn_decode_bf16.cu,
// attn_decode_e4m3.cu).
//
//   s_j = scale <q, k_j>, modified as in the forward; O = softmax(s) V,
//   LSE = ln sum_j exp(s_j), over the keys of one request.
//
// What bounds it: every visible key and value is read once, 4 D bytes per
// key and kv head (2 D in e4m3), against 4 D flops per key and query head:
// a flop per byte for each head of a group, two in e4m3.  A unit serves up to
// 32 heads, so that is at most 32 (64 in e4m3) of the tensor cores' 282, and
// the kernel is built around keeping loads in flight.
//
// Layout of the work: the keys of all requests are cut into units of 64
// or 128 keys of one (request, kv head, run of query heads); a persistent grid takes
// equal runs of consecutive units, so a long context is split over many CTAs
// and short ones share one, whatever the lengths are.  A row whose units lie
// in one CTA is finished there; else each CTA leaves its part (running max,
// sum, unnormalised O in fp32) in the workspace and a second kernel joins
// the parts in the order of the CTAs.  A CTA has at most two such parts (its
// first and its last row), so the workspace does not grow with the batch.
//
// Few rows of short contexts (a cluster's worth of CTAs for every row, and a
// few units for every CTA) take a shorter way, without the scan of lengths,
// the workspace and the second kernel: a cluster per row, whose CTAs take its
// units in turn and join through each other's shared memory.
//
// Many rows of short contexts take another: a warp per row, no joins at all.
// The host sees that from the table's width and the window; where the table
// is wide, the kernel does from the lengths that it scans anyway.
//
// Else, inside a CTA each of four warps owns a quarter of a unit's keys and is a
// pipeline of its own: it copies its keys and values into its own ring in
// shared memory and waits for nobody but itself until the row ends, where
// the warps' four partial softmaxes are joined.  The ring runs on across the
// ends of rows.  Two ways to copy, by the page size:
//  - pages that hold whole tiles of 16 keys (page_size a multiple of 16): one
//    TMA box of 16 rows per tile, swizzled, a few instructions of one lane.
//    Rows of a box that are not the request's are cleared in shared memory;
//  - others: cp.async, 16 bytes a lane, row by row, zeros for rows out of
//    range.
// Either way nothing that lies behind a sequence reaches the sums.
//
// Tensor cores: mma.sync m16n8k16 with keys (then columns of V) as the 16 rows
// and 8 query heads of the group as the 8 columns: S^T = K Q^T and O^T += V^T
// P^T, so a group of 8 heads fills the tile and O takes D / 4 registers a
// thread.  P^T comes from S^T's registers by movmatrix.  Fewer than 16 query
// rows per kv head are too few for tcgen05 (64 or 128 rows), and the work is
// a few percent of what even mma.sync does.
//
// P is rounded to the 16-bit type of the products (bf16, or fp16 for an 8-bit
// cache).  What the rounding leaves over is a second such number that is
// multiplied too, so P carries 16 bits or more and O is as exact as its own
// rounding: before that it is off by about 2e-6 of itself over 131072 keys in
// bf16, where fp32 weights give 6e-7, and of 4096 elements 9 and 2 come out as
// the other neighbour.  (A weight without a remainder times an infinite value
// is NaN, so such a column is NaN.)
//
// Measured on GB300 (keys and values read, of the 6.78 TB/s of a copy): 64
// requests up to 8192 tokens, 32 heads on 8, D 128, bf16 167 us (95%; the
// kernel alone 164); one of 131072 tokens 87 us (91%); 32 up to 16384 in e4m3
// 96 us (90%); window 1024 with soft cap, 48 x 16 heads 67.5 us (88%).  With
// the arithmetic left out the loads alone take 97 to 99% of these times.  One
// request of 500 tokens, 16 heads: 5.5 us, all latency.

#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "generation_internal.h"
#include "sm103_ptx.cuh"

namespace attn {

// Workspace of a call: one descriptor per CTA, then the parts.
struct JoinDesc {
  int32_t parts;   // CTAs that hold a part of the row this CTA's run ends in, 0: none
  int32_t first;   // part index of the first (2 c + {0, 1}); the next are 2 c' of the CTAs behind
  int32_t b;       // request
  int32_t head;    // first query head
};

// Tiles of 8 query heads of a kv head's group that one unit serves: the
// largest groups take runs of 32 heads, each of which reads the keys again.
inline int decode_tiles(int group) { return group <= 8 ? 1 : group <= 16 ? 2 : 4; }
// Most CTAs of a grid (sizes the workspace): four, three or two on each of
// 160 SMs, as the accumulators leave room.
inline int decode_max_ctas(int tiles) { return tiles == 1 ? 640 : tiles == 2 ? 480 : 320; }
inline size_t decode_desc_bytes(int tiles) { return sizeof(JoinDesc) * (size_t)decode_max_ctas(tiles); }

struct DecodeParams {
  CUtensorMap k_map, v_map;  // BULK: (128 bytes, half, row, head, page), boxes of 16 rows
  DecodeArgs a;
  uint32_t page_mul;     // key / page_size = (key * page_mul) >> page_shift for key < 2^30
  uint32_t page_shift;
  int group;             // query heads per kv head
  int runs;              // runs of 8 NT query heads per kv head
  float scale_log2;      // scale * log2 e
  float cap, inv_cap;    // soft cap times log2 e, and ln 2 / soft cap
  JoinDesc* desc;
  uint64_t budget_ns;    // longest wait for a copy
  int debug_stall;       // test hook: wait for a copy that never comes
  int cluster;           // CTAs per row, a cluster; 0: equal shares of all units
  int whole_rows;        // shares end where rows do: nothing to join
  int warps;             // warps take rows: all warps of the grid; 0: a row is its CTAs'
  int warp_keys;         // not known to the host: rows of so many keys at most are warps'
  float* parts;          // [2 * CTAs][8 NT][D + 4]: O, then m and l
};

namespace {

constexpr int kWarps = 4;
constexpr int kDecThreads = kWarps * 32;
// Most units of a CTA where a cluster takes a row.  One request of 16 heads,
// bf16, the cluster against equal shares and a join: 2 units a CTA (1000
// keys) 7.1 against 7.7 us, 4 units 9.5 against 9.0, 8 units 14 against 11.6;
// in e4m3 2 units (2000 keys) 8.0 against 8.8, 4 units 10.9 against 10.4.
// Rows of one unit are not split at all: 5.1 us without the cluster, 5.8 with.
constexpr int kClusterUnits = 3;
// Most units of a row that is never split: 64 requests of 8 kv heads, bf16, up
// to 180 keys (3 units) 10.6 us whole and 13.2 split and joined, up to 240
// (4 units) 13.6 and 13.4.
constexpr int kWholeUnits = 3;
// Most steps (of 16 or 32 keys) of a row that one warp takes: no join of the
// warps and four times the rows under way.  With four rows and more for each
// CTA, this many: 2400 rows of 4 heads, bf16, D 128, up to 8 keys 8.1 us, 19.5
// with a CTA per row; 240 keys (15 steps) 47 and 51, 480 keys 85 and 79.  From
// three rows for two CTAs on half as many, lest the longest row's warp come
// last: 1200 such rows up to 120 keys 12.6 and 18.6, but 168 x 8 up to 246 keys
// of uneven lengths 19.2 and 15.7; more than 8 heads a row save more, 16 heads
// 600 rows up to 240 keys 23 and 30.  From a row for each CTA on, 4: 600 rows
// of 4 heads up to 60 keys 7.8 and 9.0, up to 120 keys 11.7 and 11.4.  Else 1:
// 200 rows up to 8 keys 4.4 and 5.4, up to 60 7.3 and 5.9 (more than 16 heads:
// none, 9.5 and 9.6).  Rows that are copied key by key keep a warp's lanes
// busy longer, so half of that: 2400 rows up to 240 keys, pages of 24, 60.5 us
// and 59.9, up to 120 keys 34.5 and 39.7.
constexpr int kWarpSteps = 16;
constexpr int kJoinThreads = 128;
constexpr int kJoinParts = 32;  // read at once
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kMaxBias = 0x1p127f;  // times log2(e) below FLT_MAX

// P of an 8-bit cache is held in fp16, scaled by 2^14: its smallest steps
// are then 2^-38 of the row's largest weight, beyond what fp32 sums keep of a
// column to which that weight's value adds.  Where that value is 0 (8-bit
// values often are) such weights' part of the column is off by up to 2^-39 of
// their values each.
constexpr float kHalfShift = 14.0f;

__device__ __forceinline__ void dec_error(DeviceStatus* st, int site, int detail,
                                          int code = ATTN_ERR_DEVICE_CHECK) {
  if (atomicCAS(&st->code, 0, code) == 0) {
    st->where = site;
    st->block = blockIdx.x;
    st->detail = detail;
  }
}

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// 8x8 transpose of 16-bit elements across the warp.
__device__ __forceinline__ uint32_t movmatrix_t(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// D (16 x 8, fp32) += A (16 x 16) B (16 x 8); bf16, or fp16 for HALF.
template <bool HALF>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if (HALF)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two e4m3 (low 16 bits) to two fp16, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_h2(uint32_t w) {
  uint32_t r;
  const uint16_t h = (uint16_t)w;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(h));
  return r;
}

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <bool HALF>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  return HALF ? pack_h2(lo, hi) : ptx::pack_bf16x2(lo, hi);
}
// What pack2 left over of (lo, hi) in w, packed the same way.
template <bool HALF>
__device__ __forceinline__ uint32_t pack2_rest(uint32_t w, float lo, float hi) {
  float a, b;
  if (HALF) {
    asm("{\n\t.reg .f16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\t"
        "cvt.f32.f16 %1, h;\n\t}"
        : "=f"(a), "=f"(b)
        : "r"(w));
  } else {
    a = __uint_as_float(w << 16);
    b = __uint_as_float(w & 0xffff0000u);
  }
  return pack2<HALF>(lo - a, hi - b);
}

// 16 bytes global -> shared, zeros when !valid.
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool valid) {
  const uint32_t n = valid ? 16u : 0u;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// NT: tiles of 8 query heads that one unit serves.
template <int D, bool E4M3, int NT>
struct Cfg {
  static constexpr int kElem = E4M3 ? 1 : 2;
  static constexpr int kRowBytes = D * kElem;           // 256, 128 or 64
  // tiles of 16 keys, per warp and unit
  static constexpr int kKeyTiles = kRowBytes == 256 ? 1 : 2;
  // and of those, the ones in registers together: 32 heads leave room for two
  // only where a row is 64 bytes (e4m3, D 64: 71 us with two, 82 one by one),
  // but a unit of two taken one by one halves the work per unit (32 heads on
  // one, 64 requests of 16000 keys: bf16, D 64, 80 us and 88 with units of one
  // tile; e4m3, D 128, 122 and 130)
  static constexpr int kStep = NT == 4 && kRowBytes == 128 ? 1 : kKeyTiles;
  static constexpr int kWarpKeys = 16 * kKeyTiles;
  static constexpr int kUnitKeys = kWarps * kWarpKeys;
  static constexpr int kVecs = kRowBytes / 16;          // 16-byte pieces of a row
  static constexpr int kRowsPerCopy = 32 / kVecs;       // rows one warp-wide copy covers
  static constexpr int kCopies = 16 / kRowsPerCopy;     // per tile of 16 keys
  static constexpr int kHalfStage = kWarpKeys * kRowBytes;
  static constexpr int kStage = 2 * kHalfStage;         // keys, then values
  // As many CTAs as their accumulators leave room for; 12 warps rather than 8
  // are worth more than the third stage they cost (e4m3, D 128: 96 us and 107).
  // 64-column e4m3 takes 4 x 12 KB: 36 us, 42 with 3 x 16 KB; bf16 takes 3
  // (47 us and 48).
  static constexpr bool kSmall = D == 64 && E4M3 && NT == 1;
  static constexpr int kCtasPerSm =
      kSmall ? 4 : NT == 1 || (NT == 2 && D == 64) ? 3 : 2;
  static constexpr int kRingKb = kCtasPerSm == 4 ? 12 : kCtasPerSm == 3 ? 16 : 24;  // per warp
  static constexpr int kStages = kRingKb * 1024 / kStage;
  static constexpr int kRing = kWarps * kStages * kStage;
  // At the end of a row a warp's O (8 query heads at a time, fp32) goes into
  // the stage that it has just used; the heads' m and l have a place of their
  // own, [warp][head][2], as have a cluster's CTA's, [head][2].
  static_assert(kStage >= 8 * D * 4 && NT <= kWarps, "O fits a stage, a tile of heads a warp");
  static constexpr int kStats = kWarps * 8 * 2 * 4, kPartStats = 8 * NT * 2 * 4;
  static constexpr int kJoin = kStats + kPartStats;
  static constexpr int kBars = 8 * (kWarps * kStages + 1);  // mbarriers, the last for tests
  // Queries of more than 8 heads stay in shared memory, in the order the
  // lanes take them ([tile][k-step][lane], 8 bytes), and their scales.
  static constexpr bool kSharedQ = NT > 1;
  static constexpr int kQ = kSharedQ ? NT * (D / 16) * 32 * 8 + NT * 8 * 4 : 0;
  // Warps that take a row each have queries each; up to 16 heads all CTAs have
  // that room.
  static constexpr int kBase = kRing + kJoin + kQ + kBars;
  static constexpr int kWarpSmem = kBase + (kWarps - 1) * kQ;
  static constexpr int kSmem = NT <= 2 ? kWarpSmem : kBase;
  static_assert(kStages >= 2, "a stage in use and one in flight");
};

// Place of 16-byte piece v of row r in a warp's keys (or values): row behind
// row, with the swizzle of the TMA's 128-byte mode (64-byte mode for 64-byte
// rows) on lines of that length.  The pieces that one ldmatrix reads together
// fall into different banks, or two by two for rows of two lines; halves of
// such rows apart, without that conflict, took two boxes a tile and 1% more
// time.
template <int VECS>
__device__ __forceinline__ uint32_t piece(int r, int v) {
  if (VECS == 16) return (uint32_t)(r * 16 + (v ^ ((2 * r + (v >> 3)) & 7))) * 16u;
  return (uint32_t)(r * VECS + (VECS == 8 ? v ^ (r & 7) : v ^ ((r >> 1) & 3))) * 16u;
}

// Tiled copy of a box (elements of 128 bytes, halves of a row, rows) global ->
// shared, completion counted on mbarrier `bar`.
__device__ __forceinline__ void tma_load_rows(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                              int row, int head, int page) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(0), "r"(row), "r"(head), "r"(page)
      : "memory");
}

// Loads from the shared memory of any CTA of the cluster.
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float x;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(addr) : "memory");
  return x;
}
__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Bounded wait on an mbarrier phase: false once the time is up.
__device__ __forceinline__ bool wait_copy(uint32_t bar, uint32_t parity, uint64_t budget_ns) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = ptx::globaltimer_ns();
  for (;;) {
    if (ptx::mbar_try_wait_hint(bar, parity, 20000)) return true;
    if (ptx::globaltimer_ns() - t0 > budget_ns) return false;
  }
}

// tanh x to a relative error of 2^-20, without branches: below 1/4 the odd
// series to x^7 (next term 62/2835 x^8 < 2^-21 of x there), else
// 1 - 2 / (1 + e^2x) (its two roundings and the reciprocal's are below 2^-22,
// against a value of at least 0.24).  NaN stays NaN, and the ends are +-1.
__device__ __forceinline__ float tanh_scores(float x) {
  const float z = x * x;
  float q = fmaf(z, -17.0f / 315.0f, 2.0f / 15.0f);
  q = fmaf(z, q, -1.0f / 3.0f);
  const float small = fmaf(x * z, q, x);
  const float e = ptx::ex2_approx(x * (2.0f * kLog2e));
  const float large = fmaf(-2.0f, ptx::rcp_approx(1.0f + e), 1.0f);
  return fabsf(x) < 0.25f ? small : large;
}

// Keys [lo, len) of request b.
__device__ __forceinline__ void key_range(const DecodeArgs& a, int b, int& lo, int& len) {
  const int64_t most = (int64_t)a.max_pages * a.page_size;
  int64_t n = a.seq_lens[b];
  n = n < 0 ? 0 : n > most ? most : n;
  len = (int)n;
  lo = (a.window > 0 && n > a.window) ? (int)(n - a.window) : 0;
}

// The results of a request without a key, by `of` threads.
__device__ __forceinline__ void empty_request(const DecodeArgs& a, int b, int D, int i, int of) {
  uint4* o = reinterpret_cast<uint4*>(a.out + (int64_t)b * a.H * D);
  for (int j = i; j < a.H * D / 8; j += of) o[j] = make_uint4(0, 0, 0, 0);
  if (a.lse != nullptr)
    for (int j = i; j < a.H; j += of) a.lse[(int64_t)b * a.H + j] = -INFINITY;
}

// a / b of numbers >= 0; 64-bit division is many times the work.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

// `units` in G shares that differ by one at most, the larger ones first.
struct Shares {
  int64_t each;   // a share, but for the first `more`, which have one more
  int64_t more;
  __device__ __forceinline__ Shares(int64_t units, int64_t G)
      : each(quotient(units, G)), more(units - each * G) {}
  __device__ __forceinline__ int64_t begin(int64_t c) const {
    return c * each + (c < more ? c : more);
  }
  // the share that unit u is in
  __device__ __forceinline__ int64_t of(int64_t u) const {
    const int64_t first = more * (each + 1);
    return u < first ? quotient(u, each + 1) : more + quotient(u - first, each);
  }
};

// A place in the linear order of units: request, (kv head, run), unit.
struct Cursor {
  int b, hr, t;       // request, kv head * runs + run, unit of the row
  int lo, len, t0, nt;  // its keys, its first unit's index and count
};

template <int UNIT>
__device__ __forceinline__ void cursor_row(const DecodeArgs& a, Cursor& c) {
  key_range(a, c.b, c.lo, c.len);
  c.t0 = c.lo / UNIT;
  c.nt = (c.len + UNIT - 1) / UNIT - c.t0;
}
// To the next unit (of a CTA that takes every step-th); only called while
// there is one.
template <int UNIT>
__device__ __forceinline__ void cursor_next(const DecodeArgs& a, int per_b, int step, Cursor& c) {
  c.t += step;
  if (c.t < c.nt) return;
  c.t = 0;
  if (++c.hr < per_b) return;
  c.hr = 0;
  do {
    if (++c.b >= a.B) return;
    cursor_row<UNIT>(a, c);
  } while (c.nt == 0);
}
// The same of a warp that takes every warps-th row.
template <int UNIT>
__device__ __forceinline__ void cursor_next_warp(const DecodeArgs& a, int per_b, int warps,
                                                 Cursor& c) {
  if (++c.t < c.nt) return;
  c.t = 0;
  int row = c.b * per_b + c.hr;
  do {
    row += warps;
    c.b = row / per_b;
    if (c.b >= a.B) return;
    cursor_row<UNIT>(a, c);
  } while (c.nt == 0);
  c.hr = row - c.b * per_b;
}

// The kv head of a cursor's row (groups of up to 32 heads are one run).
__device__ __forceinline__ int kv_head(const DecodeParams& p, const Cursor& c) {
  return p.runs == 1 ? c.hr : c.hr / p.runs;
}

// The units [u0, u1) from cc on of a CTA, or of a warp that takes every
// warps-th row (WARPS).
template <int D, bool E4M3, int NT, bool MODS, bool BULK, bool WARPS>
__device__ __forceinline__ void decode_rows(const DecodeParams& p, unsigned char* smem, Cursor cc,
                                            int64_t u0, int64_t u1, int64_t units, int64_t G,
                                            int warps) {
  using C = Cfg<D, E4M3, NT>;
  constexpr int kUnit = WARPS ? C::kWarpKeys : C::kUnitKeys;
  const DecodeArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int gid = lane >> 2, tig = lane & 3;
  const int64_t me = blockIdx.x;
  const int per_b = a.H_kv * p.runs, step = p.cluster > 0 ? p.cluster : 1;
  float* s_ml = reinterpret_cast<float*>(smem + C::kRing);
  float* s_part_ml = reinterpret_cast<float*>(smem + C::kRing + C::kStats);
  const uint32_t bars0 = ptx::smem_addr(smem) + C::kRing + C::kJoin + C::kQ;
  const uint32_t bars = bars0 + (uint32_t)(w * C::kStages * 8);
  const uint32_t never = bars0 + kWarps * C::kStages * 8;
  auto next = [&](Cursor& c) {
    if (WARPS)
      cursor_next_warp<kUnit>(a, per_b, warps, c);
    else
      cursor_next<kUnit>(a, per_b, step, c);
  };
  const int first_key = WARPS ? 0 : w * C::kWarpKeys;  // of the warp, in a unit
  // warps that take rows have queries of their own, all but the first's at the end
  uint2* s_q = reinterpret_cast<uint2*>(
      smem + (WARPS && w > 0 ? C::kBase + (w - 1) * C::kQ : C::kRing + C::kJoin));
  float* s_down = reinterpret_cast<float*>(s_q + NT * (D / 16) * 32);
  if (BULK && (ptx::smem_addr(smem) & 1023u) != 0) {  // the boxes' swizzle goes by address
    if (tid == 0) dec_error(a.status, kSiteWait, -1);
    u1 = u0;
  }
  if (u0 >= u1 && (WARPS || p.cluster == 0)) return;
  // p.cluster: this CTA's part of its row.  The O of tile n of the heads lies
  // in the second stage of warp n's ring, which no copy is on its way to when
  // the row ends.
  auto part_row = [&](int head) {
    return reinterpret_cast<float*>(smem + (head >> 3) * C::kStages * C::kStage + C::kStage) +
           (head & 7) * D;
  };
  if (!WARPS && p.cluster > 0 && u0 >= u1) {
    for (int i = tid; i < 8 * NT * D; i += kDecThreads) part_row(i / D)[i % D] = 0.f;
    if (tid < 8 * NT) {
      s_part_ml[2 * tid] = -INFINITY;
      s_part_ml[2 * tid + 1] = 0.f;
    }
  }

  // ---- the ring -----------------------------------------------------------
  const uint32_t ring = ptx::smem_addr(smem) + (uint32_t)(w * C::kStages * C::kStage);
  Cursor lc = cc;      // the unit being loaded
  int64_t lu = u0;
  int ring_load = 0;   // stage the next load goes to
  // Pages of the unit being loaded, as read from the table, and the row in
  // them: BULK: of the lane's tile of 16 keys (the first lanes), else of the
  // lane's key.  The table is read one unit ahead and its entry not looked at
  // before the load that needs it, so its latency passes behind the
  // arithmetic of a unit.
  int page = 0, row_in_page = 0;
  bool seen = false;   // a key is one of the row's, so page was read
  auto look_up = [&]() {
    const int first = (lc.t0 + lc.t) * kUnit + first_key;
    const int key = first + (BULK ? 16 * lane : lane & (C::kWarpKeys - 1));
    seen = key + (BULK ? 15 : 0) >= lc.lo && key < lc.len && (!BULK || lane < C::kKeyTiles);
    if (seen) {
      const int col = (int)(((uint64_t)(uint32_t)key * p.page_mul) >> p.page_shift);
      row_in_page = key - col * a.page_size;
      page = a.table[lc.b * a.table_stride + col];
    }
  };
  const int cv = lane % C::kVecs, cr = lane / C::kVecs;
  auto load = [&]() {  // the unit at lc into the next stage, then look ahead
    if (lu < u1) {
      const int h = kv_head(p, lc);
      const uint32_t st = ring + (uint32_t)(ring_load * C::kStage);
      const bool held = seen && (unsigned)page < (unsigned)a.num_pages;
      if (seen && !held) dec_error(a.status, kSiteTable, page);
      if (BULK) {
        constexpr int kTileBytes = 16 * C::kRowBytes;
        const uint32_t bar = bars + 8 * ring_load;
        const int tiles = __popc(__ballot_sync(0xffffffffu, seen));
        if (lane == 0) ptx::mbar_arrive_expect_tx(bar, (uint32_t)(tiles * 2 * kTileBytes));
        __syncwarp();
        if (seen) {
          // a page outside the cache is out of the map's bounds: zeros
          const int pg = held ? page : a.num_pages;
          const uint32_t dst = st + lane * kTileBytes;
          tma_load_rows(dst, &p.k_map, bar, row_in_page, h, pg);
          tma_load_rows(dst + C::kHalfStage, &p.v_map, bar, row_in_page, h, pg);
        }
        __syncwarp();
      } else {
        const char* kb = static_cast<const char*>(a.kc) + (h * a.kcs[1]) * C::kElem + cv * 16;
        const char* vb = static_cast<const char*>(a.vc) + (h * a.vcs[1]) * C::kElem + cv * 16;
#pragma unroll
        for (int i = 0; i < C::kKeyTiles * C::kCopies; ++i) {
          const int r = cr + i * C::kRowsPerCopy;
          const int pg = __shfl_sync(0xffffffffu, held ? page : -1, r);
          const int rp = __shfl_sync(0xffffffffu, row_in_page, r);
          const bool ok = pg >= 0;
          const int64_t ko = ok ? pg * a.kcs[0] + rp * a.kcs[2] : 0;
          const int64_t vo = ok ? pg * a.vcs[0] + rp * a.vcs[2] : 0;
          cp16(st + piece<C::kVecs>(r, cv), kb + ko * C::kElem, ok);
          cp16(st + C::kHalfStage + piece<C::kVecs>(r, cv), vb + vo * C::kElem, ok);
        }
      }
      if (++lu < u1) {
        next(lc);
        look_up();
      }
    }
    if (!BULK) cp_commit();
    if (++ring_load == C::kStages) ring_load = 0;
  };
  look_up();
#pragma unroll 1
  for (int i = 0; i < C::kStages - 1; ++i) load();

  // ---- the rows -----------------------------------------------------------
  // Thread (gid, tig) of a warp: keys gid and gid + 8 of a tile (columns of
  // V later), query heads 2 tig and 2 tig + 1 of a tile of 8.
  constexpr int kSteps = D / 16;      // k-steps of S, and 16-column tiles of O
  uint32_t qf[kSteps][2];             // one tile's queries (a warp's share of more tiles)
  float o[kSteps][NT][4];
  float m[NT][2], l[NT][2], qscale[NT][2];
  float slope[NT][2];                 // ALiBi, in units of log2
  int ring_use = 0;
  uint32_t phase = 0;
  bool dead = false;   // a copy did not come in time: no more loads, no results
  bool fresh = true;
  const int lr = lane & 7, lm = lane >> 3;
  // Reads tile n of the queries from head q0 of kv head h into qf; returns
  // the factor that undoes the scaling of head gid (8-bit caches).
  auto read_queries = [&](int h, int q0, int n) {
    const int r = q0 + 8 * n + gid;
    const bool have = r < p.group;
    // lane's columns of a k-step: 2 tig, 2 tig + 1 and the same + 8; for an
    // 8-bit cache 4 tig .. 4 tig + 3, the order that ldmatrix hands out the
    // keys' bytes in
    const __nv_bfloat16* src = a.q +
                               (have ? cc.b * a.qs[0] + (h * p.group + r) * a.qs[1] : 0) +
                               tig * (E4M3 ? 4 : 2);
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      qf[k][0] = have ? *reinterpret_cast<const uint32_t*>(src + 16 * k) : 0u;
      qf[k][1] = have ? *reinterpret_cast<const uint32_t*>(src + 16 * k + (E4M3 ? 2 : 8)) : 0u;
    }
    if (!E4M3) return 1.0f;
    // bf16 queries to fp16, exactly but for parts below 2^-28 of the head's
    // largest element: scaled by a power of two that puts that one at
    // 2^13 .. 2^14
    float big = 0.f;
#pragma unroll
    for (int k = 0; k < kSteps; ++k)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        big = fmaxf(big, fmaxf(fabsf(__uint_as_float(qf[k][j] << 16)),
                               fabsf(__uint_as_float(qf[k][j] & 0xffff0000u))));
    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
    int e = 0;
    if (big > 0.f && big < INFINITY) {
      e = 14 - (ilogbf(big) + 1);
      e = e > 100 ? 100 : e;
    }
    const float up = ldexpf(1.0f, e);
#pragma unroll
    for (int k = 0; k < kSteps; ++k)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        qf[k][j] = pack_h2(__uint_as_float(qf[k][j] << 16) * up,
                           __uint_as_float(qf[k][j] & 0xffff0000u) * up);
    return ldexpf(1.0f, -e);
  };
  for (int64_t u = u0; u < u1; ++u) {
    if (fresh) {  // a row begins: its queries, an empty softmax
      fresh = false;
      const int h = kv_head(p, cc);
      const int q0 = (cc.hr - h * p.runs) * 8 * NT;  // first head of the group's run
      const float ks = (E4M3 && a.k_scale != nullptr) ? a.k_scale[h] : 1.0f;
      float down = 1.0f;
      if (C::kSharedQ) {  // the last row's readers have met at its end
        constexpr bool alone = WARPS;
        for (int n = alone ? 0 : w; n < NT; n += alone ? 1 : kWarps) {
          down = read_queries(h, q0, n);
#pragma unroll
          for (int k = 0; k < kSteps; ++k)
            s_q[(n * kSteps + k) * 32 + lane] = make_uint2(qf[k][0], qf[k][1]);
          if (tig == 0) s_down[8 * n + gid] = down;
        }
        if (alone)
          __syncwarp();
        else
          __syncthreads();
      } else {
        down = read_queries(h, q0, 0);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          qscale[n][i] = p.scale_log2 * ks;
          if (E4M3) {
            qscale[n][i] *= C::kSharedQ ? s_down[8 * n + 2 * tig + i]
                                        : __shfl_sync(0xffffffffu, down, 4 * (2 * tig + i));
            qscale[n][i] = fmaxf(qscale[n][i], FLT_MIN);  // not 0, which masks (-inf) are times
          }
          if (MODS) {
            const int ri = q0 + 8 * n + 2 * tig + i, head = h * p.group + ri;
            slope[n][i] = 0.f;
            if ((a.score_flags & ATTN_SCORE_ALIBI) && ri < p.group)
              slope[n][i] = kLog2e * (a.alibi_slopes != nullptr
                                          ? a.alibi_slopes[head]
                                          : exp2f(-8.0f * (float)(head + 1) / (float)a.H));
          }
          m[n][i] = -INFINITY;
          l[n][i] = 0.f;
        }
#pragma unroll
        for (int k = 0; k < kSteps; ++k) o[k][n][0] = o[k][n][1] = o[k][n][2] = o[k][n][3] = 0.f;
      }
    }

    const int key0 = (cc.t0 + cc.t) * kUnit + first_key;
    const bool whole = key0 >= cc.lo && key0 + C::kWarpKeys <= cc.len;
    const uint32_t st = ring + (uint32_t)(ring_use * C::kStage);
    if (BULK) {
      // once dead, what is still in flight gets a short time to land
      bool here = u >= lu || wait_copy(p.debug_stall && !dead ? never : bars + 8 * ring_use,
                                       phase, dead ? 1000000 : p.budget_ns);
      if (__any_sync(0xffffffffu, !here) && !dead) {
        dead = true;
        if (lane == 0) dec_error(a.status, kSiteWait, ring_use, ATTN_ERR_TIMEOUT);
        if (p.debug_stall) wait_copy(bars + 8 * ring_use, phase, 1000000);
      }
    } else {
      cp_wait<C::kStages - 2>();
    }
    __syncwarp();
    // the stage used last is free now: every lane has passed its reads
    if (!dead) load();
    __syncwarp();  // the matrix instructions below want the warp together

    if (++ring_use == C::kStages) {
      ring_use = 0;
      phase ^= 1;
    }
    if (!dead && key0 < cc.len && key0 + C::kWarpKeys > cc.lo) {
      if (BULK && !whole) {
        // values of rows that are not the request's: a weight of 0 times
        // whatever lies there must be 0.  (Scores of such keys are replaced.)
        for (int i = lane; i < C::kWarpKeys * C::kVecs; i += 32) {
          const int key = key0 + i / C::kVecs;
          if (key < cc.lo || key >= cc.len)
            ptx::sts_v4(st + C::kHalfStage + piece<C::kVecs>(i / C::kVecs, i % C::kVecs), 0, 0, 0, 0);
        }
        ptx::fence_proxy_async_smem();  // before the copy that comes here next
        __syncwarp();
      }
#pragma unroll 1
      for (int j0 = 0; j0 < C::kKeyTiles; j0 += C::kStep) {
      if (C::kStep < C::kKeyTiles &&
          (key0 + 16 * j0 >= cc.len || key0 + 16 * (j0 + C::kStep) <= cc.lo))
        continue;  // none of the row's keys
      // ---- S^T = K Q^T: tiles of 16 keys x 8 heads ------------------------
      float s[C::kStep][NT][4];
#pragma unroll
      for (int j = 0; j < C::kStep; ++j) {
#pragma unroll
        for (int n = 0; n < NT; ++n) s[j][n][0] = s[j][n][1] = s[j][n][2] = s[j][n][3] = 0.f;
        if (!E4M3) {
#pragma unroll
          for (int k = 0; k < kSteps; ++k) {
            uint32_t f[4];  // keys 0-7, 8-15 of the step's first 8 columns, then its last 8
            ldsm_x4(st + piece<C::kVecs>(16 * (j0 + j) + lr + 8 * (lm & 1), 2 * k + (lm >> 1)), f);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const uint2 q = C::kSharedQ ? s_q[(n * kSteps + k) * 32 + lane]
                                          : make_uint2(qf[k][0], qf[k][1]);
              mma16816<false>(s[j][n], f, q.x, q.y);
            }
          }
        } else {
#pragma unroll
          for (int k = 0; k < kSteps; k += 2) {
            uint32_t f[4];  // step k: keys 0-7, keys 8-15; then step k + 1
            ldsm_x4(st + piece<C::kVecs>(16 * (j0 + j) + lr + 8 * (lm & 1), k + (lm >> 1)), f);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint32_t g[4] = {e4m3x2_to_h2(f[2 * x]), e4m3x2_to_h2(f[2 * x + 1]),
                                     e4m3x2_to_h2(f[2 * x] >> 16),
                                     e4m3x2_to_h2(f[2 * x + 1] >> 16)};
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                const uint2 q = C::kSharedQ ? s_q[(n * kSteps + k + x) * 32 + lane]
                                            : make_uint2(qf[k + x][0], qf[k + x][1]);
                mma16816<true>(s[j][n], g, q.x, q.y);
              }
            }
          }
        }
      }

      // ---- running softmax in units of log2 -------------------------------
      // A head's maximum m is one for the warp, but looked at lane by lane:
      // only when some lane's score is above its m (seldom, once a row is
      // under way) do the lanes agree on a new one.
      if (MODS) {
#pragma unroll
        for (int j = 0; j < C::kStep; ++j)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x) s[j][n][x] *= qscale[n][x & 1];
        const int back0 = cc.len - 1 - (key0 + gid);  // query position minus the first key's
        if (a.score_flags & ATTN_SCORE_ALIBI) {
#pragma unroll
          for (int j = 0; j < C::kStep; ++j)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const float back = (float)(back0 - 16 * (j0 + j) - 8 * (x >> 1));
#pragma unroll
              for (int n = 0; n < NT; ++n)
                s[j][n][x] = fmaf(-slope[n][x & 1], back, s[j][n][x]);
            }
        }
        if (a.score_flags & ATTN_SCORE_RELBIAS) {
          const int h = kv_head(p, cc), q0 = (cc.hr - h * p.runs) * 8 * NT;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int64_t head = h * p.group + min(q0 + 8 * n + 2 * tig + i, p.group - 1);
              const float* bias =
                  a.rel_bias + head * (2 * (int64_t)a.rel_max + 1) + a.rel_max;
#pragma unroll
              for (int j = 0; j < C::kStep; ++j)
#pragma unroll
                for (int x = i; x < 4; x += 2) {
                  const int back = back0 - 16 * (j0 + j) - 8 * (x >> 1);  // < 0 behind the last key
                  float t = bias[-min(max(back, 0), a.rel_max)];
                  // a row of nothing but the type's lowest value is no empty
                  // row: finite biases stay finite in units of log2
                  if (fabsf(t) > kMaxBias && fabsf(t) < INFINITY) t = copysignf(kMaxBias, t);
                  s[j][n][x] = fmaf(t, kLog2e, s[j][n][x]);
                }
            }
        }
        if (a.score_flags & ATTN_SCORE_SOFTCAP) {
#pragma unroll
          for (int j = 0; j < C::kStep; ++j)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int x = 0; x < 4; ++x)
                s[j][n][x] = p.cap * tanh_scores(s[j][n][x] * p.inv_cap);
        }
      }
      float top[NT][2];
      bool grows = false;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          top[n][i] = -INFINITY;
#pragma unroll
          for (int j = 0; j < C::kStep; ++j)
#pragma unroll
            for (int x = i; x < 4; x += 2) {
              const int key = key0 + 16 * (j0 + j) + gid + 8 * (x >> 1);
              if (!whole && (key < cc.lo || key >= cc.len)) s[j][n][x] = -INFINITY;
              top[n][i] = fmaxf(top[n][i], s[j][n][x]);
            }
          if (!MODS) top[n][i] *= qscale[n][i];  // > 0
          grows |= top[n][i] > m[n][i];
        }
      }
      if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float mn = top[n][i];
            mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, 4));
            mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, 8));
            mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, 16));
            mn = fmaxf(mn, m[n][i]);
            // from the first key on mn is a number; exp2(-inf) starts at 0
            const float f = m[n][i] == mn ? 1.0f : exp2f(m[n][i] - mn);
            l[n][i] *= f;
            m[n][i] = mn;
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
              o[k][n][i] *= f;
              o[k][n][2 + i] *= f;
            }
          }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float base = (m[n][i] == -INFINITY ? 0.f : m[n][i]) - (E4M3 ? kHalfShift : 0.f);
#pragma unroll
          for (int j = 0; j < C::kStep; ++j)
#pragma unroll
            for (int x = i; x < 4; x += 2) {
              const float t = s[j][n][x];
              float e = ptx::ex2_approx(MODS ? t - base : fmaf(t, qscale[n][i], -base));
              l[n][i] += e;
              s[j][n][x] = e;
            }
        }

      // ---- O^T += V^T P^T ---------------------------------------------------
      const uint32_t sv = st + C::kHalfStage;
#pragma unroll
      for (int j = 0; j < C::kStep; ++j) {
        uint32_t pf[NT][2], pr[NT][2];  // P^T of keys 0-7 and 8-15, and what is left over
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t t = pack2<E4M3>(s[j][n][2 * x], s[j][n][2 * x + 1]);
            pf[n][x] = movmatrix_t(t);
            pr[n][x] = movmatrix_t(pack2_rest<E4M3>(t, s[j][n][2 * x], s[j][n][2 * x + 1]));
          }
        if (!E4M3) {
#pragma unroll
          for (int k = 0; k < kSteps; ++k) {
            uint32_t f[4];  // columns 0-7, 8-15 of keys 0-7, then of keys 8-15
            ldsm_x4_t(sv + piece<C::kVecs>(16 * (j0 + j) + lr + 8 * (lm >> 1), 2 * k + (lm & 1)), f);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma16816<false>(o[k][n], f, pf[n][0], pf[n][1]);
              mma16816<false>(o[k][n], f, pr[n][0], pr[n][1]);
            }
          }
        } else {
          // A transposed 16-bit unit holds two neighbouring columns of a key:
          // row gid of the tile is the even one (low byte), row gid + 8 the
          // odd one, of the 16-column piece's pair gid
#pragma unroll
          for (int k = 0; k < kSteps; k += 2) {
            uint32_t f[4];  // piece k: keys 0-7, keys 8-15; then piece k + 1
            ldsm_x4_t(sv + piece<C::kVecs>(16 * (j0 + j) + lr + 8 * (lm & 1), k + (lm >> 1)), f);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint32_t g[4] = {e4m3x2_to_h2(__byte_perm(f[2 * x], 0, 0x0020)),
                                     e4m3x2_to_h2(__byte_perm(f[2 * x], 0, 0x0031)),
                                     e4m3x2_to_h2(__byte_perm(f[2 * x + 1], 0, 0x0020)),
                                     e4m3x2_to_h2(__byte_perm(f[2 * x + 1], 0, 0x0031))};
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                mma16816<true>(o[k + x][n], g, pf[n][0], pf[n][1]);
                mma16816<true>(o[k + x][n], g, pr[n][0], pr[n][1]);
              }
            }
          }
        }
      }
      }
    }

    // ---- the row's last unit here: join the warps, write it out -----------
    if constexpr (WARPS) {
      if (cc.t + 1 == cc.nt) {
        const int h = kv_head(p, cc);
        const int q0 = (cc.hr - h * p.runs) * 8 * NT;
        const float vs = (E4M3 && a.v_scale != nullptr) ? a.v_scale[h] : 1.0f;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float g[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float lx = l[n][i];
            lx += __shfl_xor_sync(0xffffffffu, lx, 4);
            lx += __shfl_xor_sync(0xffffffffu, lx, 8);
            lx += __shfl_xor_sync(0xffffffffu, lx, 16);
            g[i] = (lx == 0.f ? 0.f : 1.0f / lx) * vs;
            const int r = q0 + 8 * n + 2 * tig + i;
            if (gid == 0 && r < p.group && a.lse != nullptr)
              a.lse[(int64_t)cc.b * a.H + h * p.group + r] =
                  lx == 0.f ? -INFINITY
                            : (m[n][i] + log2f(lx) - (E4M3 ? kHalfShift : 0.f)) * kLn2;
          }
          // 8 columns by 8 heads turned over, a head's columns to its lanes
          const int r = q0 + 8 * n + gid;
          __nv_bfloat16* out = a.out + ((int64_t)cc.b * a.H + h * p.group + r) * D;
#pragma unroll
          for (int k = 0; k < kSteps; ++k) {
            const uint32_t x =
                movmatrix_t(ptx::pack_bf16x2(o[k][n][0] * g[0], o[k][n][1] * g[1]));
            const uint32_t y =
                movmatrix_t(ptx::pack_bf16x2(o[k][n][2] * g[0], o[k][n][3] * g[1]));
            if (E4M3 && r < p.group) {  // x the even columns, y the odd ones
              *reinterpret_cast<uint2*>(out + 16 * k + 4 * tig) =
                  make_uint2(__byte_perm(x, y, 0x5410), __byte_perm(x, y, 0x7632));
            } else if (r < p.group) {
              *reinterpret_cast<uint32_t*>(out + 16 * k + 2 * tig) = x;
              *reinterpret_cast<uint32_t*>(out + 16 * k + 8 + 2 * tig) = y;
            }
            __syncwarp();
          }
        }
        fresh = true;
        __syncwarp();  // the queries have been read
      }
    } else if (cc.t + 1 == cc.nt || u + 1 == u1) {
      const int h = kv_head(p, cc);
      const int q0 = (cc.hr - h * p.runs) * 8 * NT;
      const int64_t row_u0 = u - cc.t, row_u1 = row_u0 + cc.nt;  // the row's units
      const bool complete = p.cluster == 0 && row_u0 >= u0 && row_u1 <= u1;
      const int part = (int)(2 * me) + (row_u0 > u0 ? 1 : 0);  // 0: this CTA's first row
      // the row goes on behind this CTA, and this CTA has its first unit
      if (tid == 0 && p.cluster == 0 && row_u0 >= u0 && row_u1 > u1) {
        const int64_t last = Shares(units, G).of(row_u1 - 1);  // CTA of the row's last unit
        p.desc[me] = JoinDesc{(int)(last - me + 1), part, cc.b, h * p.group + q0};
      }
      const float vs = (E4M3 && a.v_scale != nullptr) ? a.v_scale[h] : 1.0f;
      // the stage of this unit (a cluster's row: the first, all are done with)
      const int stage = p.cluster > 0 ? 0 : (int)(st - ring) / C::kStage;
      auto warp_o = [&](int warp) {
        return reinterpret_cast<float*>(smem + (warp * C::kStages + stage) * C::kStage);
      };
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        // columns are exchanged in eights by the head's pair, so that the
        // heads' stores fall into different banks
        float* mine = warp_o(w);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float lx = l[n][i];
          lx += __shfl_xor_sync(0xffffffffu, lx, 4);
          lx += __shfl_xor_sync(0xffffffffu, lx, 8);
          lx += __shfl_xor_sync(0xffffffffu, lx, 16);
          const int r = 2 * tig + i;
#pragma unroll
          for (int k = 0; k < kSteps; ++k) {
            if (E4M3) {
              *reinterpret_cast<float2*>(mine + r * D + ((16 * k + 2 * gid) ^ (tig << 3))) =
                  make_float2(o[k][n][i], o[k][n][2 + i]);
            } else {
              mine[r * D + ((16 * k + gid) ^ (tig << 3))] = o[k][n][i];
              mine[r * D + ((16 * k + gid + 8) ^ (tig << 3))] = o[k][n][2 + i];
            }
          }
          if (gid == 0)
            *reinterpret_cast<float2*>(s_ml + 2 * (w * 8 + r)) = make_float2(m[n][i], lx);
        }
        __syncthreads();
        const int jr = tid >> 4, r = q0 + 8 * n + jr;  // 16 threads a head
        float f[kWarps], top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) top = fmaxf(top, s_ml[2 * (i * 8 + jr)]);
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
          const float2 ml = *reinterpret_cast<const float2*>(s_ml + 2 * (i * 8 + jr));
          f[i] = ml.x == top ? 1.0f : ptx::ex2_approx(ml.x - top);
          sum = fmaf(ml.y, f[i], sum);
        }
        const float g = complete ? (sum == 0.f ? 0.f : 1.0f / sum) * vs : vs;
#pragma unroll
        for (int half = 0; half < D / 64; ++half) {
          const int col = 64 * half + 4 * (tid & 15);
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int i = 0; i < kWarps; ++i) {
            const float4 y = *reinterpret_cast<const float4*>(warp_o(i) + jr * D +
                                                              (col ^ ((jr >> 1) << 3)));
            acc.x = fmaf(y.x, f[i], acc.x);
            acc.y = fmaf(y.y, f[i], acc.y);
            acc.z = fmaf(y.z, f[i], acc.z);
            acc.w = fmaf(y.w, f[i], acc.w);
          }
          acc.x *= g, acc.y *= g, acc.z *= g, acc.w *= g;
          if (p.cluster > 0) {
            *reinterpret_cast<float4*>(part_row(8 * n + jr) + col) = acc;
          } else if (r < p.group) {
            if (complete)
              *reinterpret_cast<uint2*>(a.out + ((int64_t)cc.b * a.H + h * p.group + r) * D + col) =
                  make_uint2(ptx::pack_bf16x2(acc.x, acc.y), ptx::pack_bf16x2(acc.z, acc.w));
            else
              *reinterpret_cast<float4*>(
                  p.parts + ((int64_t)part * 8 * NT + 8 * n + jr) * (D + 4) + col) = acc;
          }
        }
        if ((tid & 15) == 0) {
          if (p.cluster > 0) {
            *reinterpret_cast<float2*>(s_part_ml + 2 * (8 * n + jr)) = make_float2(top, sum);
          } else if (r < p.group) {
            if (!complete)
              *reinterpret_cast<float2*>(
                  p.parts + ((int64_t)part * 8 * NT + 8 * n + jr) * (D + 4) + D) =
                  make_float2(top, sum);
            else if (a.lse != nullptr)
              a.lse[(int64_t)cc.b * a.H + h * p.group + r] =
                  sum == 0.f ? -INFINITY
                             : (top + log2f(sum) - (E4M3 ? kHalfShift : 0.f)) * kLn2;
          }
        }
        if (BULK) ptx::fence_proxy_async_smem();  // before the copies that come here next
        __syncthreads();
      }
      fresh = true;
    }
    if (u + 1 < u1) next(cc);
  }
  if (!BULK) cp_wait<0>();

  if (!WARPS && p.cluster > 0) {  // join the row's CTAs: 16-byte pieces of its O, a thread each
    __syncthreads();
    ptx::cluster_sync();
    const int rank = (int)me % step;
    const int h = kv_head(p, cc), q0 = (cc.hr - h * p.runs) * 8 * NT;
    for (int i = rank * kDecThreads + tid; i < 8 * NT * (D / 4); i += step * kDecThreads) {
      const int r = i / (D / 4), col = 4 * (i % (D / 4));
      if (q0 + r >= p.group) continue;
      const uint32_t row = ptx::smem_addr(part_row(r) + col);
      const uint32_t ml = ptx::smem_addr(s_part_ml + 2 * r);
      float top = -INFINITY, sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int c = 0; c < step; ++c) top = fmaxf(top, ld_cluster(ptx::mapa(ml, c)));
      for (int c = 0; c < step; ++c) {
        const float mc = ld_cluster(ptx::mapa(ml, c));
        const float f = mc == top ? 1.0f : ptx::ex2_approx(mc - top);
        const float4 y = ld_cluster_v4(ptx::mapa(row, c));
        sum = fmaf(ld_cluster(ptx::mapa(ml, c) + 4), f, sum);
        acc.x = fmaf(y.x, f, acc.x);
        acc.y = fmaf(y.y, f, acc.y);
        acc.z = fmaf(y.z, f, acc.z);
        acc.w = fmaf(y.w, f, acc.w);
      }
      const float inv = sum == 0.f ? 0.f : 1.0f / sum;
      const int64_t orow = (int64_t)cc.b * a.H + h * p.group + q0 + r;
      *reinterpret_cast<uint2*>(a.out + orow * D + col) = make_uint2(
          ptx::pack_bf16x2(acc.x * inv, acc.y * inv), ptx::pack_bf16x2(acc.z * inv, acc.w * inv));
      if (a.lse != nullptr && col == 0)
        a.lse[orow] = sum == 0.f ? -INFINITY
                                 : (top + log2f(sum) - (E4M3 ? kHalfShift : 0.f)) * kLn2;
    }
    __syncthreads();
    ptx::cluster_sync();  // nobody leaves while others read its part
  }
}

template <int D, bool E4M3, int NT, bool MODS, bool BULK>
__global__ void __launch_bounds__(kDecThreads, Cfg<D, E4M3, NT>::kCtasPerSm)
    decode_kernel(const __grid_constant__ DecodeParams p) {
  using C = Cfg<D, E4M3, NT>;
  extern __shared__ __align__(1024) unsigned char smem[];
  const DecodeArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  float* s_ml = reinterpret_cast<float*>(smem + C::kRing);
  const uint32_t bars0 = ptx::smem_addr(smem) + C::kRing + C::kJoin + C::kQ;
  const uint32_t bars = bars0 + (uint32_t)(w * C::kStages * 8);
  const uint32_t never = bars0 + kWarps * C::kStages * 8;
  if (BULK && lane == 0) {
    for (int i = 0; i < C::kStages; ++i) ptx::mbar_init(bars + 8 * i, 1);
    if (w == 0) {
      ptx::mbar_init(never, 1);
      ptx::prefetch_tmap(&p.k_map);
      ptx::prefetch_tmap(&p.v_map);
    }
    ptx::fence_mbar_init();
  }
  __syncthreads();
  // nothing of an earlier kernel's is read, and nothing it may read written,
  // before it is done
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int per_b = a.H_kv * p.runs;

  // ---- this CTA's run of units ----------------------------------------
  const int64_t me = blockIdx.x;
  int64_t units = 0, G = 0, u0 = 0, u1 = 0;
  const int step = p.cluster > 0 ? p.cluster : 1;
  int warps = p.warps;  // of a grid whose warps take rows, or 0
  Cursor cc;  // the unit being computed
  cc.b = cc.hr = cc.t = 0;
  if (p.cluster > 0) {
    const int row = (int)me / step, rank = (int)me - row * step;
    cc.b = row / per_b;
    cc.hr = row - cc.b * per_b;
    cc.t = rank;
    cursor_row<C::kUnitKeys>(a, cc);
    u1 = cc.nt > rank ? (cc.nt - rank + step - 1) / step : 0;
    if (tid == 0 && rank == 0 && cc.hr == 0 && a.seq_lens[cc.b] != cc.len)
      dec_error(a.status, kSiteSeqLen, cc.b);
  } else if (warps == 0) {
    // Each thread sums the units of a run of requests; the one whose run holds
    // the CTA's first unit walks it, and leaves the place for all.
    int64_t* s_sum = reinterpret_cast<int64_t*>(s_ml);  // [kWarps]
    Cursor* s_first = reinterpret_cast<Cursor*>(s_sum + kWarps);
    int* s_end = reinterpret_cast<int*>(s_first + 1);  // unit in its row of the one behind the last
    const int per = (a.B + kDecThreads - 1) / kDecThreads;
    const int rb0 = min(a.B, tid * per), rb1 = min(a.B, rb0 + per);
    int64_t mine = 0;
    bool empty = false;  // a request without a key
    bool too_long = p.warp_keys == 0;
    Cursor c;            // the run's last request; its only one in batches up to 128
    c.b = c.hr = c.t = c.lo = c.len = c.t0 = c.nt = 0;
    for (int b = rb0; b < rb1; ++b) {
      c.b = b;
      cursor_row<C::kUnitKeys>(a, c);
      mine += c.nt;
      empty |= c.nt == 0;
      too_long |= c.len - c.lo > p.warp_keys;
      if (blockIdx.x == 0 && a.seq_lens[b] != c.len) dec_error(a.status, kSiteSeqLen, b);
    }
    int64_t incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == 31) s_sum[w] = incl;
    empty = __syncthreads_or(empty);
    if (p.warp_keys != 0 && !__syncthreads_or(too_long))  // short rows after all
      warps = kWarps * (int)gridDim.x;
    units = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      if (i < w) incl += s_sum[i];
      units += s_sum[i];
    }
    units *= per_b;
    // CTAs c < G have shares, of at least one unit
    G = units < gridDim.x ? units : gridDim.x;
    if (me < G && warps == 0) {
      const Shares shares(units, G);
      u0 = shares.begin(me);
      u1 = shares.begin(me + 1);
    }
    const int64_t before = (incl - mine) * per_b;
    auto locate = [&](int64_t unit) {  // c to a unit of this thread's run
      int64_t rest = unit - before;
      if (per > 1)
        for (c.b = rb0; c.b < rb1; ++c.b) {
          cursor_row<C::kUnitKeys>(a, c);
          const int64_t n = (int64_t)c.nt * per_b;
          if (rest < n) break;
          rest -= n;
        }
      c.hr = (int)quotient(rest, c.nt);
      c.t = (int)(rest - (int64_t)c.hr * c.nt);
    };
    auto has = [&](int64_t unit) { return unit >= before && unit < incl * per_b; };
    if (u0 < u1 && has(u0)) {
      locate(u0);
      *s_first = c;
    }
    if (p.whole_rows && u0 < u1 && has(u1)) {  // nobody has unit `units`
      locate(u1);
      *s_end = c.t;
    }
    __syncthreads();
    if (u0 < u1) {
      cc = *s_first;
      if (p.whole_rows) {  // both ends back to the beginning of their row
        if (u1 < units) u1 -= *s_end;
        u0 -= cc.t;
        cc.t = 0;
      }
    }
    __syncthreads();  // all have the place: the rows may use the memory
    if (tid == 0) p.desc[me].parts = 0;
    // rows without a key, if there are any
    for (int b = (int)me; warps == 0 && empty && b < a.B; b += (int)gridDim.x) {
      int lo, len;
      key_range(a, b, lo, len);
      if (len > 0) continue;
      empty_request(a, b, D, tid, kDecThreads);
    }
  }
  if (warps != 0) {
    // This warp's rows: first, first + warps, ..
    const int first = w * (int)gridDim.x + (int)me, rows = a.B * per_b;
    int sum = 0;
    for (int64_t r = first + (int64_t)lane * warps; r < rows; r += 32 * (int64_t)warps) {
      Cursor c;
      c.b = (int)r / per_b;
      cursor_row<C::kWarpKeys>(a, c);
      sum += c.nt;
    }
    u1 = __reduce_add_sync(0xffffffffu, sum);
    if (u1 > 0) {  // to the first with a key
      cc.b = first / per_b;
      cc.hr = first - cc.b * per_b;
      cursor_row<C::kWarpKeys>(a, cc);
      if (cc.nt == 0) cursor_next_warp<C::kWarpKeys>(a, per_b, warps, cc);
    }
    for (int b = first; b < a.B; b += warps) {
      int lo, len;
      key_range(a, b, lo, len);
      if (a.seq_lens[b] != len && lane == 0) dec_error(a.status, kSiteSeqLen, b);
      if (len == 0) empty_request(a, b, D, lane, 32);
    }
  }
  if (warps != 0)
    decode_rows<D, E4M3, NT, MODS, BULK, true>(p, smem, cc, u0, u1, units, G, warps);
  else
    decode_rows<D, E4M3, NT, MODS, BULK, false>(p, smem, cc, u0, u1, units, G, 0);
}

// Joins the parts of the rows that several CTAs share: block (c, r) the row
// r of the run of query heads that CTA c's units end in, if that CTA has its
// first part.  A tile of parts is read at once, sums and statistics side by
// side, so a join costs about two memory latencies behind its descriptor.
template <int D, bool E4M3, int NT>
__global__ void __launch_bounds__(kJoinThreads)
    join_kernel(const __grid_constant__ DecodeParams p) {
  constexpr int kLanes = D / 4;                      // 16-byte pieces of a part
  constexpr int kGroups = kJoinThreads / kLanes;     // parts side by side
  constexpr int kDepth = kJoinParts / kGroups;               // and one behind the other
  __shared__ float s_m[kJoinParts], s_l[kJoinParts];
  __shared__ float4 s_o[kGroups][kLanes];
  const DecodeArgs& a = p.a;
  ptx::griddep_wait();
  const JoinDesc d = p.desc[blockIdx.x];
  const int r = blockIdx.y;
  if (d.parts == 0) return;
  if (d.head % p.group + r >= p.group) return;
  const int tid = threadIdx.x, col = tid % kLanes, grp = tid / kLanes;
  float top = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  // part i is in CTA c + i: there the first row, but for i = 0
  auto part = [&](int i) {
    const int64_t at = i == 0 ? d.first : 2 * ((int64_t)blockIdx.x + i);
    return p.parts + (at * 8 * NT + r) * (D + 4);
  };
  for (int i0 = 0; i0 < d.parts; i0 += kJoinParts) {
    const int n = min(kJoinParts, d.parts - i0);
    float4 v[kDepth];
#pragma unroll
    for (int k = 0; k < kDepth; ++k) {
      const int i = grp + k * kGroups;
      v[k] = i < n ? *reinterpret_cast<const float4*>(part(i0 + i) + 4 * col)
                   : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (tid < kJoinParts) {
      s_m[tid] = tid < n ? part(i0 + tid)[D] : -INFINITY;
      s_l[tid] = tid < n ? part(i0 + tid)[D + 1] : 0.f;
    }
    __syncthreads();
    // every warp takes the tile's statistics for itself
    const int lane = tid & 31;
    static_assert(kJoinParts == 32, "one part a lane");
    const float ml = s_m[lane];
    float mx = ml;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
    mx = fmaxf(mx, top);
    float sum = s_l[lane] * (ml == mx ? 1.0f : exp2f(ml - mx));
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    const float f = top == mx ? 1.0f : exp2f(top - mx);
    l = l * f + sum;
    acc.x *= f, acc.y *= f, acc.z *= f, acc.w *= f;
    top = mx;
#pragma unroll
    for (int k = 0; k < kDepth; ++k) {
      if (grp + k * kGroups >= n) break;
      const float mi = s_m[grp + k * kGroups];
      const float g = mi == top ? 1.0f : exp2f(mi - top);
      acc.x = fmaf(v[k].x, g, acc.x);
      acc.y = fmaf(v[k].y, g, acc.y);
      acc.z = fmaf(v[k].z, g, acc.z);
      acc.w = fmaf(v[k].w, g, acc.w);
    }
    __syncthreads();  // the statistics have been read
  }
  s_o[grp][col] = acc;
  __syncthreads();
  if (grp > 0) return;
#pragma unroll
  for (int i = 1; i < kGroups; ++i) {
    const float4 y = s_o[i][col];
    acc.x += y.x, acc.y += y.y, acc.z += y.z, acc.w += y.w;
  }
  const float inv = l == 0.f ? 0.f : 1.0f / l;
  const int64_t orow = (int64_t)d.b * a.H + d.head + r;
  *reinterpret_cast<uint2*>(a.out + orow * D + 4 * col) = make_uint2(
      ptx::pack_bf16x2(acc.x * inv, acc.y * inv), ptx::pack_bf16x2(acc.z * inv, acc.w * inv));
  if (a.lse != nullptr && col == 0)
    a.lse[orow] = l == 0.f ? -INFINITY : (top + log2f(l) - (E4M3 ? kHalfShift : 0.f)) * kLn2;
}

template <int D, bool E4M3, int NT, bool MODS, bool BULK>
cudaError_t launch_variant(DecodeParams& p, int dev, cudaStream_t stream) {
  using C = Cfg<D, E4M3, NT>;
  auto kern = decode_kernel<D, E4M3, NT, MODS, BULK>;
  // resident CTAs per device, looked up once
  static std::atomic<int> grid_of[64], warp_grid_of[64];
  int grid = dev < 64 ? grid_of[dev].load(std::memory_order_relaxed) : 0;
  int warp_grid = dev < 64 ? warp_grid_of[dev].load(std::memory_order_relaxed) : 0;
  if (grid == 0 || warp_grid == 0) {
    int sms = 0, per_sm = 0, per_sm_warp = 0;
    cudaError_t err = cudaFuncSetAttribute(
        kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kWarpSmem);
    if (err == cudaSuccess)
      err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (err == cudaSuccess)
      err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kDecThreads, C::kSmem);
    if (err == cudaSuccess)
      err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm_warp, kern, kDecThreads,
                                                          C::kWarpSmem);
    if (err != cudaSuccess) return err;
    if (per_sm < 1 || per_sm_warp < 1) return cudaErrorInvalidConfiguration;
    grid = sms * per_sm;
    warp_grid = sms * per_sm_warp;
    if (grid > decode_max_ctas(NT)) grid = decode_max_ctas(NT);
    if (dev < 64) {
      grid_of[dev].store(grid, std::memory_order_relaxed);
      warp_grid_of[dev].store(warp_grid, std::memory_order_relaxed);
    }
  }
  // The most units a row can have, by the table's width and the window: w keys
  // in a row that begin with a unit's last one reach into (w - 2) / unit + 2.
  const int64_t room = (int64_t)p.a.max_pages * p.a.page_size;
  int64_t most = (room + C::kUnitKeys - 1) / C::kUnitKeys;
  if (p.a.window > 0) {
    const int64_t w = ((int64_t)p.a.window + C::kUnitKeys - 2) / C::kUnitKeys + 1;
    if (most > w) most = w;
  }
  const int64_t rows = (int64_t)p.a.B * p.a.H_kv * p.runs;
  int cs = 8;
  while (cs > 1 && rows * cs > grid) cs /= 2;
  if (cs > 1 && most > 1 && most <= (int64_t)cs * kClusterUnits) {
    p.cluster = cs;
    return launch_overlapped(kern, dim3((unsigned)(rows * cs)), dim3(kDecThreads), C::kSmem,
                             (unsigned)cs, stream, p);
  }
  // Rows short enough for a warp each, the more the more rows there are to
  // keep all warps busy.
  const int64_t keys = p.a.window > 0 && room > p.a.window ? p.a.window : room;
  int steps = 2 * rows < 3 * (int64_t)grid              ? 4
              : NT == 1 && rows < 4 * (int64_t)grid ? kWarpSteps / 2
                                                    : kWarpSteps;
  if (!BULK) steps /= 2;
  if (rows < grid) steps = NT <= 2 ? 1 : 0;
  const int warp_keys = rows < ((int64_t)1 << 30) ? 16 * C::kStep * steps : 0;
  if (keys <= warp_keys) {
    if (warp_grid > rows) warp_grid = (int)rows;
    p.warps = kWarps * warp_grid;
    return launch_overlapped(kern, dim3((unsigned)warp_grid), dim3(kDecThreads), C::kWarpSmem, 0,
                             stream, p);
  }
  if (NT <= 2) p.warp_keys = warp_keys;
  p.whole_rows = most <= kWholeUnits;
  cudaError_t err = launch_overlapped(kern, dim3((unsigned)grid), dim3(kDecThreads), C::kSmem, 0,
                                      stream, p);
  if (err != cudaSuccess || p.whole_rows) return err;
  return launch_overlapped(join_kernel<D, E4M3, NT>,
                           dim3((unsigned)grid, (unsigned)(p.group < 8 * NT ? p.group : 8 * NT)),
                           dim3(kJoinThreads), 0, 0, stream, p);
}

template <int D, bool E4M3, int NT>
cudaError_t launch_tiles(DecodeParams& p, bool bulk, int dev, cudaStream_t stream) {
  if (p.a.score_flags != 0)
    return bulk ? launch_variant<D, E4M3, NT, true, true>(p, dev, stream)
                : launch_variant<D, E4M3, NT, true, false>(p, dev, stream);
  return bulk ? launch_variant<D, E4M3, NT, false, true>(p, dev, stream)
              : launch_variant<D, E4M3, NT, false, false>(p, dev, stream);
}
template <int D, bool E4M3>
cudaError_t launch_group(DecodeParams& p, bool bulk, int dev, cudaStream_t stream) {
  switch (decode_tiles(p.group)) {
    case 1:
      return launch_tiles<D, E4M3, 1>(p, bulk, dev, stream);
    case 2:
      return launch_tiles<D, E4M3, 2>(p, bulk, dev, stream);
    default:
      return launch_tiles<D, E4M3, 4>(p, bulk, dev, stream);
  }
}

}  // namespace

// bulk: copies by TMA boxes (p.k_map and p.v_map are set).
template <bool E4M3>
cudaError_t launch_decode_cache(DecodeParams& p, bool bulk, int dev, cudaStream_t stream) {
  return p.a.D == 128 ? launch_group<128, E4M3>(p, bulk, dev, stream)
                      : launch_group<64, E4M3>(p, bulk, dev, stream);
}

}  // namespace attn
