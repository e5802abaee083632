// attn_decode_bf16.cu -- the one-token attention over bf16 caches, and the
// launcher of both cache types.
#include <atomic>

#include "attn_decode_sm103.cuh"

namespace attn {

cudaError_t launch_decode_e4m3(DecodeParams& p, bool bulk, int dev, cudaStream_t stream);

namespace {

cudaError_t launch_decode_bf16(DecodeParams& p, bool bulk, int dev, cudaStream_t stream) {
  return launch_decode_cache<false>(p, bulk, dev, stream);
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled() {
  static std::atomic<EncodeTiledFn> fn{nullptr};
  EncodeTiledFn f = fn.load(std::memory_order_relaxed);
  if (f == nullptr) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      f = reinterpret_cast<EncodeTiledFn>(ptr);
    fn.store(f, std::memory_order_relaxed);
  }
  return f;
}

// Keys or values as (up to 128 bytes of a row, half of the row, row of a page,
// kv head, page); boxes of 16 rows.  False where the strides are beyond what a
// map can hold.
bool make_cache_map(CUtensorMap* map, const void* ptr, const int64_t* strides, const DecodeArgs& a,
                    int elem) {
  EncodeTiledFn enc = encode_tiled();
  if (enc == nullptr) return false;
  const int row = a.D * elem, line = row > 128 ? 128 : row;
  const cuuint64_t dims[5] = {(cuuint64_t)(line / elem), (cuuint64_t)(row / line),
                              (cuuint64_t)a.page_size, (cuuint64_t)a.H_kv,
                              (cuuint64_t)a.num_pages};
  cuuint64_t st[4] = {(cuuint64_t)line, (cuuint64_t)strides[2] * elem,
                      (cuuint64_t)strides[1] * elem, (cuuint64_t)strides[0] * elem};
  for (int i = 1; i < 4; ++i)
    if (dims[i + 1] == 1) st[i] = (cuuint64_t)row;  // never stepped
  const cuuint32_t box[5] = {(cuuint32_t)dims[0], (cuuint32_t)dims[1], 16, 1, 1};
  const cuuint32_t one[5] = {1, 1, 1, 1, 1};
  return enc(map, elem == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 5,
             const_cast<void*>(ptr), dims, st, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             line == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

size_t decode_workspace_bytes(int H, int H_kv, int D) {
  const int tiles = decode_tiles(H / H_kv);
  return decode_desc_bytes(tiles) + sizeof(float) * 2 * (size_t)decode_max_ctas(tiles) * 8 *
                                        (size_t)tiles * (size_t)(D + 4);
}

cudaError_t launch_decode(const DecodeArgs& a, bool e4m3, cudaStream_t stream) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  DecodeParams p;
  p.a = a;
  // key / page_size by a product: mul = ceil(2^shift / page_size), shift =
  // 30 + ceil(log2 page_size); the excess is below 2^shift / 2^30
  int lg = 0;
  while ((1u << lg) < (uint32_t)a.page_size) ++lg;
  p.page_shift = 30u + (uint32_t)lg;
  p.page_mul = (uint32_t)(((1ull << p.page_shift) + (uint64_t)a.page_size - 1) /
                          (uint64_t)a.page_size);
  p.group = a.H / a.H_kv;
  const int tiles = decode_tiles(p.group), rows = 8 * tiles;
  p.runs = (p.group + rows - 1) / rows;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  // the scores come in units of log2, tanh takes s / cap; a cap at either end
  // of fp32 counts as the nearest whose product and quotient are finite
  const float cap = fminf(fmaxf(a.softcap, FLT_MIN), 0x1p127f);
  p.cap = cap * 1.4426950408889634f;
  p.inv_cap = 0.6931471805599453f / cap;
  p.desc = static_cast<JoinDesc*>(a.workspace);
  p.parts = reinterpret_cast<float*>(static_cast<char*>(a.workspace) +
                                     decode_desc_bytes(tiles));
  p.budget_ns = (uint64_t)(a.wait_budget_ms * 1.0e6);
  p.debug_stall = a.debug_stall;
  p.cluster = 0;
  p.whole_rows = 0;
  p.warps = p.warp_keys = 0;
  const int elem = e4m3 ? 1 : 2;
  const bool bulk = a.page_size % 16 == 0 && make_cache_map(&p.k_map, a.kc, a.kcs, a, elem) &&
                    make_cache_map(&p.v_map, a.vc, a.vcs, a, elem);
  return e4m3 ? launch_decode_e4m3(p, bulk, dev, stream)
              : launch_decode_bf16(p, bulk, dev, stream);
}

}  // namespace attn
