// generation_internal.h -- parameters shared by the host side and the kernels of
// the generation entry points (not part of the public ABI).
#pragma once

#include <cuda_bf16.h>

#include "attn_internal.h"

namespace attn {

// Launches a kernel that may start while the one before it in the stream ends:
// it waits for that one (griddep_wait) before it touches global memory.  The
// short kernels let the next one start early in turn, so a step's chain of
// them does not pay each launch's latency (a captured step of 4 layers, one
// request: 41 us, 43 without; rope of 268 MB after itself: 50.3 us, 52.3
// without).  cluster: CTAs of a cluster, 0 for none.
template <typename... Params, typename... Args>
cudaError_t launch_overlapped(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem,
                              unsigned cluster, cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 0 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Args&&>(args)...);
}

// The current device's status word.
attn_status device_status_word(DeviceStatus** out);
// The options that bound the kernels' waits.
void wait_options(double* wait_budget_ms, int* debug_stall);
// A caller's descriptor in the current layout, its flags and fields checked
// for a problem of one query and one key (doc_ids' S_q == S_k holds there).
attn_status load_checked_mod(const attn_mod_desc* in, attn_mod_desc* out);

// Where a device check of these kernels failed (DeviceStatus::where).
enum GenerationSite : int32_t {
  kSiteSlot = 201,     // attn_cache_append: slot beyond the cache
  kSiteSlotMap = 202,  // attn_cache_slots: step that cannot be served
  kSitePage = 203,     // attn_cache_slots: page id outside the cache
  kSiteSeqLen = 204,   // attn_decode: length outside the table
  kSiteTable = 205,    // attn_decode: page id outside the cache
  kSiteWait = 206      // attn_decode: a copy did not come in time
};

struct RopeArgs {
  const __nv_bfloat16* x;
  __nv_bfloat16* out;
  int64_t xs[3], os[3];  // batch, head, token strides
  int B, H, S, D;
  const int32_t* positions;
  int64_t pos_stride;
  int32_t offset;
  float sign;            // -1: backwards
  int heads_per_block;  // set by the launcher
  attn_rope_plan plan;
};
// width: elements of an access, 8, 4, 2 or 1 (alignment checked by the caller)
cudaError_t launch_rope(const RopeArgs& a, int width, cudaStream_t stream);

struct AppendArgs {
  const __nv_bfloat16 *q, *k, *v;
  __nv_bfloat16* q_out;
  void *kc, *vc;
  int64_t qs[2], ks[2], vs[2], qos[2];  // token, head strides
  int64_t kcs[3], vcs[3];               // page, head, token strides
  int T, H, H_kv, D;
  int num_pages, page_size;
  const int32_t* positions;
  const int64_t* slots;
  const float *k_scale, *v_scale;
  DeviceStatus* status;
  int rotate;
  int heads_per_block;  // set by the launcher
  attn_rope_plan plan;
};
cudaError_t launch_append(const AppendArgs& a, int width, bool e4m3, cudaStream_t stream);

struct SlotArgs {
  const int32_t *ctx_lens, *new_lens;
  int B, page_size, num_pages;
  int32_t* table;
  int64_t table_stride;
  int max_pages;
  const int32_t* free_pages;
  int free_cap;
  const int32_t* n_free;
  int32_t *seq_lens, *cu_new, *token_req, *positions;
  int64_t* slots;
  int32_t* n_free_out;
  int max_tokens;
  DeviceStatus* status;
  int in_place;  // set by the launcher: an output is its input
};
cudaError_t launch_slots(const SlotArgs& a, cudaStream_t stream);

struct DecodeArgs {
  const __nv_bfloat16* q;
  int64_t qs[2];  // batch, head strides
  const void *kc, *vc;
  int64_t kcs[3], vcs[3];  // page, head, token strides (elements)
  int num_pages, page_size;
  const int32_t* table;
  int64_t table_stride;
  int max_pages;
  const int32_t* seq_lens;
  const float *k_scale, *v_scale;
  __nv_bfloat16* out;
  float* lse;
  int B, H, H_kv, D;
  float scale;
  int window;  // 0: none
  uint32_t score_flags;
  float softcap;
  const float* alibi_slopes;
  const float* rel_bias;
  int rel_max;
  void* workspace;
  DeviceStatus* status;
  double wait_budget_ms;
  int debug_stall;  // test hook: warps wait for a copy that never comes
};
cudaError_t launch_decode(const DecodeArgs& a, bool e4m3, cudaStream_t stream);
size_t decode_workspace_bytes(int H, int H_kv, int D);

}  // namespace attn
