// Attention of the hybrid model's full-attention layers: over whole prompts, and over the paged
// cache for one token or a tree of drafted tokens per request.
//   o_i = sum_j w_ij v_j,  w_ij = softmax over the visible j of scale q_i . k_j;  no visible j: 0.
// The kernels are in tb_attn_prompt.cu and tb_attn_tree.cu; here are the entry points' checks.
#include <cuda_runtime.h>
#include <math.h>

#include "tb_attention.cuh"
#include "tb_common.cuh"
#include "tb_host.h"

namespace tb {

constexpr int64_t kMaxLd = 1ll << 31;  // a tensor map's strides are below 2^40 bytes

}  // namespace tb

extern "C" int tb_prompt_attention(const uint16_t* q, int64_t ldq, const uint16_t* k, int64_t ldk, const uint16_t* v,
                                   int64_t ldv, int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hkv, int64_t D,
                                   const int32_t* q_start, const int32_t* k_start, int64_t B, float scale, uint16_t* o,
                                   int32_t* dev_status, void* stream) {
  using namespace tb;
  if (Tq < 0 || Tq > INT32_MAX || Tk < 0 || Tk > INT32_MAX || B < 1 || B > INT32_MAX || Hkv < 1 || Hq < Hkv ||
      Hq > 1024 || Hq % Hkv)
    return TB_ERR_SHAPE;
  if (!supported_head(D)) return TB_ERR_UNSUPPORTED;
  if (ldq < Hq * D || ldk < Hkv * D || ldv < Hkv * D || ldq % 8 || ldk % 8 || ldv % 8 || ldq > kMaxLd || ldk > kMaxLd ||
      ldv > kMaxLd)
    return TB_ERR_SHAPE;
  if (!(scale > 0.f && scale < INFINITY)) return TB_ERR_VALUE;
  if (Tq == 0) return TB_OK;
  if (!q || !o || !q_start || !k_start || (Tk && (!k || !v))) return TB_ERR_NULL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned_to(q_start, 4) || !aligned_to(k_start, 4))
    return TB_ERR_ALIGN;
  AttnArgs a = {};
  a.q = reinterpret_cast<const __half*>(q);
  a.k = reinterpret_cast<const __half*>(k);
  a.v = reinterpret_cast<const __half*>(v);
  a.q_start = q_start;
  a.k_start = k_start;
  a.o = reinterpret_cast<__half*>(o);
  a.status = dev_status;
  a.ldq = ldq;
  a.ldk = ldk;
  a.ldv = ldv;
  a.T = Tq;
  a.Tk = Tk;
  a.B = (int)B;
  a.Hq = (int)Hq;
  a.Hkv = (int)Hkv;
  a.scale_log2 = scale * kLog2e;
  return launch_prompt_tiles(a, D, static_cast<cudaStream_t>(stream));
}

extern "C" size_t tb_tree_attention_workspace_size(int64_t B, int64_t T, int64_t max_q, int64_t Hq, int64_t Hkv,
                                                   int64_t D) {
  using namespace tb;
  (void)T;
  if (B < 1 || max_q < 1 || max_q > 64 || Hkv < 1 || Hq < Hkv || Hq % Hkv || !supported_head(D)) return 0;
  return tree_workspace(B, max_q, Hq, Hkv, D);
}

extern "C" int tb_tree_attention(const uint16_t* q, int64_t ldq, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                                 const uint16_t* k_cache, const uint16_t* v_cache, int64_t pages, int64_t page,
                                 const int32_t* table, int64_t max_pages, const int32_t* total,
                                 const int32_t* row_start, int64_t B, int64_t max_q, const uint64_t* tree, float scale,
                                 uint16_t* o, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                 void* stream) {
  using namespace tb;
  if (T < 0 || T > INT32_MAX || B < 1 || B > INT32_MAX || Hkv < 1 || Hq < Hkv || Hq > 1024 || Hq % Hkv || pages < 1 ||
      pages > INT32_MAX || max_pages < 1 || max_pages > INT32_MAX || max_q < 1)
    return TB_ERR_SHAPE;
  if (!supported_head(D) || !supported_page(page)) return TB_ERR_UNSUPPORTED;
  if (ldq < Hq * D || ldq % 8 || ldq > kMaxLd) return TB_ERR_SHAPE;
  // the schedule counts tiles of work, of 128 keys of a request's longest context, in 32 bits
  if (max_q > 64 || pages * Hkv > INT32_MAX || T * Hq > INT32_MAX ||
      (double)tree_items(B, max_q, Hq, Hkv) * ((double)max_pages * (double)page / 128 + 1) > INT32_MAX)
    return TB_ERR_TOO_LARGE;
  if (!(scale > 0.f && scale < INFINITY)) return TB_ERR_VALUE;
  if (T == 0) return TB_OK;
  if (!q || !k_cache || !v_cache || !table || !total || !row_start || !o) return TB_ERR_NULL;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned_to(table, 4) || !aligned_to(total, 4) ||
      !aligned_to(row_start, 4) || !aligned_to(tree, 8) || !aligned16(o) || !aligned16(workspace))
    return TB_ERR_ALIGN;
  if (!workspace || workspace_bytes < tb_tree_attention_workspace_size(B, T, max_q, Hq, Hkv, D)) return TB_ERR_WORKSPACE;
  AttnArgs a = {};
  a.q = reinterpret_cast<const __half*>(q);
  a.k = reinterpret_cast<const __half*>(k_cache);
  a.v = reinterpret_cast<const __half*>(v_cache);
  a.q_start = row_start;
  a.table = table;
  a.total = total;
  a.tree = reinterpret_cast<const int64_t*>(tree);
  a.o = reinterpret_cast<__half*>(o);
  a.status = dev_status;
  a.ldq = ldq;
  a.T = T;
  a.pages = pages;
  a.max_pages = max_pages;
  a.B = (int)B;
  a.Hq = (int)Hq;
  a.Hkv = (int)Hkv;
  a.page_log2 = log2_of(page);
  a.max_q = (int)max_q;
  a.scale_log2 = scale * kLog2e;
  return launch_tree_tiles(a, D, workspace, static_cast<cudaStream_t>(stream));
}
