// What the attention kernels share: the arguments, and one row by one warp.
#pragma once

#include <cuda.h>
#include <math.h>

#include "tb_common.cuh"

namespace tb {

constexpr float kLog2e = 1.4426950408889634f;

struct AttnArgs {
  const __half* q;
  const __half* k;
  const __half* v;
  const int32_t* q_start;
  const int32_t* k_start;  // prompt form
  const int32_t* table;    // paged form
  const int32_t* total;
  const int64_t* tree;
  __half* o;
  int32_t* status;
  int64_t ldq, ldk, ldv, T, Tk, pages, max_pages;
  int B, Hq, Hkv, page_log2, max_q;
  float scale_log2;
};

// o of row t, query head h, from keys [0, end) of request b, by one warp: the lanes share the head's
// elements, one key at a time, with the softmax's running maximum and sum, so every key and value is
// read once.  k0: the request's first key row (packed form); from `prefix` on only keys whose bit
// is set in `word` count (paged form).  Only keys the row sees are read.
template <int D, bool PAGED>
TB_DEVI void attend_row(const AttnArgs& a, int64_t t, int h, int64_t b, int64_t k0, int64_t end, int64_t prefix,
                        uint64_t word, int lane) {
  constexpr int E = D / 32;  // elements per lane
  const int hk = h / (a.Hq / a.Hkv);
  float q[E], acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __half2float(a.q[t * a.ldq + h * D + e * 32 + lane]) * a.scale_log2;
    acc[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int64_t j = 0; j < end; ++j) {
    if (PAGED && j >= prefix && !((word >> (j - prefix)) & 1)) continue;
    int64_t at_k, at_v;
    if (PAGED) {
      const int64_t pg = __ldg(a.table + b * a.max_pages + (j >> a.page_log2));
      if (pg < 0 || pg >= a.pages) {
        if (lane == 0) set_status(a.status, TB_DEV_BAD_SLOT);
        continue;
      }
      at_k = at_v = (((pg * a.Hkv + hk) << a.page_log2) + (j & ((1ll << a.page_log2) - 1))) * D;
    } else {
      at_k = (k0 + j) * a.ldk + hk * D;
      at_v = (k0 + j) * a.ldv + hk * D;
    }
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(q[e], __half2float(a.k[at_k + e * 32 + lane]), s);
#pragma unroll
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    const float m2 = fmaxf(m, s);
    if (m2 == -INFINITY && s == -INFINITY) continue;  // a weight of zero
    const float c = exp2f(m - m2), w = exp2f(s - m2);
    l = l * c + w;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = fmaf(w, __half2float(a.v[at_v + e * 32 + lane]), acc[e] * c);
    m = m2;
  }
  const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) a.o[(t * a.Hq + h) * D + e * 32 + lane] = __float2half_rn(acc[e] * inv);
}

// query heads of one KV head in a tile of 128 rows: the largest divisor of the group that leaves at
// most 8 rows unused (a group that is a prime above 128 falls back to one head per tile)
inline int heads_per_tile(int group) {
  int best = 1;
  for (int d = 1; d <= group && d <= 128; ++d)
    if (group % d == 0 && 128 / d * d >= 120) best = d;
  return best;
}

// tensor map of fp16 [tokens, heads, D] with `ld` elements between tokens; box 64 x heads x tokens
int token_map(CUtensorMap* m, const __half* p, int64_t tokens, int64_t heads, int64_t D, int64_t ld, int box_heads,
              int box_tokens);

// prompt form on the tensor cores
int launch_prompt_tiles(const AttnArgs& a, int64_t D, cudaStream_t s);

// paged form on the tensor cores; its items of work at most, and its workspace
int launch_tree_tiles(const AttnArgs& a, int64_t D, void* workspace, cudaStream_t s);
int64_t tree_items(int64_t B, int64_t max_q, int64_t Hq, int64_t Hkv);
size_t tree_workspace(int64_t B, int64_t max_q, int64_t Hq, int64_t Hkv, int64_t D);

}  // namespace tb
