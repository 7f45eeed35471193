// What the attention kernels share: the arguments, and a row's keys by one warp.
#pragma once

#include <cuda.h>
#include <math.h>

#include "tb_common.cuh"

namespace tb {

constexpr float kLog2e = 1.4426950408889634f;
// A weight is 2^7 at the maximum that it refers to, and as that may be 2^8 too small, 2^15 at most: fp16's top.  So
// weights of a 2^21st of the largest keep all of fp16's bits as the operand of P V, and what is rounded off those
// below is under 2^-32 of it (with 1 at the maximum, weights below 2^-25 were in the sum but not in the output).
constexpr float kPTop = 7.f;

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

// lane's E consecutive fp16 elements of a row: their bits, and as fp32
template <int E>
TB_DEVI void load_bits(const __half* p, int lane, uint32_t (&w)[E / 2]) {
  if constexpr (E == 8) {
    const uint4 y = __ldcg(reinterpret_cast<const uint4*>(p) + lane);
    w[0] = y.x, w[1] = y.y, w[2] = y.z, w[3] = y.w;
  } else if constexpr (E == 4) {
    const uint2 y = __ldcg(reinterpret_cast<const uint2*>(p) + lane);
    w[0] = y.x, w[1] = y.y;
  } else {
    w[0] = __ldcg(reinterpret_cast<const uint32_t*>(p) + lane);
  }
}
template <int E>
TB_DEVI void load_row(const __half* p, int lane, float (&x)[E]) {
  uint32_t w[E / 2];
  load_bits<E>(p, lane, w);
#pragma unroll
  for (int e = 0; e < E / 2; ++e) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[e]));
    x[2 * e] = f.x;
    x[2 * e + 1] = f.y;
  }
}
// Output bits of a row whose sum of weights is not finite: a score it sees is NaN or infinite, so that NaN is what
// it comes to.  Conversions to fp16 give the other sign, which is how such rows are told from those that zero times
// a value they do not see has made NaN.
constexpr uint32_t kNanRow = 0xffffu;
TB_DEVI bool not_finite_h(uint32_t h) { return (h & 0x7c00u) == 0x7c00u; }
template <int N>
TB_DEVI bool any_to_mend(const uint32_t (&w)[N]) {  // among these pairs
  bool odd = false;
#pragma unroll
  for (int e = 0; e < N; ++e)
    odd |= (not_finite_h(w[e]) && (w[e] & 0xffffu) != kNanRow) || (not_finite_h(w[e] >> 16) && w[e] >> 16 != kNanRow);
  return odd;
}

// A row whose output came out not finite, again, from the keys that it sees alone: what the tensor cores add up
// has zero times what a row does not see in it.  One warp takes the keys j0, j0 + step, .. below `end` of row t,
// query head h, of request b, four at a time (the loads of four rows of K, then of V, are under way together), with
// the softmax's running maximum m (log2 units) and sum l; acc: o's elements E lane .. before the division.  k0: the
// request's first key row (packed form); from `prefix` on only keys whose bit is set in `word` count (paged form).
// Nothing may wait for this under a limit: it takes as long as the row has keys.
template <int D, bool PAGED>
TB_DEVI void attend_keys(const AttnArgs& a, int64_t t, int h, int64_t b, int64_t k0, int64_t j0, int64_t step, int64_t end,
                         int64_t prefix, uint64_t word, int lane, float& m, float& l, float (&acc)[D / 32]) {
  constexpr int E = D / 32, N = 4;
  const int hk = h / (a.Hq / a.Hkv);
  float q[E];
  load_row<E>(a.q + t * a.ldq + h * D, lane, q);
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] *= a.scale_log2;
    acc[e] = 0.f;
  }
  m = -INFINITY;
  l = 0.f;
  for (int64_t j = j0; j < end; j += N * step) {
    int64_t at_v[N];
    bool on[N];
    float s[N], x[N][E];
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const int64_t i = j + u * step;
      on[u] = i < end;
      int64_t at_k = 0;
      at_v[u] = 0;
      if (PAGED) {
        on[u] = on[u] && (i < prefix || ((word >> (i - prefix)) & 1));
        const int64_t pg = on[u] ? __ldg(a.table + b * a.max_pages + (i >> a.page_log2)) : -1;
        on[u] = pg >= 0 && pg < a.pages;
        if (on[u]) at_k = at_v[u] = (((pg * a.Hkv + hk) << a.page_log2) + (i & ((1ll << a.page_log2) - 1))) * D;
      } else if (on[u]) {
        at_k = (k0 + i) * a.ldk + hk * D;
        at_v[u] = (k0 + i) * a.ldv + hk * D;
      }
      if (on[u]) load_row<E>(a.k + at_k, lane, x[u]);
      else
#pragma unroll
        for (int e = 0; e < E; ++e) x[u][e] = 0.f;
    }
#pragma unroll
    for (int u = 0; u < N; ++u) {
      s[u] = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) s[u] = fmaf(q[e], x[u][e], s[u]);
    }
#pragma unroll
    for (int d = 16; d; d >>= 1)
#pragma unroll
      for (int u = 0; u < N; ++u) s[u] += __shfl_xor_sync(0xffffffffu, s[u], d);
    float m2 = m;
#pragma unroll
    for (int u = 0; u < N; ++u) {
      if (!on[u]) s[u] = -INFINITY;
      m2 = fmaxf(m2, s[u]);  // (passes over NaN, which the sum takes up)
    }
    const float c = m == m2 ? 1.f : exp2f(m - m2);
    m = m2;
    l *= c;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= c;
#pragma unroll
    for (int u = 0; u < N; ++u)
      if (on[u]) load_row<E>(a.v + at_v[u], lane, x[u]);  // (of a key that is not there, K's zeros)
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const float w = s[u] == -INFINITY ? 0.f : exp2f(s[u] - m);
      l += w;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(w, x[u][e], acc[e]);
    }
  }
}

// what a sum of weights divides by
TB_DEVI float inverse_sum(float l) { return l < INFINITY ? (l > 0.f ? 1.f / l : 0.f) : NAN; }

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
