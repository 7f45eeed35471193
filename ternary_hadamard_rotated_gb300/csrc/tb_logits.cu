// Changes to the logits before a token is chosen: penalties for tokens that a request's history holds, biases,
// and grammar masks.
//
// Per row and token, in this order, in fp32 with every step rounded as written (no product joined to a sum, so
// that the same formulas give the same bits anywhere):
//   l <- l > 0 ? l / repetition : l * repetition   if the token is in the history (or among the row's drafts)
//   l <- l - frequency * count - presence          if it was generated, count times
//   l <- l + bias                                  if it has one
//   l <- -infinity                                 if its bit of the mask is 0
#include <cuda_runtime.h>
#include <limits.h>

#include "tb_common.cuh"
#include "tb_host.h"

namespace tb {

struct LogitsArgs {
  const __half* in;
  void* out;
  const int32_t *row_start, *history, *slot, *hist_len, *prompt_len, *fresh;
  const unsigned long long* tree;
  const float *repetition, *presence, *frequency;
  const int32_t *bias_start, *bias_ids;
  const float* bias_values;
  const uint32_t* mask;
  const int32_t* mask_row;
  int32_t* status;
  int64_t ld, ldo, ldh, n_hist, n_bias, mask_rows;
  int T, V, B;
  int span;  // tokens of the vocabulary a CTA takes, a multiple of 32
};

constexpr int kLogitsThreads = 512;
constexpr uint32_t kPromptBit = 0x80000000u;  // of a token's count: in the prompt

template <typename Out>
__global__ void __launch_bounds__(kLogitsThreads) logits_kernel(const LogitsArgs a) {
  extern __shared__ __align__(16) uint32_t logits_smem[];
  uint32_t* count = logits_smem;           // [span] times generated, and kPromptBit
  uint32_t* bias = logits_smem + a.span;   // [span] number of the token's bias in the lists + 1
  const int tid = threadIdx.x, t = blockIdx.y, v0 = blockIdx.x * a.span;
  const int width = min(a.span, a.V - v0);
  int b = t, first = t, fresh = 1;  // the row's request, its first row and its rows
  if (a.row_start) {
    if (blockIdx.x == 0 && t == 0)
      for (int i = tid; i < a.B; i += kLogitsThreads)
        if (__ldg(a.row_start + i) < 0 || __ldg(a.row_start + i + 1) < __ldg(a.row_start + i) || __ldg(a.row_start + i + 1) > a.T)
          set_status(a.status, TB_DEV_BAD_LEN);
    int lo = 0, hi = a.B - 1;
    while (lo < hi) {  // the last request that begins at or before row t
      const int mid = (lo + hi + 1) >> 1;
      if (__ldg(a.row_start + mid) <= t) lo = mid;
      else hi = mid - 1;
    }
    b = lo;
    first = __ldg(a.row_start + b);
    const int end = __ldg(a.row_start + b + 1);
    if (first < 0 || t < first || t >= end || end > a.T) return;  // a row of no request
    fresh = end - first;
  }
  int bad = 0;
  for (int i = tid; i < width; i += kLogitsThreads) count[i] = 0;
  if (a.bias_ids)
    for (int i = tid; i < width; i += kLogitsThreads) bias[i] = 0;
  __syncthreads();
  // the history
  const int64_t row = a.slot ? __ldg(a.slot + b) : b;
  int len = __ldg(a.hist_len + b);
  const int prompt = a.prompt_len ? __ldg(a.prompt_len + b) : 0;
  if (row >= a.n_hist) bad |= TB_DEV_BAD_ID;
  if (len < 0 || len > a.ldh || prompt < 0 || prompt > len) bad |= TB_DEV_BAD_LEN;
  if (row < 0 || row >= a.n_hist || len < 0) len = 0;
  if (len > a.ldh) len = (int)a.ldh;
  for (int i = tid; i < len; i += kLogitsThreads) {
    const int id = __ldg(a.history + row * a.ldh + i);
    if (id >= a.V) bad |= TB_DEV_BAD_ID;
    const unsigned at = (unsigned)(id - v0);
    if (id < 0 || at >= (unsigned)width) continue;
    if (i < prompt) atomicOr(count + at, kPromptBit);
    else atomicAdd(count + at, 1u);
  }
  // the row's own path of drafted tokens
  if (a.fresh) {
    if (fresh > 64) bad |= TB_DEV_BAD_LEN;
    const unsigned long long path = a.tree ? a.tree[t] : t - first < 63 ? (2ull << (t - first)) - 1 : ~0ull;
    if (tid < 64 && tid < fresh && (path >> tid & 1)) {
      const int id = __ldg(a.fresh + first + tid);
      if (id >= a.V) bad |= TB_DEV_BAD_ID;
      const unsigned at = (unsigned)(id - v0);
      if (id >= 0 && at < (unsigned)width) atomicAdd(count + at, 1u);
    }
  }
  if (a.bias_ids) {
    int s = __ldg(a.bias_start + b), e = __ldg(a.bias_start + b + 1);
    if (s < 0 || e < s || e > a.n_bias) {
      bad |= TB_DEV_BAD_LEN;
      s = e = 0;
    }
    for (int i = s + tid; i < e; i += kLogitsThreads) {
      const int id = __ldg(a.bias_ids + i);
      if (id >= a.V) bad |= TB_DEV_BAD_ID;
      const unsigned at = (unsigned)(id - v0);
      if (id >= 0 && at < (unsigned)width) atomicMax(bias + at, (uint32_t)i + 1);  // the last of a token's biases
    }
  }
  const uint32_t* mask = nullptr;
  if (a.mask) {
    const int64_t m = a.mask_row ? __ldg(a.mask_row + t) : t;
    if (m >= a.mask_rows) bad |= TB_DEV_BAD_ID;
    else if (m >= 0) mask = a.mask + m * ((a.V + 31) / 32) + v0 / 32;
  }
  if (bad) set_status(a.status, bad);
  __syncthreads();
  const float rho = a.repetition ? __ldg(a.repetition + b) : 1.f;
  const float presence = a.presence ? __ldg(a.presence + b) : 0.f, frequency = a.frequency ? __ldg(a.frequency + b) : 0.f;
  const __half* in = a.in + t * a.ld + v0;
  Out* out = static_cast<Out*>(a.out) + t * a.ldo + v0;
  for (int i = tid; i < width; i += kLogitsThreads) {
    float l = __half2float(in[i]);
    const uint32_t c = count[i];
    if (c) {
      l = l > 0.f ? __fdiv_rn(l, rho) : __fmul_rn(l, rho);
      const uint32_t n = c & ~kPromptBit;
      if (n) l = __fsub_rn(__fsub_rn(l, __fmul_rn(frequency, (float)n)), presence);
    }
    if (a.bias_ids && bias[i]) l = __fadd_rn(l, __ldg(a.bias_values + bias[i] - 1));
    if (mask && !(mask[i / 32] >> (i & 31) & 1)) l = -INFINITY;
    out[i] = (Out)l;
  }
}

}  // namespace tb

extern "C" int tb_logits_adjust(const uint16_t* logits, int64_t ld, int64_t T, int64_t V, const int32_t* row_start, int64_t B,
                                const int32_t* history, int64_t n_hist, int64_t ldh, const int32_t* slot, const int32_t* hist_len,
                                const int32_t* prompt_len, const int32_t* fresh, const uint64_t* tree, const float* repetition,
                                const float* presence, const float* frequency, const int32_t* bias_start, const int32_t* bias_ids,
                                const float* bias_values, int64_t n_bias, const uint32_t* mask, int64_t mask_rows,
                                const int32_t* mask_row, void* out, int64_t ldo, int out_type, int32_t* dev_status, void* stream) {
  using namespace tb;
  if (T < 0 || T > INT_MAX || V < 1 || V > (1 << 24) || ld < V || ldo < V || B < 1 || n_hist < 1 || ldh < 0 || n_bias < 0 ||
      n_bias >= INT_MAX || mask_rows < 0)
    return TB_ERR_SHAPE;
  if (!row_start && B != T) return TB_ERR_SHAPE;  // row t is request t's
  if (!slot && n_hist < B) return TB_ERR_SHAPE;
  if (mask && !mask_row && mask_rows < T) return TB_ERR_SHAPE;
  if (out_type != TB_OUT_F16 && out_type != TB_OUT_F32) return TB_ERR_UNSUPPORTED;
  if (T > 65535 || B > 65535) return TB_ERR_TOO_LARGE;
  if (T == 0) return TB_OK;
  if (!logits || !out || !hist_len || (ldh && !history) || (n_bias && (!bias_start || !bias_ids || !bias_values)) || (tree && !fresh))
    return TB_ERR_NULL;
  if (!aligned16(logits) || !aligned16(out) || !aligned_to(row_start, 4) || !aligned_to(history, 4) || !aligned_to(slot, 4) ||
      !aligned_to(hist_len, 4) || !aligned_to(prompt_len, 4) || !aligned_to(fresh, 4) || !aligned_to(tree, 8) ||
      !aligned_to(repetition, 4) || !aligned_to(presence, 4) || !aligned_to(frequency, 4) || !aligned_to(bias_start, 4) ||
      !aligned_to(bias_ids, 4) || !aligned_to(bias_values, 4) || !aligned_to(mask, 4) || !aligned_to(mask_row, 4))
    return TB_ERR_ALIGN;
  if (out == logits && (out_type != TB_OUT_F16 || (ldo != ld && T > 1))) return TB_ERR_SHAPE;  // in place only element for element
  DeviceFacts f;
  int rc = device_facts(&f);
  if (rc != TB_OK) return rc;
  LogitsArgs a = {};
  a.in = reinterpret_cast<const __half*>(logits);
  a.out = out;
  a.row_start = row_start;
  a.history = history;
  a.slot = slot;
  a.hist_len = hist_len;
  a.prompt_len = prompt_len;
  a.fresh = fresh;
  a.tree = reinterpret_cast<const unsigned long long*>(tree);
  a.repetition = repetition;
  a.presence = presence;
  a.frequency = frequency;
  a.bias_start = bias_start;
  a.bias_ids = n_bias ? bias_ids : nullptr;
  a.bias_values = bias_values;
  a.mask = mask;
  a.mask_row = mask_row;
  a.status = dev_status;
  a.ld = ld;
  a.ldo = ldo;
  a.ldh = ldh;
  a.n_hist = n_hist;
  a.n_bias = n_bias;
  a.mask_rows = mask_rows;
  a.T = (int)T;
  a.V = (int)V;
  a.B = (int)B;
  a.span = 8192;
  const int smem = a.span * 8;
  const dim3 grid((unsigned)((V + a.span - 1) / a.span), (unsigned)T);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const void* fn = out_type == TB_OUT_F16 ? reinterpret_cast<const void*>(logits_kernel<__half>) : reinterpret_cast<const void*>(logits_kernel<float>);
  rc = ensure_dynamic_smem(fn, f.device, smem);
  if (rc != TB_OK) return rc;
  if (out_type == TB_OUT_F16)
    logits_kernel<__half><<<grid, kLogitsThreads, smem, s>>>(a);
  else
    logits_kernel<float><<<grid, kLogitsThreads, smem, s>>>(a);
  return check_launch();
}
