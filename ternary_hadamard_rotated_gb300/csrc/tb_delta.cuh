// What the kernels of the gated delta rule share.
#pragma once

#include "tb_common.cuh"

namespace tb {

constexpr int kDeltaD = 128;           // head width of q, k and v
constexpr float kDeltaEps = 1e-6f;     // under the root of the 2-norms of q and k

struct DeltaArgs {
  const __half* q;  // [T, Hk, 128], rows ldq apart
  const __half* k;
  const __half* v;  // [T, Hv, 128]
  const float* g;   // [T, Hv]
  const float* beta;
  const int32_t* row_start;  // [B + 1]
  const float* state_in;     // [n_in, Hv, 128 (k), 128 (v)] or null (zeros)
  float* state_out;          // or null
  const int32_t* slot_in;    // [B] or null (b)
  const int32_t* slot_out;
  __half* o;  // [T, Hv, 128]
  int32_t* status;
  int64_t ldq, ldk, ldv, n_in, n_out, T;
  int B, Hk, Hv, normalise;
  float scale;
};

// rows [t0, t0 + n) of request b; false where row_start does not lie in order inside [0, T]
TB_DEVI bool delta_rows(const DeltaArgs& a, int b, int64_t& t0, int64_t& n) {
  const int64_t x = __ldg(a.row_start + b), y = __ldg(a.row_start + b + 1);
  t0 = x;
  n = y - x;
  return x >= 0 && y >= x && y <= a.T;
}

// row of the state pool for request b; -1 (no state) for a negative or outlying index
TB_DEVI int64_t delta_slot(const int32_t* slots, int b, int64_t n, int32_t* status) {
  const int64_t s = slots ? __ldg(slots + b) : b;
  if (s >= n) {
    if (slots && n > 0) set_status(status, TB_DEV_BAD_ID);
    return -1;
  }
  return s;
}

// Requests of up to so many tokens take the recurrent kernel: all in fp32 and without a workspace, for the runs of
// drafted tokens that are verified at once.  Up to 8 tokens it is the faster one throughout; from 12 on it depends
// on how many (request, head) pairs there are, which the rule does not look at.  Recurrent / chunked, us:
//   16/48 heads, 4, 8, 12, 16, 24 tokens:   1 request     7 / 26   12 / 27   18 / 26   23 / 27   32 / 27
//                                           4 requests   16 / 39   28 / 39   40 / 39   51 / 39   75 / 39
//                                          16 requests   29 / 96   49 / 97   68 / 98   87 /101  125 / 98
//                                          64 requests  112 /331  181 /330  254 /328  328 /328  488 /325
//   16/16 heads:                           16 requests   22 / 43   39 / 43   57 / 43   75 / 43  109 / 43
//                                          64 requests   37 /127   61 /126   85 /126  111 /126  164 /125
constexpr int64_t kDeltaStepTokens = 16;

// the chunked form, and its workspace
int launch_delta_chunks(const DeltaArgs& a, void* workspace, cudaStream_t s);
size_t delta_chunk_workspace(int64_t T, int64_t B, int64_t Hv);

TB_DEVI float4 load_half4(const __half* p) {
  const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w.x));
  const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
  return make_float4(x.x, x.y, y.x, y.y);
}
TB_DEVI float dot4(const float4& x, const float4& y) { return x.x * y.x + x.y * y.y + x.z * y.z + x.w * y.w; }
TB_DEVI void fma4(float4& d, float s, const float4& x) {
  d.x = fmaf(s, x.x, d.x);
  d.y = fmaf(s, x.y, d.y);
  d.z = fmaf(s, x.z, d.z);
  d.w = fmaf(s, x.w, d.w);
}
TB_DEVI void add4(float4& d, const float4& x) {
  d.x += x.x;
  d.y += x.y;
  d.z += x.z;
  d.w += x.w;
}
TB_DEVI void add4_xor(float4& d, int m) {
  d.x += __shfl_xor_sync(0xffffffffu, d.x, m);
  d.y += __shfl_xor_sync(0xffffffffu, d.y, m);
  d.z += __shfl_xor_sync(0xffffffffu, d.z, m);
  d.w += __shfl_xor_sync(0xffffffffu, d.w, m);
}

}  // namespace tb
