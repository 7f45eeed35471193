// Low-rank adapters of many requests beside a shared linear: out[t] = y[t] + scale[g] B[g] (A[g] x[t]), g the
// adapter of token t's request.
#include <cuda_runtime.h>
#include <limits.h>

#include "tb_adapter.cuh"
#include "tb_common.cuh"
#include "tb_host.h"

namespace tb {

struct AdapterArgs {
  const __half *x, *a, *b, *y;
  __half* out;
  const int32_t* rank;
  const float* scale;
  const AdapterPlan* plan;
  const int32_t* order;
  const AdapterTile* tiles;
  float* h;
  int32_t* status;
  int64_t ldx, ldy, ldo;
  int T, n, K, N, R;
};

TB_DEVI bool plan_fits(const AdapterArgs& a) {
  const bool ok = a.plan->magic == kAdapterMagic && a.plan->T == a.T && a.plan->n == a.n;
  if (!ok && blockIdx.x == 0 && threadIdx.x == 0) set_status(a.status, TB_DEV_BAD_PLAN);
  return ok;
}

TB_DEVI int live_rank(const AdapterArgs& a, int g) {
  if (g >= a.n) return 0;
  const int r = a.rank ? __ldg(a.rank + g) : a.R;
  return r < 0 ? 0 : min(r, a.R);
}

// h = scale A x: a warp per (token, row of A)
__global__ void __launch_bounds__(256) adapter_down_kernel(const AdapterArgs a) {
  if (!plan_fits(a)) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = blockIdx.x; i < a.plan->tiles[0]; i += gridDim.x) {
    const AdapterTile t = a.tiles[i];
    const int live = live_rank(a, t.adapter);
    for (int j = warp; j < t.count * live; j += 8) {
      const int p = j / live, r = j - p * live;
      const __half* x = a.x + a.order[t.first + p] * a.ldx;
      const __half* w = a.a + ((int64_t)t.adapter * a.R + r) * a.K;
      float s = 0.f;
      for (int k = lane; k < a.K; k += 32) s = fmaf(__half2float(x[k]), __half2float(w[k]), s);
#pragma unroll
      for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
      if (lane == 0) a.h[(int64_t)(t.first + p) * a.R + r] = s * a.scale[t.adapter];
    }
  }
}

// out = y + B h: a thread per (token, column)
__global__ void __launch_bounds__(256) adapter_up_kernel(const AdapterArgs a) {
  if (!plan_fits(a)) return;
  for (int i = blockIdx.x; i < a.plan->tiles[0]; i += gridDim.x) {
    const AdapterTile t = a.tiles[i];
    const int live = live_rank(a, t.adapter);
    if (!live && a.out == a.y) continue;
    for (int p = 0; p < t.count; ++p) {
      const int tok = a.order[t.first + p];
      for (int c = blockIdx.y * 256 + threadIdx.x; c < a.N; c += gridDim.y * 256) {
        const __half y = a.y[tok * a.ldy + c];
        if (!live) {
          a.out[tok * a.ldo + c] = y;
          continue;
        }
        float s = 0.f;
        for (int r = 0; r < live; ++r) s = fmaf(a.h[(int64_t)(t.first + p) * a.R + r], __half2float(a.b[((int64_t)t.adapter * a.N + c) * a.R + r]), s);
        a.out[tok * a.ldo + c] = __float2half_rn(__half2float(y) + s);
      }
    }
  }
}

}  // namespace tb

extern "C" size_t tb_adapter_linear_workspace_size(int64_t T, int64_t n, int64_t K, int64_t N, int64_t R) {
  using namespace tb;
  if (T < 0 || T > INT_MAX / 2 || n < 1 || K < 8 || N < 8 || R < 8 || R > kAdapterMaxR) return 0;
  return (size_t)T * R * 4;
}

extern "C" int tb_adapter_linear(const uint16_t* x, int64_t ldx, int64_t T, int64_t K, const uint16_t* a, const uint16_t* b, int64_t n,
                                 int64_t R, int64_t N, const int32_t* rank, const float* scale, const void* plan, const uint16_t* y,
                                 int64_t ldy, uint16_t* out, int64_t ldo, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                 void* stream) {
  using namespace tb;
  if (T < 0 || T > INT_MAX / 2 || K < 8 || K % 8 || K > (1 << 20) || N < 8 || N % 8 || N > (1 << 20) || R < 8 || R % 8 || n < 1) return TB_ERR_SHAPE;
  if (ldx < K || ldx % 8 || ldy < N || ldy % 8 || ldo < N || ldo % 8) return TB_ERR_SHAPE;
  if (R > kAdapterMaxR) return TB_ERR_UNSUPPORTED;
  if (n > kAdapterMaxN) return TB_ERR_TOO_LARGE;
  if (T == 0) return TB_OK;
  if (!x || !a || !b || !scale || !plan || !y || !out) return TB_ERR_NULL;
  if (!aligned16(x) || !aligned16(a) || !aligned16(b) || !aligned16(plan) || !aligned16(y) || !aligned16(out) || !aligned16(workspace) ||
      !aligned_to(rank, 4) || !aligned_to(scale, 4))
    return TB_ERR_ALIGN;
  if (out == y && ldo != ldy && T > 1) return TB_ERR_SHAPE;  // in place only element for element
  const size_t need = tb_adapter_linear_workspace_size(T, n, K, N, R);
  if (need && (!workspace || workspace_bytes < need)) return TB_ERR_WORKSPACE;
  DeviceFacts f;
  const int rc = device_facts(&f);
  if (rc != TB_OK) return rc;
  AdapterArgs g;
  g.x = reinterpret_cast<const __half*>(x);
  g.a = reinterpret_cast<const __half*>(a);
  g.b = reinterpret_cast<const __half*>(b);
  g.y = reinterpret_cast<const __half*>(y);
  g.out = reinterpret_cast<__half*>(out);
  g.rank = rank;
  g.scale = scale;
  const char* base = static_cast<const char*>(plan);
  g.plan = static_cast<const AdapterPlan*>(plan);
  g.order = reinterpret_cast<const int32_t*>(base + adapter_order_at());
  g.tiles = reinterpret_cast<const AdapterTile*>(base + adapter_tiles_at(T, n, 0));
  g.h = static_cast<float*>(workspace);
  g.status = dev_status;
  g.ldx = ldx;
  g.ldy = ldy;
  g.ldo = ldo;
  g.T = (int)T;
  g.n = (int)n;
  g.K = (int)K;
  g.N = (int)N;
  g.R = (int)R;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  int64_t tiles = adapter_max_tiles(T, n, 0);
  if (tiles > 4096) tiles = 4096;
  adapter_down_kernel<<<(int)tiles, 256, 0, s>>>(g);
  adapter_up_kernel<<<dim3((unsigned)tiles, (unsigned)((N + 1023) / 1024)), 256, 0, s>>>(g);
  return check_launch();
}
