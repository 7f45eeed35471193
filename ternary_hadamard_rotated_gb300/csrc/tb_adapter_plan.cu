// The adapters' plan: a step's tokens grouped by adapter, once for all its linears.
#include <cuda_runtime.h>
#include <limits.h>

#include "tb_adapter.cuh"
#include "tb_common.cuh"
#include "tb_host.h"

namespace tb {

constexpr int kGroupThreads = 1024;
constexpr int kLongRequest = 256;  // tokens from which all CTAs write a request's tokens together

struct GroupArgs {
  const int32_t *row_start, *adapter;
  AdapterPlan* plan;
  int32_t* order;
  AdapterTile* tiles[kTileKinds];
  int32_t* status;
  int B, T, n;
};

// inclusive sum over the block; `warps` is shared scratch
TB_DEVI int block_sum(int v, int* warps) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += u;
  }
  __syncthreads();
  if (lane == 31) warps[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int w = warps[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, w, d);
      if (lane >= d) w += u;
    }
    warps[lane] = w;
  }
  __syncthreads();
  return warp ? v + warps[warp - 1] : v;
}

TB_DEVI int block_max(int v, int* warps) {  // inclusive maximum, the same way
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v = max(v, u);
  }
  __syncthreads();
  if (lane == 31) warps[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int w = warps[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, w, d);
      if (lane >= d) w = max(w, u);
    }
    warps[lane] = w;
  }
  __syncthreads();
  return warp ? max(v, warps[warp - 1]) : v;
}

// Every CTA groups all requests itself (they are few, and no CTA then waits for another); what is written is
// shared out.  A request counts where no row start before it is above its own and it ends at or before T: such
// requests never overlap, so their tokens are T at most, whatever the row starts hold.
// Bound by latency (count, sums over adapters, order): 64 requests of one token 6.3 us, 13 prompts of 5935 7.7, 1000 of
// 100000 15.2.
__global__ void __launch_bounds__(kGroupThreads) adapter_plan_kernel(const GroupArgs a) {
  extern __shared__ int32_t group_smem[];
  int32_t* start = group_smem;              // [n + 2] tokens, then where a group begins in `order`
  int32_t* tiles = group_smem + a.n + 2;    // [n] where a group's tiles begin
  int32_t* at = group_smem + 2 * (a.n + 2); // [B] where a request's tokens begin in `order`, -1: none
  __shared__ int warps[32];
  __shared__ int highest;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int groups = a.n + 1;
  int bad = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // what came before is over (see launch_early)
  for (int i = tid; i < a.n + 2; i += kGroupThreads) start[i] = 0;
  if (tid == 0) highest = 0;
  __syncthreads();
  // which requests count, and the groups' tokens
  for (int b0 = 0; b0 < a.B; b0 += kGroupThreads) {
    const int b = b0 + tid;
    int s = INT_MIN, e = INT_MIN, g = 0;
    if (b < a.B) {
      s = a.row_start[b];
      e = a.row_start[b + 1];
      g = a.adapter[b];
    }
    const int top = max(block_max(s, warps), highest);
    if (b < a.B) {
      if (g >= a.n) bad |= TB_DEV_BAD_ID;
      if (g < 0 || g >= a.n) g = a.n;
      const bool fits = s >= 0 && s == top && e >= s && e <= a.T;
      if (!fits) bad |= TB_DEV_BAD_LEN;
      at[b] = fits && e > s ? g : -1;
      if (fits && e > s) atomicAdd(&start[g], e - s);
    }
    __syncthreads();
    if (tid == kGroupThreads - 1) highest = top;
    __syncthreads();
  }
  // the groups' beginnings, and those of their tiles
  int total = 0;
  for (int g0 = 0; g0 < groups; g0 += kGroupThreads) {
    const int g = g0 + tid, c = g < groups ? start[g] : 0;
    const int sum = block_sum(c, warps);
    if (g < groups) start[g] = total + sum - c;
    total += warps[31];
    __syncthreads();
  }
  if (tid == 0) start[groups] = total;
  __syncthreads();
  for (int kind = 0; kind < kTileKinds; ++kind) {
    const int rows = tile_rows(kind);
    int sums = 0;
    for (int g0 = 0; g0 < a.n; g0 += kGroupThreads) {
      const int g = g0 + tid, c = g < a.n ? (start[g + 1] - start[g] + rows - 1) / rows : 0;
      const int sum = block_sum(c, warps);
      if (g < a.n) tiles[g] = sums + sum - c;
      sums += warps[31];
      __syncthreads();
    }
    for (int i = blockIdx.x * kGroupThreads + tid; i < sums; i += gridDim.x * kGroupThreads) {
      int lo = 0, hi = a.n - 1;
      while (lo < hi) {  // the last group whose tiles begin at or before i
        const int mid = (lo + hi + 1) >> 1;
        if (tiles[mid] <= i) lo = mid;
        else hi = mid - 1;
      }
      AdapterTile t;
      t.adapter = lo;
      t.first = start[lo] + (i - tiles[lo]) * rows;
      t.count = min(rows, start[lo + 1] - t.first);
      t.pad = 0;
      a.tiles[kind][i] = t;
    }
    if (blockIdx.x == 0 && tid == 0) a.plan->tiles[kind] = sums;
    __syncthreads();
  }
  if (blockIdx.x == 0) {
    if (tid == 0) {
      a.plan->magic = kAdapterMagic;
      a.plan->T = a.T;
      a.plan->n = a.n;
      a.plan->bare = start[a.n];
      a.plan->rows = total;
      a.plan->pad = 0;
    }
    if (bad) set_status(a.status, bad);
  }
  // a request's place: behind those of its group that come before it.  Inside a warp by comparing all pairs,
  // between warps in turn (start[g] moves on as the group's requests are placed)
  for (int b0 = 0; b0 < a.B; b0 += kGroupThreads) {
    const int b = b0 + tid, g = b < a.B ? at[b] : -1;
    const int len = g >= 0 ? a.row_start[b + 1] - a.row_start[b] : 0;
    int before = 0, all = 0;
#pragma unroll
    for (int l = 0; l < 32; ++l) {
      const int og = __shfl_sync(0xffffffffu, g, l), ol = __shfl_sync(0xffffffffu, len, l);
      if (og == g) {
        all += ol;
        if (l < lane) before += ol;
      }
    }
    const int turns = min((a.B - b0 + 31) / 32, kGroupThreads / 32);
    for (int w = 0; w < turns; ++w) {
      if (w == warp && g >= 0) at[b] = start[g] + before;
      __syncwarp();
      if (w == warp && g >= 0 && before + len == all) start[g] += all;  // the last of its group in the warp
      __syncthreads();
    }
  }
  // the tokens: a warp for a short request, all CTAs for a long one
  const int warp_all = blockIdx.x * (kGroupThreads / 32) + warp, n_warps = gridDim.x * (kGroupThreads / 32);
  for (int b = warp_all; b < a.B; b += n_warps) {
    const int p = at[b];
    if (p < 0) continue;
    const int s = a.row_start[b], len = a.row_start[b + 1] - s;
    if (len <= kLongRequest)
      for (int i = lane; i < len; i += 32) a.order[p + i] = s + i;
  }
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int b = b0 + lane;
    const bool is_long = b < a.B && at[b] >= 0 && a.row_start[b + 1] - a.row_start[b] > kLongRequest;
    for (unsigned m = __ballot_sync(0xffffffffu, is_long); m; m &= m - 1) {
      const int c = b0 + __ffs(m) - 1;
      const int s = a.row_start[c], len = a.row_start[c + 1] - s;
      for (int i = blockIdx.x * kGroupThreads + tid; i < len; i += gridDim.x * kGroupThreads) a.order[at[c] + i] = s + i;
    }
  }
}

}  // namespace tb

extern "C" size_t tb_adapter_plan_size(int64_t T, int64_t n) {
  using namespace tb;
  if (T < 0 || T > INT_MAX / 2 || n < 1 || n > kAdapterMaxN) return 0;
  return adapter_tiles_at(T, n, kTileKinds);
}

extern "C" int tb_adapter_plan(const int32_t* row_start, const int32_t* adapter, int64_t B, int64_t T, int64_t n, void* plan,
                               size_t plan_bytes, int32_t* dev_status, void* stream) {
  using namespace tb;
  if (B < 1 || T < 0 || T > INT_MAX / 2 || n < 1) return TB_ERR_SHAPE;
  if (B > kAdapterMaxB || n > kAdapterMaxN) return TB_ERR_TOO_LARGE;
  if (!row_start || !adapter || !plan) return TB_ERR_NULL;
  if (!aligned_to(row_start, 4) || !aligned_to(adapter, 4) || !aligned16(plan)) return TB_ERR_ALIGN;
  if (plan_bytes < tb_adapter_plan_size(T, n)) return TB_ERR_WORKSPACE;
  DeviceFacts f;
  int rc = device_facts(&f);
  if (rc != TB_OK) return rc;
  const int smem = (int)(B + 2 * (n + 2)) * 4;
  rc = ensure_dynamic_smem(reinterpret_cast<const void*>(adapter_plan_kernel), f.device, smem);
  if (rc != TB_OK) return rc;
  GroupArgs a;
  a.row_start = row_start;
  a.adapter = adapter;
  a.plan = static_cast<AdapterPlan*>(plan);
  char* base = static_cast<char*>(plan);
  a.order = reinterpret_cast<int32_t*>(base + adapter_order_at());
  for (int i = 0; i < kTileKinds; ++i) a.tiles[i] = reinterpret_cast<AdapterTile*>(base + adapter_tiles_at(T, n, i));
  a.status = dev_status;
  a.B = (int)B;
  a.T = (int)T;
  a.n = (int)n;
  int64_t blocks = (T > B * 32 ? T : B * 32) / kGroupThreads + 1;
  if (blocks > f.sms) blocks = f.sms;
  return launch_early(adapter_plan_kernel, dim3((unsigned)blocks), kGroupThreads, (size_t)smem, static_cast<cudaStream_t>(stream), a);
}
