// The paged K/V cache: its bookkeeping (block tables, slot maps) and the write of new tokens.
//
// Cache layout: [pages, Hkv, page, D] fp16, one array for K and one for V.  The rows of one KV
// head in one page are one contiguous block, which is what the attention that reads the cache
// streams.  A slot is the token's place in the pool: page number * page + place in the page.
#include <cuda_runtime.h>
#include <limits.h>

#include "tb_common.cuh"
#include "tb_host.h"

namespace tb {

// ---------------------------------------------------------------- plan
// need_b = ceil((cached_b + fresh_b) / page), have_b = ceil(cached_b / page); request b's i-th
// new page is free[sum_{a<b} (need_a - have_a) + i].  Every CTA scans all lengths itself (at most
// 16384 requests: one pass over L2-resident words), so no CTA waits for another and one launch
// does it all; the sums stay in shared memory, and each CTA then fills its share of the slots (by
// tokens, so that one long prompt is spread over all CTAs) and of the table (by requests).
// Bound by latency: 256 requests of one token 3.8 us, 500 of 1000 tokens each (4 MB of slots) 8.1 us, in a
// replayed graph (7.1 and 10.2 us a call).
constexpr int kPlanThreads = 512;
constexpr int kPlanMaxB = 16384;

struct PlanArgs {
  const int32_t* cached;
  const int32_t* fresh;
  const int32_t* free_pages;
  int32_t* table;
  int64_t* slots;
  int32_t* row_start;
  int32_t* total;
  int32_t* used;
  int32_t* status;
  int64_t n_free, max_pages, T;
  int B, page_log2;
};

struct PlanLen {
  int32_t cached, fresh;  // as used: clipped to what the arguments can hold
  int64_t have, need;     // pages, clipped to the table's width
  int bad;
};

TB_DEVI PlanLen plan_len(const PlanArgs& a, int b) {
  PlanLen r;
  r.bad = 0;
  int64_t c = __ldg(a.cached + b), f = __ldg(a.fresh + b);
  if (c < 0 || f < 0 || f > a.T || c + f > INT_MAX) {
    r.bad = TB_DEV_BAD_LEN;
    c = c < 0 ? 0 : c;
    f = f < 0 ? 0 : (f > a.T ? a.T : f);
    if (c + f > INT_MAX) f = INT_MAX - c;
  }
  r.cached = (int32_t)c;
  r.fresh = (int32_t)f;
  const int64_t m = (1ll << a.page_log2) - 1;
  r.have = (c + m) >> a.page_log2;
  r.need = (c + f + m) >> a.page_log2;
  if (r.need > a.max_pages) {
    r.need = a.max_pages;
    if (f > 0) r.bad |= TB_DEV_NO_PAGE;
  }
  if (r.have > r.need) r.have = r.need;
  return r;
}

TB_DEVI int32_t clip_int(int64_t v) { return v > INT_MAX ? INT_MAX : (int32_t)v; }

__global__ void __launch_bounds__(kPlanThreads) cache_plan_kernel(const PlanArgs a) {
  extern __shared__ int32_t plan_smem[];
  int32_t* first_tok = plan_smem;          // [B] tokens of the requests before b
  int32_t* first_new = plan_smem + a.B;    // [B] new pages of the requests before b
  __shared__ int64_t warp_tok[kPlanThreads / 32], warp_new[kPlanThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int64_t base_tok = 0, base_new = 0;
  int bad = 0;
  for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    PlanLen l = {0, 0, 0, 0, 0};
    if (b < a.B) l = plan_len(a, b);
    bad |= l.bad;
    int64_t st = l.fresh, sn = l.need - l.have;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t t = __shfl_up_sync(0xffffffffu, st, d), n = __shfl_up_sync(0xffffffffu, sn, d);
      if (lane >= d) {
        st += t;
        sn += n;
      }
    }
    __syncthreads();  // the previous round's sums have been read
    if (lane == 31) {
      warp_tok[warp] = st;
      warp_new[warp] = sn;
    }
    __syncthreads();
    int64_t wt = base_tok, wn = base_new;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
      if (w == warp) {
        wt = base_tok;
        wn = base_new;
      }
      base_tok += warp_tok[w];
      base_new += warp_new[w];
    }
    if (b < a.B) {
      first_tok[b] = clip_int(wt + st - l.fresh);
      first_new[b] = clip_int(wn + sn - (l.need - l.have));
      if (blockIdx.x == 0) {
        a.row_start[b] = clip_int(wt + st - l.fresh);
        a.total[b] = l.cached + l.fresh;
      }
    }
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    if (tid == 0) {
      a.row_start[a.B] = clip_int(base_tok);
      if (a.used) *a.used = clip_int(base_new < a.n_free ? base_new : a.n_free);
      if (base_tok > a.T) bad |= TB_DEV_BAD_LEN;
      if (base_new > a.n_free) bad |= TB_DEV_NO_PAGE;
    }
    if (bad) set_status(a.status, bad);
  }
  // the table: one warp per request, its new pages
  const int warps = (int)gridDim.x * (kPlanThreads / 32);
  for (int b = (int)blockIdx.x * (kPlanThreads / 32) + warp; b < a.B; b += warps) {
    const PlanLen l = plan_len(a, b);
    for (int64_t p = l.have + lane; p < l.need; p += 32) {
      const int64_t f = (int64_t)first_new[b] + (p - l.have);
      a.table[(int64_t)b * a.max_pages + p] = f < a.n_free ? __ldg(a.free_pages + f) : -1;
    }
  }
  // the slots: a run of tokens per warp, so that a lane finds its first token's request by bisection of
  // the sums and the next ones' by going on from there
  const int64_t have_tok = base_tok < a.T ? base_tok : a.T;
  const int64_t run = ((a.T + warps - 1) / warps + 31) & ~31ll;
  const int64_t t0 = ((int64_t)blockIdx.x * (kPlanThreads / 32) + warp) * run;
  const int64_t t1 = t0 + run < a.T ? t0 + run : a.T;
  const int64_t pmask = (1ll << a.page_log2) - 1;
  int b = -1;
  int64_t b_end = 0;  // the request's tokens end here
  PlanLen l = {0, 0, 0, 0, 0};
  for (int64_t t = t0 + lane; t < t1; t += 32) {
    int64_t slot = -1;
    if (t < have_tok) {
      if (t >= b_end) {
        int lo = b < 0 ? 0 : b, hi = a.B - 1;
        if (b < 0) {
          while (lo < hi) {  // the last request whose first token is at or before t
            const int mid = (lo + hi + 1) >> 1;
            if (first_tok[mid] <= t) lo = mid;
            else hi = mid - 1;
          }
        } else {
          while (lo < hi && first_tok[lo + 1] <= t) ++lo;
        }
        b = lo;
        l = plan_len(a, b);
        b_end = (int64_t)first_tok[b] + l.fresh;
      }
      const int64_t pos = (int64_t)l.cached + (t - first_tok[b]);
      const int64_t p = pos >> a.page_log2;
      int32_t pg = -1;
      if (p < l.have) {
        pg = a.table[(int64_t)b * a.max_pages + p];
        if (pg < 0) set_status(a.status, TB_DEV_BAD_SLOT);
      } else if (p < l.need) {
        const int64_t f = (int64_t)first_new[b] + (p - l.have);
        if (f < a.n_free) pg = __ldg(a.free_pages + f);
      }
      if (pg >= 0) slot = ((int64_t)pg << a.page_log2) + (pos & pmask);
    }
    a.slots[t] = slot;
  }
}

// ---------------------------------------------------------------- write
// A warp per token: 16 bytes a lane, four pieces of K and of V in flight, so that a head's row is one
// contiguous run on both sides.  Bound by the bytes: 40001 tokens of 4 heads of 256 (328 MB) in 52.5 us,
// 0.92 of measured HBM, in a replayed graph; 54.9 us a call, 0.88.
constexpr int kWriteThreads = 256, kWriteUnroll = 4;

__global__ void __launch_bounds__(kWriteThreads) cache_write_kernel(
    const __half* __restrict__ k, int64_t ldk, const __half* __restrict__ v, int64_t ldv,
    const int64_t* __restrict__ slots, int64_t T, int Hkv, int D, __half* __restrict__ kc,
    __half* __restrict__ vc, int64_t n_slots, int page_log2, int32_t* __restrict__ status) {
  const int lane = threadIdx.x & 31;
  const unsigned vec = (unsigned)D / 8, row = (unsigned)Hkv * vec;  // 16-byte pieces of a head's row and of a token
  const int64_t pmask = (1ll << page_log2) - 1;
  const int64_t step = (int64_t)gridDim.x * (kWriteThreads / 32);
  for (int64_t t = blockIdx.x * (int64_t)(kWriteThreads / 32) + (threadIdx.x >> 5); t < T; t += step) {
    const int64_t slot = __ldg(slots + t);
    if (slot < 0) continue;  // a padded token
    if (slot >= n_slots) {
      if (lane == 0) set_status(status, TB_DEV_BAD_SLOT);
      continue;
    }
    // head h of the token: page, h, place in the page
    const int64_t base = ((((slot >> page_log2) * Hkv) << page_log2) + (slot & pmask)) * D;
    const int64_t head = (int64_t)D << page_log2;
    const uint4 *ks = reinterpret_cast<const uint4*>(k + t * ldk), *vs = reinterpret_cast<const uint4*>(v + t * ldv);
    for (unsigned c0 = lane; c0 < row; c0 += 32 * kWriteUnroll) {
      uint4 kk[kWriteUnroll], vv[kWriteUnroll];
#pragma unroll
      for (int u = 0; u < kWriteUnroll; ++u) {
        const unsigned c = c0 + 32 * u;
        if (c < row) {
          kk[u] = __ldcs(ks + c);
          vv[u] = __ldcs(vs + c);
        }
      }
#pragma unroll
      for (int u = 0; u < kWriteUnroll; ++u) {
        const unsigned c = c0 + 32 * u, h = c / vec;
        if (c < row) {
          const int64_t dst = base + h * head + (c - h * vec) * 8;
          *reinterpret_cast<uint4*>(kc + dst) = kk[u];
          *reinterpret_cast<uint4*>(vc + dst) = vv[u];
        }
      }
    }
  }
}

}  // namespace tb

extern "C" int tb_cache_plan(const int32_t* cached, const int32_t* fresh, int64_t B, int64_t page,
                             const int32_t* free_pages, int64_t n_free, int32_t* table,
                             int64_t max_pages, int64_t* slots, int64_t T, int32_t* row_start,
                             int32_t* total, int32_t* used, int32_t* dev_status, void* stream) {
  using namespace tb;
  if (B < 1 || T < 0 || T > INT_MAX || n_free < 0 || n_free > INT_MAX || max_pages < 1 || max_pages > INT_MAX)
    return TB_ERR_SHAPE;
  if (!supported_page(page)) return TB_ERR_UNSUPPORTED;
  if (B > kPlanMaxB) return TB_ERR_TOO_LARGE;
  if (!cached || !fresh || !table || !row_start || !total || (T && !slots) || (n_free && !free_pages))
    return TB_ERR_NULL;
  if (!aligned_to(cached, 4) || !aligned_to(fresh, 4) || !aligned_to(table, 4) || !aligned_to(row_start, 4) ||
      !aligned_to(total, 4) || !aligned_to(slots, 8) || !aligned_to(free_pages, 4) || !aligned_to(used, 4))
    return TB_ERR_ALIGN;
  DeviceFacts f;
  int rc = device_facts(&f);
  if (rc != TB_OK) return rc;
  const int smem = (int)B * 8;
  rc = ensure_dynamic_smem(reinterpret_cast<const void*>(cache_plan_kernel), f.device, smem);
  if (rc != TB_OK) return rc;
  PlanArgs a;
  a.cached = cached;
  a.fresh = fresh;
  a.free_pages = free_pages;
  a.table = table;
  a.slots = slots;
  a.row_start = row_start;
  a.total = total;
  a.used = used;
  a.status = dev_status;
  a.n_free = n_free;
  a.max_pages = max_pages;
  a.T = T;
  a.B = (int)B;
  a.page_log2 = log2_of(page);
  int64_t work = T > B * 32 ? T : B * 32;  // a thread per token, a warp per request
  int64_t blocks = (work + kPlanThreads - 1) / kPlanThreads;
  if (blocks > f.sms) blocks = f.sms;
  cache_plan_kernel<<<(int)blocks, kPlanThreads, smem, static_cast<cudaStream_t>(stream)>>>(a);
  return check_launch();
}

extern "C" int tb_cache_write(const uint16_t* k, int64_t ldk, const uint16_t* v, int64_t ldv,
                              const int64_t* slots, int64_t T, int64_t Hkv, int64_t D,
                              uint16_t* k_cache, uint16_t* v_cache, int64_t pages, int64_t page,
                              int32_t* dev_status, void* stream) {
  using namespace tb;
  if (T < 0 || Hkv < 1 || Hkv > 1024 || D < 8 || D > 1024 || D % 8 || pages < 1 || pages > INT_MAX)
    return TB_ERR_SHAPE;
  if (ldk < Hkv * D || ldv < Hkv * D || ldk % 8 || ldv % 8) return TB_ERR_SHAPE;
  if (!supported_page(page)) return TB_ERR_UNSUPPORTED;
  if (T == 0) return TB_OK;
  if (!k || !v || !slots || !k_cache || !v_cache) return TB_ERR_NULL;
  if (!aligned16(k) || !aligned16(v) || !aligned_to(slots, 8) || !aligned16(k_cache) || !aligned16(v_cache))
    return TB_ERR_ALIGN;
  DeviceFacts f;
  int rc = device_facts(&f);
  if (rc != TB_OK) return rc;
  int64_t blocks = (T + kWriteThreads / 32 - 1) / (kWriteThreads / 32);
  const int64_t cap = (int64_t)f.sms * 8;
  if (blocks > cap) blocks = cap;
  cache_write_kernel<<<(int)blocks, kWriteThreads, 0, static_cast<cudaStream_t>(stream)>>>(
      reinterpret_cast<const __half*>(k), ldk, reinterpret_cast<const __half*>(v), ldv, slots, T,
      (int)Hkv, (int)D, reinterpret_cast<__half*>(k_cache), reinterpret_cast<__half*>(v_cache),
      pages * page, log2_of(page), dev_status);
  return check_launch();
}
