// Low-rank adapters of many requests beside a shared linear: out[t] = y[t] + scale[g] B[g] (A[g] x[t]), g the
// adapter of token t's request.
//
// Two launches, the second (programmatic) loading what the first does not write before it waits for it:
//   down  h = scale A x, fp32 [T, R] in the order of the plan; mma.sync on tiles of 16 or 32 tokens of one adapter
//   up    out = y + B h, mma.sync with h as two fp16 terms; few tokens: tiles of 16, bound by the weights, which go
//         from global memory straight to the registers; many: tiles of 128, bound by y and out
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <limits.h>

#include "tb_adapter.cuh"
#include "tb_common.cuh"
#include "tb_host.h"

namespace tb {

namespace cg = cooperative_groups;

struct AdapterArgs {
  const __half *x, *a, *b, *y;
  __half* out;
  const int32_t* rank;
  const float* scale;
  const AdapterPlan* plan;
  const int32_t* order;
  const AdapterTile* down_tiles;
  const AdapterTile* up_tiles;
  float* h;
  int32_t* status;
  int64_t ldx, ldy, ldo;
  int T, n, K, N, R;
  int cluster, down_kind, up_kind;
  int groups;  // of column tiles: CTAs a row tile has
};

TB_DEVI bool plan_fits(const AdapterArgs& a) {
  const AdapterPlan& p = *a.plan;
  return p.magic == kAdapterMagic && p.T == a.T && p.n == a.n;
}

TB_DEVI int live_rank(const AdapterArgs& a, int g) {
  if (g >= a.n) return 0;
  const int r = a.rank ? __ldg(a.rank + g) : a.R;
  return r < 0 ? 0 : min(r, a.R);
}

TB_DEVI void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

TB_DEVI void cp_async16(uint32_t dst, const void* src, int bytes) {  // the rest of the 16 bytes is zeroed
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
TB_DEVI void ldmatrix4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}

// ---------------------------------------------------------------- down
// Parts of a tile's h, [PARTS][M][N] in shared memory, summed in their order, then over the cluster's CTAs in theirs.
template <int PARTS, int M, int N, int THREADS>
TB_DEVI void join_down(const AdapterArgs& a, const AdapterTile& t, float* part, int share, int r0, int live) {
  const int tid = threadIdx.x;
  const float scale = __ldg(a.scale + t.adapter);
  auto store = [&](int e, float s) {
    const int row = e / N, r = r0 + e % N;
    if (row < t.count && r < a.R) a.h[(int64_t)(t.first + row) * a.R + r] = r < live ? s * scale : 0.f;
  };
  __syncthreads();
  for (int e = tid; e < M * N; e += THREADS) {
    float s = part[e];
#pragma unroll
    for (int w = 1; w < PARTS; ++w) s += part[w * M * N + e];
    if (a.cluster == 1) store(e, s);
    else part[e] = s;
  }
  if (a.cluster == 1) return;
  cg::cluster_group cl = cg::this_cluster();
  cl.sync();
  for (int e = share * THREADS + tid; e < M * N; e += a.cluster * THREADS) {
    float s = 0.f;
    for (int r = 0; r < a.cluster; ++r) s += *cl.map_shared_rank(part + e, r);
    store(e, s);
  }
  cl.sync();  // the parts stay until they have been read
}

// Few tokens: a CTA takes 16 tokens by NT x 8 rows of A; its warps and those of its cluster share out K in steps of
// 32.  A step's operands go from global memory straight to the mma's registers: thread (g, c) of a warp holds 8
// neighbouring elements of rows g (and g + 8), which serve as the k's 2c, 2c + 1, 2c + 8 and 2c + 9 of two MMAs: a
// product over k does not mind their order, if both operands have the same.
constexpr int kDownThreads = 256, kDownWarps = kDownThreads / 32;

template <int NT>
__global__ void __launch_bounds__(kDownThreads, 2) adapter_down_few_kernel(const AdapterArgs a) {
  constexpr int N = NT * 8;
  constexpr int kUnroll = NT <= 2 ? 4 : 2;
  extern __shared__ __align__(128) unsigned char down_smem[];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (!plan_fits(a)) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) set_status(a.status, TB_DEV_BAD_PLAN);
    return;
  }
  const int tile = blockIdx.x / a.cluster, share = blockIdx.x - tile * a.cluster;
  if (tile >= a.plan->tiles[a.down_kind]) return;  // (all CTAs of the cluster)
  const AdapterTile t = a.down_tiles[tile];
  if (t.adapter >= a.n) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const int r0 = blockIdx.y * N, live = live_rank(a, t.adapter);
  const int nt_live = min(NT, max(0, (live - r0 + 7) >> 3));

  const __half* xr[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) xr[i] = i * 8 + g < t.count ? a.x + a.order[t.first + i * 8 + g] * a.ldx + c * 8 : nullptr;
  const __half* ar = a.a + ((int64_t)t.adapter * a.R + r0 + g) * a.K + c * 8;
  float acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
  const int steps = (a.K + 31) >> 5, stride = a.cluster * kDownWarps;
  if (nt_live > 0) {
    for (int s = share * kDownWarps + warp; s < steps; s += stride * kUnroll) {
      uint4 xv[kUnroll][2], av[kUnroll][NT];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int k = (s + u * stride) * 32;
        const bool in = k + c * 8 < a.K;
#pragma unroll
        for (int i = 0; i < 2; ++i)
          xv[u][i] = in && xr[i] ? __ldg(reinterpret_cast<const uint4*>(xr[i] + k)) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int n = 0; n < NT; ++n)
          av[u][n] = in && n < nt_live && r0 + n * 8 + g < a.R ? __ldg(reinterpret_cast<const uint4*>(ar + (int64_t)n * 8 * a.K + k)) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const uint4 p = xv[u][0], q = xv[u][1];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma_16816(acc[n], p.x, q.x, p.y, q.y, av[u][n].x, av[u][n].y);
          mma_16816(acc[n], p.z, q.z, p.w, q.w, av[u][n].z, av[u][n].w);
        }
      }
    }
  }
  float* part = reinterpret_cast<float*>(down_smem) + warp * 16 * N;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    *reinterpret_cast<float2*>(part + g * N + n * 8 + 2 * c) = make_float2(acc[n][0], acc[n][1]);
    *reinterpret_cast<float2*>(part + (g + 8) * N + n * 8 + 2 * c) = make_float2(acc[n][2], acc[n][3]);
  }
  join_down<kDownWarps, 16, N, kDownThreads>(a, t, reinterpret_cast<float*>(down_smem), share, r0, live);
}

// Many tokens: a CTA takes 32 tokens by NT x 8 rows of A, both through shared memory by cp.async, 64 of K a stage and
// kStages - 1 stages ahead; rows of 128 bytes, their 16-byte pieces exchanged by row (piece ^ row mod 8), so that
// ldmatrix finds eight rows in eight different banks.  Warps: two by rows, four by the stage's k's.
constexpr int kManyRows = 32, kStages = 8;

template <int NT>
constexpr int down_many_smem() {
  const int stages = kStages * (kManyRows + NT * 8) * 128, parts = 4 * kManyRows * NT * 8 * 4;
  return stages > parts ? stages : parts;
}

template <int NT>
__global__ void __launch_bounds__(kDownThreads, 2) adapter_down_many_kernel(const AdapterArgs a) {
  constexpr int N = NT * 8, kStageBytes = (kManyRows + N) * 128;
  extern __shared__ __align__(128) unsigned char down_smem[];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (!plan_fits(a)) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) set_status(a.status, TB_DEV_BAD_PLAN);
    return;
  }
  const int tile = blockIdx.x / a.cluster, share = blockIdx.x - tile * a.cluster;
  if (tile >= a.plan->tiles[a.down_kind]) return;  // (all CTAs of the cluster)
  const AdapterTile t = a.down_tiles[tile];
  if (t.adapter >= a.n) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const int r0 = blockIdx.y * N, live = live_rank(a, t.adapter);
  const uint32_t base = smem_u32(down_smem);
  const int steps = (a.K + 63) >> 6, mine = (steps - share + a.cluster - 1) / a.cluster;

  // a thread's pieces of a stage: one of x, NT / 4 of A
  const int row = tid >> 3, piece = tid & 7;
  const uint32_t at = row * 128 + ((piece ^ (row & 7)) << 4);
  const bool has_x = row < t.count;
  const __half* xp = a.x + (has_x ? a.order[t.first + row] * a.ldx : 0) + piece * 8;
  const __half* ap = a.a + ((int64_t)t.adapter * a.R + r0 + row) * a.K + piece * 8;
  auto fetch = [&](int i) {
    const int k = (share + i * a.cluster) * 64;
    const uint32_t dst = base + (i % kStages) * kStageBytes + at;
    const bool in = k + piece * 8 < a.K;
    cp_async16(dst, has_x && in ? xp + k : a.x, has_x && in ? 16 : 0);
#pragma unroll
    for (int j = 0; j < (NT + 3) / 4; ++j)
      if (NT >= 4 || row < N) {
        const bool have = in && r0 + row + j * 32 < live;
        cp_async16(dst + (kManyRows + j * 32) * 128, have ? ap + (int64_t)j * 32 * a.K + k : a.a, have ? 16 : 0);
      }
  };
  float acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
  if (r0 < live) {
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
      if (i < mine) fetch(i);
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
    const int wm = warp & 1, wk = (warp >> 1) * 2;  // rows of 16, pieces of the stage
    // ldmatrix: lanes 0-15 rows, lanes 16-31 the same rows' next piece; for A rows 0-7, their next piece, rows 8-15
    const int xr = wm * 16 + (lane & 15), br = (lane & 7) + (lane >> 4) * 8;
    const uint32_t x_at = xr * 128 + (((wk + (lane >> 4)) ^ (xr & 7)) << 4);
    const uint32_t b_at = (kManyRows + br) * 128 + (((wk + (lane >> 3 & 1)) ^ (br & 7)) << 4);
    for (int i = 0; i < mine; ++i) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
      __syncthreads();  // stage i is there, and stage i - 1 has been used
      if (i + kStages - 1 < mine) fetch(i + kStages - 1);
      asm volatile("cp.async.commit_group;" ::: "memory");
      const uint32_t st = base + (i % kStages) * kStageBytes;
      uint32_t x[4], b[4];
      ldmatrix4(x, st + x_at);
#pragma unroll
      for (int n = 0; n < NT; n += 2) {
        ldmatrix4(b, st + b_at + n * 8 * 128);
        mma_16816(acc[n], x[0], x[1], x[2], x[3], b[0], b[1]);
        mma_16816(acc[n + 1], x[0], x[1], x[2], x[3], b[2], b[3]);
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();  // the stages' place is the parts' now
  }
  float* part = reinterpret_cast<float*>(down_smem) + (warp >> 1) * kManyRows * N + (warp & 1) * 16 * N;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    *reinterpret_cast<float2*>(part + g * N + n * 8 + 2 * c) = make_float2(acc[n][0], acc[n][1]);
    *reinterpret_cast<float2*>(part + (g + 8) * N + n * 8 + 2 * c) = make_float2(acc[n][2], acc[n][3]);
  }
  join_down<4, kManyRows, N, kDownThreads>(a, t, reinterpret_cast<float*>(down_smem), share, r0, live);
}

// ---------------------------------------------------------------- h as fp16
// h 2^e = hi + lo with 2^e of the token's own (its largest h 2^e in [2^14, 2^15)): 22 bits, of h down to 2^-39 of the
// token's largest; fp32 sums of hi B and lo B, then 2^-e.

// 2^e and 2^-e for a token whose largest |h| is top; 0 and what is not finite stay as they are
TB_DEVI float up_scale(float top, float& back) {
  int e = 14 - ((int)(__float_as_uint(top) >> 23) - 127);
  if (!(top > 0.f) || !(top < INFINITY)) e = 0;
  e = max(-126, min(126, e));
  back = __uint_as_float((uint32_t)(127 - e) << 23);
  return __uint_as_float((uint32_t)(127 + e) << 23);
}

TB_DEVI void two_terms(float4 v, float up, uint2& hi, uint2& lo) {
  const float f[4] = {v.x * up, v.y * up, v.z * up, v.w * up};
  __half h[4], l[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    h[j] = __float2half_rn(f[j]);
    const float b = __half2float(h[j]);
    l[j] = fabsf(b) < INFINITY ? __float2half_rn(f[j] - b) : __half();
  }
  hi = *reinterpret_cast<const uint2*>(h);
  lo = *reinterpret_cast<const uint2*>(l);
}

// ---------------------------------------------------------------- up, few tokens
// The columns of out (rows of B) are the mma's 16 rows and the tokens its 8 columns, so that a weight is read once
// for a tile of 16 tokens and an idle token costs nothing but its place.  A warp takes 32 columns at a time, and
// every CTA an equal run of all tiles' columns.  Thread (g, c) holds columns n0 + 4 g .. + 3: 8 bytes of y and out a
// token, and 8 neighbouring elements of each of their rows of B, as in `down`.  The next columns' rows of B are
// loaded before the present ones are used.
constexpr int kUpFewThreads = 256, kUpFewWarps = kUpFewThreads / 32;

// W: elements of a row of B a thread loads at a time, by 4 threads: 16, 32 or 64 ranks a pass
template <int W>
__global__ void __launch_bounds__(kUpFewThreads, 2) adapter_up_few_kernel(const AdapterArgs a) {
  constexpr int kPass = W * 4, kMma = W / 4;  // ranks of a pass, its MMAs of 16
  extern __shared__ __align__(16) unsigned char up_few_smem[];  // hi, lo of [16][pitch] ranks
  __shared__ int tok[16];
  __shared__ float back[16];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  if (!plan_fits(a)) return;
  const int tiles = a.plan->tiles[a.up_kind], units = (a.N + 31) / 32, passes = (a.R + kPass - 1) / kPass;
  const int pitch = passes * kPass * 2 + 16;  // bytes of a token's hi or lo
  const int64_t all = (int64_t)tiles * units;
  int64_t at = all * blockIdx.x / gridDim.x;
  const int64_t stop = all * (blockIdx.x + 1) / gridDim.x;
  bool waited = false;
  while (at < stop) {
    const int tile = (int)(at / units), begin = (int)(at - (int64_t)tile * units);
    const int end = (int)(stop - at < units - begin ? begin + (stop - at) : units);
    at += end - begin;
    const AdapterTile t = a.up_tiles[tile];
    const int live = live_rank(a, t.adapter);
    if (live == 0 && a.out == a.y) continue;
    const __half* b = a.b + (int64_t)min(t.adapter, a.n - 1) * a.N * a.R + c * W;
    uint32_t w[4][W / 2], next[4][W / 2];
    auto load = [&](uint32_t (&v)[4][W / 2], int u, int pass) {  // rows 4 g .. + 3 of unit u
      const int r = pass * kPass;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int row = u * 32 + 4 * g + j;
#pragma unroll
        for (int i = 0; i < W; i += 8) {
          const int left = row < a.N ? live - r - c * W - i : 0;
          const __half* p = b + (int64_t)row * a.R + r + i;
          if constexpr (W == 4) {
            const uint2 q = left > 0 ? __ldg(reinterpret_cast<const uint2*>(p)) : make_uint2(0, 0);
            v[j][0] = q.x, v[j][1] = q.y;
          } else {
            const uint4 q = left > 0 ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0);
            v[j][i / 2] = q.x, v[j][i / 2 + 1] = q.y, v[j][i / 2 + 2] = q.z, v[j][i / 2 + 3] = q.w;
          }
        }
      }
    };
    auto cut = [&](uint32_t (&v)[4][W / 2], int pass) {  // what the rank ends inside a thread's elements
      const int left = live - pass * kPass - c * W;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < W / 2; ++i) v[j][i] = left <= 2 * i ? 0u : left == 2 * i + 1 ? v[j][i] & 0xffffu : v[j][i];
    };
    int u = begin + warp;
    if (live && u < end) load(w, u, 0);
    __syncthreads();  // the tile before is done
    if (tid < 16) tok[tid] = tid < t.count ? a.order[t.first + tid] : -1;
    if (live) {
      if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");  // h is written
      waited = true;
      const int p = tid >> 4, q = tid & 15;  // 16 threads a token
      const float* h = a.h + (int64_t)(t.first + min(p, t.count - 1)) * a.R;
      float top = 0.f;
      for (int r = q * 4; r < live; r += 64) {
        const float4 v = *reinterpret_cast<const float4*>(h + r);
        top = fmaxf(fmaxf(top, fmaxf(fabsf(v.x), fabsf(v.y))), fmaxf(fabsf(v.z), fabsf(v.w)));
      }
#pragma unroll
      for (int d = 8; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      float bk;
      const float up = up_scale(top, bk);
      if (q == 0) back[p] = bk;
      for (int r = q * 4; r < passes * kPass; r += 64) {
        const float4 v = p < t.count && r < a.R ? *reinterpret_cast<const float4*>(h + r) : make_float4(0, 0, 0, 0);
        uint2 hi, lo;
        two_terms(v, up, hi, lo);
        *reinterpret_cast<uint2*>(up_few_smem + p * pitch + r * 2) = hi;
        *reinterpret_cast<uint2*>(up_few_smem + (16 + p) * pitch + r * 2) = lo;
      }
    }
    __syncthreads();
    const int nt = t.count > 8 ? 2 : 1;
    int my_tok[4];
    float my_back[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // tokens 2 c, 2 c + 1 of each eight
      const int p = (i >> 1) * 8 + 2 * c + (i & 1);
      my_tok[i] = tok[p];
      my_back[i] = live ? back[p] : 0.f;
    }
    const uint32_t terms = smem_u32(up_few_smem) + g * pitch + c * W * 2;
    for (; u < end; u += kUpFewWarps) {
      const int col = u * 32 + 4 * g;
      uint2 y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (my_tok[i] >= 0 && col < a.N) y[i] = *reinterpret_cast<const uint2*>(a.y + my_tok[i] * a.ldy + col);
      float acc[2][2][4];  // [rows 4 g, 4 g + 1 or 4 g + 2, 4 g + 3][eight tokens]
#pragma unroll
      for (int i = 0; i < 16; ++i) (&acc[0][0][0])[i] = 0.f;
      for (int pass = 0; pass * kPass < live; ++pass) {
        if ((pass + 1) * kPass < live) load(next, u, pass + 1);
        else if (u + kUpFewWarps < end) load(next, u + kUpFewWarps, 0);
        if (live & 7) cut(w, pass);
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          if (n >= nt) break;
#pragma unroll
          for (int term = 1; term >= 0; --term) {
            uint32_t h[W / 2];
            const uint32_t p = terms + (n * 8 + term * 16) * pitch + pass * kPass * 2;
            if constexpr (W == 4) {
              const uint2 v = ld_shared_v2(p);
              h[0] = v.x, h[1] = v.y;
            } else {
#pragma unroll
              for (int i = 0; i < W / 8; ++i) {
                const uint4 v = ld_shared_v4(p + i * 16);
                h[4 * i] = v.x, h[4 * i + 1] = v.y, h[4 * i + 2] = v.z, h[4 * i + 3] = v.w;
              }
            }
#pragma unroll
            for (int m = 0; m < kMma; ++m)
#pragma unroll
              for (int q = 0; q < 2; ++q)
                mma_16816(acc[q][n], w[2 * q][2 * m], w[2 * q + 1][2 * m], w[2 * q][2 * m + 1], w[2 * q + 1][2 * m + 1], h[2 * m], h[2 * m + 1]);
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < W / 2; ++i) w[j][i] = next[j][i];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (my_tok[i] < 0 || col >= a.N) continue;
        uint2 o = y[i];
        if (live) {
          const int n = i >> 1, k = i & 1;
          const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&y[i].x)), hi = __half22float2(*reinterpret_cast<const __half2*>(&y[i].y));
          const float f = my_back[i];
          o.x = pack_half2(fmaf(acc[0][n][k], f, lo.x), fmaf(acc[0][n][2 + k], f, lo.y));
          o.y = pack_half2(fmaf(acc[1][n][k], f, hi.x), fmaf(acc[1][n][2 + k], f, hi.y));
        }
        *reinterpret_cast<uint2*>(a.out + my_tok[i] * a.ldo + col) = o;
      }
    }
  }
}

// ---------------------------------------------------------------- up, many tokens
// A CTA takes a tile of at most 128 tokens and a run of column tiles of 64, a warp 16 of the tokens.  A thread keeps its
// tokens' terms as the mma's left operand (up to 64 ranks; above, they are read from shared memory), and B's rows
// come by cp.async two column tiles ahead.  Which column of out is which of the MMAs' columns is free: thread (g, c)
// has 16 neighbouring ones of tokens g and g + 8, so that y and out go between global memory and registers in whole
// sectors, y one column tile ahead.
constexpr int kUpThreads = 256, kUpCols = 64, kUpStages = 3;

// bytes of a row of B in shared memory: an odd number of 32, so that four rows' 32 bytes lie in different banks
__host__ __device__ __forceinline__ int up_pitch(int R) { return ((R + 15) / 16 | 1) * 32; }

// KS: steps of 16 ranks; kept in registers up to 4
template <int KS>
__global__ void __launch_bounds__(kUpThreads, KS <= 8 ? 2 : 1) adapter_up_many_kernel(const AdapterArgs a) {
  constexpr bool kKeep = KS <= 4;
  extern __shared__ __align__(128) unsigned char up_smem[];
  if (!plan_fits(a)) return;
  const int tile = blockIdx.x, group = blockIdx.y;  // tiles first: those of one adapter read the same rows of B
  if (tile >= a.plan->tiles[a.up_kind]) return;
  const AdapterTile t = a.up_tiles[tile];
  const int live = live_rank(a, t.adapter);
  if (live == 0 && a.out == a.y) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const int pitch = up_pitch(a.R), ks = (live + 15) >> 4, pieces = a.R >> 3;
  const uint32_t base = smem_u32(up_smem), stage_bytes = kUpCols * pitch, terms_at = base + kUpStages * stage_bytes;
  const int tiles = (a.N + kUpCols - 1) / kUpCols;
  const int begin = (int)((int64_t)tiles * group / a.groups), end = (int)((int64_t)tiles * (group + 1) / a.groups);

  // column 16 c + 2 j + i of a tile is column 2 c + i of MMA j: its row of B lies at 8 j + 2 c + i
  const __half* bg = a.b + (int64_t)min(t.adapter, a.n - 1) * a.N * a.R;
  auto fetch = [&](int nt) {
    const uint32_t st = base + (nt - begin) % kUpStages * stage_bytes;
    const int rows = min(kUpCols, a.N - nt * kUpCols);
    const __half* src = bg + (int64_t)nt * kUpCols * a.R;
    for (int i = tid; i < rows * pieces; i += kUpThreads) {  // (a tile's rows of B are one run of memory)
      const int col = i / pieces, p = i - col * pieces;
      const int at = (col >> 1 & 7) * 8 + (col >> 4) * 2 + (col & 1);
      if (p * 8 < live) cp_async16(st + at * pitch + p * 16, src + i * 8, 16);
    }
  };
  const int p0 = warp * 16 + g;  // the thread's tokens: p0 and p0 + 8 of the tile
  int tok[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) tok[i] = p0 + 8 * i < t.count ? a.order[t.first + p0 + 8 * i] : -1;
  uint4 y[2][2];
  auto load_y = [&](uint4 (&v)[2][2], int nt) {
    const int col = nt * kUpCols + 16 * c;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int q = 0; q < 2; ++q)
        if (tok[i] >= 0 && col + 8 * q < a.N) v[i][q] = __ldcs(reinterpret_cast<const uint4*>(a.y + tok[i] * a.ldy + col) + q);
  };
  if (live) {
#pragma unroll
    for (int i = 0; i < kUpStages - 1; ++i) {
      if (begin + i < end) fetch(begin + i);
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  }
  load_y(y, begin);
  uint32_t hi[kKeep ? KS : 1][4], lo[kKeep ? KS : 1][4];
  float back[2];
  if (live) {
    asm volatile("griddepcontrol.wait;" ::: "memory");  // h is written
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float* h = a.h + (int64_t)(t.first + min(p0 + 8 * i, t.count - 1)) * a.R;
      float top = 0.f;
      for (int r = 4 * c; r < live; r += 16) {
        const float4 v = *reinterpret_cast<const float4*>(h + r);
        top = fmaxf(fmaxf(top, fmaxf(fabsf(v.x), fabsf(v.y))), fmaxf(fabsf(v.z), fabsf(v.w)));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const float up = up_scale(top, back[i]);
      // ranks 16 k + 4 c .. + 3 serve as the k's 2 c, 2 c + 1, 2 c + 8, 2 c + 9; B's are permuted below alike
      auto at_step = [&](int k, uint2& h2, uint2& l2) {
        const int r = 16 * k + 4 * c;
        two_terms(r < a.R ? *reinterpret_cast<const float4*>(h + r) : make_float4(0, 0, 0, 0), up, h2, l2);
      };
      if constexpr (kKeep) {
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          uint2 h2, l2;
          at_step(k, h2, l2);
          hi[k][i] = h2.x, hi[k][i + 2] = h2.y;
          lo[k][i] = l2.x, lo[k][i + 2] = l2.y;
        }
      } else {
        for (int k = 0; k < ks; ++k) {  // a lane's own 16 bytes of each term a step
          uint2 h2, l2;
          at_step(k, h2, l2);
          uint32_t* p = reinterpret_cast<uint32_t*>(up_smem + kUpStages * stage_bytes + (((warp * KS + k) * 2) * 32 + lane) * 16);
          p[i] = h2.x, p[i + 2] = h2.y;
          p[i + 128] = l2.x, p[i + 130] = l2.y;
        }
      }
    }
  }
  // the rank's end inside a step: what B holds behind it
  const int left = live - (ks - 1) * 16 - 4 * c;
  const uint32_t m0 = left <= 0 ? 0u : left == 1 ? 0xffffu : ~0u, m1 = left <= 2 ? 0u : left == 3 ? 0xffffu : ~0u;
  for (int nt = begin; nt < end; ++nt) {
    uint4 next[2][2];
    float acc[8][4];
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
    if (nt + 1 < end) load_y(next, nt + 1);
    if (live) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kUpStages - 2) : "memory");
      __syncthreads();  // tile nt is there, and tile nt - 1 has been used
      if (nt + kUpStages - 1 < end) fetch(nt + kUpStages - 1);
      asm volatile("cp.async.commit_group;" ::: "memory");
      const uint32_t st = base + (nt - begin) % kUpStages * stage_bytes + g * pitch + c * 8;
      auto step = [&](int k, const uint32_t (&h)[4], const uint32_t (&l)[4], bool last) {
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          uint2 b = ld_shared_v2(st + n * 8 * pitch + k * 32);
          if (last) b.x &= m0, b.y &= m1;
          mma_16816(acc[n], l[0], l[1], l[2], l[3], b.x, b.y);
          mma_16816(acc[n], h[0], h[1], h[2], h[3], b.x, b.y);
        }
      };
      if (warp * 16 < t.count) {
        if constexpr (kKeep) {
#pragma unroll
          for (int k = 0; k < KS; ++k)
            if (k < ks) step(k, hi[k], lo[k], k == ks - 1);
        } else {
          for (int k = 0; k < ks; ++k) {
            uint32_t h[4], l[4];
            const uint32_t p = terms_at + (((warp * KS + k) * 2) * 32 + lane) * 16;
            const uint4 u = ld_shared_v4(p), v = ld_shared_v4(p + 512);
            h[0] = u.x, h[1] = u.y, h[2] = u.z, h[3] = u.w;
            l[0] = v.x, l[1] = v.y, l[2] = v.z, l[3] = v.w;
            step(k, h, l, k == ks - 1);
          }
        }
      }
    }
    const int col = nt * kUpCols + 16 * c;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        if (tok[i] < 0 || col + 8 * q >= a.N) continue;
        uint4 o = y[i][q];
        if (live) {
          uint32_t* w = reinterpret_cast<uint32_t*>(&o);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
            w[j] = pack_half2(fmaf(acc[4 * q + j][2 * i], back[i], f.x), fmaf(acc[4 * q + j][2 * i + 1], back[i], f.y));
          }
        }
        __stcs(reinterpret_cast<uint4*>(a.out + tok[i] * a.ldo + col) + q, o);
      }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int q = 0; q < 2; ++q) y[i][q] = next[i][q];
  }
}

static size_t up_many_smem(int R) {
  const size_t pitch = up_pitch(R);
  const int steps = R <= 64 ? 0 : R <= 128 ? 8 : 16;
  return kUpStages * kUpCols * pitch + (size_t)steps * 8 * 2 * 512;
}

template <typename... Args>
static cudaError_t launch(void (*fn)(Args...), dim3 grid, int threads, size_t smem, cudaStream_t s, int cluster, bool dependent, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  int n = 0;
  if (cluster > 1) {
    at[n].id = cudaLaunchAttributeClusterDimension;
    at[n].val.clusterDim.x = (unsigned)cluster;
    at[n].val.clusterDim.y = at[n].val.clusterDim.z = 1;
    ++n;
  }
  if (dependent) {
    at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = at;
  cfg.numAttrs = (unsigned)n;
  return cudaLaunchKernelEx(&cfg, fn, args...);
}

// Up to this many tokens of a step the tiles are of 16.
constexpr int kFewTokens = 256;

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
  int rc = device_facts(&f);
  if (rc != TB_OK) return rc;
  AdapterArgs g;
  g.x = reinterpret_cast<const __half*>(x);
  g.a = reinterpret_cast<const __half*>(a);
  g.b = reinterpret_cast<const __half*>(b);
  g.y = reinterpret_cast<const __half*>(y);
  g.out = reinterpret_cast<__half*>(out);
  g.rank = rank;
  g.scale = scale;
  const bool few = T <= kFewTokens;
  g.down_kind = few ? 0 : 1;
  g.up_kind = few ? 0 : 2;
  const char* base = static_cast<const char*>(plan);
  g.plan = static_cast<const AdapterPlan*>(plan);
  g.order = reinterpret_cast<const int32_t*>(base + adapter_order_at());
  g.down_tiles = reinterpret_cast<const AdapterTile*>(base + adapter_tiles_at(T, n, g.down_kind));
  g.up_tiles = reinterpret_cast<const AdapterTile*>(base + adapter_tiles_at(T, n, g.up_kind));
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
  const int64_t down = adapter_max_tiles(T, n, g.down_kind), up = adapter_max_tiles(T, n, g.up_kind);
  // few tokens: K is split over a cluster until there are two CTAs an SM, of at least four steps a warp; many: until
  // every SM has one
  g.cluster = 1;
  if (few)
    while (g.cluster < 8 && down * g.cluster < 2 * f.sms && K / 32 >= g.cluster * 2 * kDownWarps) g.cluster *= 2;
  else
    while (g.cluster < 8 && down * g.cluster * 2 <= 2 * f.sms && K / 64 >= g.cluster * 2 * kStages) g.cluster *= 2;
  const int nt = R <= 16 ? 2 : R <= 32 ? 4 : 8;
  const dim3 grid((unsigned)(down * g.cluster), (unsigned)((R + nt * 8 - 1) / (nt * 8)));
  cudaError_t e;
#define TB_DOWN_FEW(NT) launch(adapter_down_few_kernel<NT>, grid, kDownThreads, (size_t)kDownWarps * 16 * NT * 8 * 4, s, g.cluster, false, g)
#define TB_DOWN_MANY(NT)                                                                                                        \
  ((rc = ensure_dynamic_smem(reinterpret_cast<const void*>(adapter_down_many_kernel<NT>), f.device, down_many_smem<NT>())) != TB_OK \
       ? cudaErrorUnknown                                                                                                       \
       : launch(adapter_down_many_kernel<NT>, grid, kDownThreads, (size_t)down_many_smem<NT>(), s, g.cluster, false, g))
  if (few)
    e = nt == 2 ? TB_DOWN_FEW(2) : nt == 4 ? TB_DOWN_FEW(4) : TB_DOWN_FEW(8);
  else
    e = nt == 2 ? TB_DOWN_MANY(2) : nt == 4 ? TB_DOWN_MANY(4) : TB_DOWN_MANY(8);
#undef TB_DOWN_FEW
#undef TB_DOWN_MANY
  if (rc != TB_OK) return rc;
  if (e == cudaSuccess) {
    if (few) {
      // two CTAs an SM share all tiles' columns; at least 128 columns each
      const int W = R <= 16 ? 4 : R <= 32 ? 8 : 16;
      const size_t smem = (size_t)32 * ((R + W * 4 - 1) / (W * 4) * W * 8 + 16);
      int64_t ctas = up * ((N + 127) / 128);
      if (ctas > 2 * f.sms) ctas = 2 * f.sms;
      const dim3 some((unsigned)ctas);
      e = W == 4   ? launch(adapter_up_few_kernel<4>, some, kUpFewThreads, smem, s, 1, true, g)
          : W == 8 ? launch(adapter_up_few_kernel<8>, some, kUpFewThreads, smem, s, 1, true, g)
                   : launch(adapter_up_few_kernel<16>, some, kUpFewThreads, smem, s, 1, true, g);
    } else {
      const size_t smem = up_many_smem((int)R);
      // several CTAs a row tile, each with a run of column tiles
      const int64_t col_tiles = (N + kUpCols - 1) / kUpCols;
      int64_t groups = (6ll * f.sms + up - 1) / up;
      g.groups = (int)(groups < 1 ? 1 : groups > col_tiles ? col_tiles : groups);
      const dim3 some((unsigned)up, (unsigned)g.groups);
#define TB_UP(KS)                                                                                                           \
  ((rc = ensure_dynamic_smem(reinterpret_cast<const void*>(adapter_up_many_kernel<KS>), f.device, (int)smem)) != TB_OK \
       ? cudaErrorUnknown                                                                                                   \
       : launch(adapter_up_many_kernel<KS>, some, kUpThreads, smem, s, 1, true, g))
      e = R <= 16 ? TB_UP(1) : R <= 32 ? TB_UP(2) : R <= 64 ? TB_UP(4) : R <= 128 ? TB_UP(8) : TB_UP(16);
#undef TB_UP
      if (rc != TB_OK) return rc;
    }
  }
  if (e != cudaSuccess) {
    record_cuda_error(e);
    return TB_ERR_CUDA;
  }
  return check_launch();
}
