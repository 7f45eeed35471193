// Low-rank adapters of many requests beside a shared linear: out[t] = y[t] + scale[g] B[g] (A[g] x[t]), g the
// adapter of token t's request.
//
// Two launches, the second (programmatic) beside the first, loading what that does not write before it waits for it:
//   down  h = scale A x, to the workspace in the plan's order; few tokens: mma.sync on tiles of 16 tokens of one adapter;
//         many: tcgen05 on tiles of 128
//   up    out = y + B h, mma.sync; few tokens: tiles of 16, bound by the weights, which go from global memory straight
//         to the registers; many: tiles of 128, bound by y and out
//
// h goes from one to the other as fp16 in two terms, h 2^e = hi + lo 2^-12, with 2^e of the token's own for up to 64 ranks
// (their largest |h| 2^e in [2^14, 2^15)).  What hi leaves is at most 2^3 there, and less in proportion below, so that lo
// holds 11 bits more of it wherever hi is a normal number: h is off by at most 2^-22 of itself or 2^-51 of that largest, the
// greater of the two (hi + lo at one scale is off by 2^-40 of the largest: half a thousandth of an h that is 2^-29 of it,
// all that a column has whose B is 0 for the largest).  Products and sums are fp32; the
// sum with lo takes 2^-12 before it meets that with hi, and 2^-e is applied to both.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <limits.h>

#include "tb_adapter.cuh"
#include "tb_attn_tc.cuh"
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
  const AdapterTile* tiles;
  __half* terms;  // [T][blocks][hi, lo][block]
  float* back;    // [T][blocks], 2^-e
  int32_t* status;
  int64_t ldx, ldy, ldo;
  int T, n, K, N, R;
  int block, blocks;  // ranks of a block (16, 32 or 64), blocks of R
  int cluster, kind;  // CTAs that share out K, kind of tiles
};

TB_DEVI bool plan_fits(const AdapterArgs& a) {
  const AdapterPlan& p = *a.plan;
  return p.magic == kAdapterMagic && p.T == a.T && p.n == a.n;
}

TB_DEVI int live_rank(const AdapterArgs& a, int g) {
  const int r = a.rank ? a.rank[g] : a.R;
  return r < 0 ? 0 : min(r, a.R);
}

TB_DEVI void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the same with no sum before it
TB_DEVI void mma_16816_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

TB_DEVI void cp_async16(uint32_t dst, const void* src, int bytes) {  // the rest of the 16 bytes is zeroed
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// ---------------------------------------------------------------- h as fp16
constexpr float kLowScale = 0x1p12f;  // of the low terms
// 2^e and 2^-e for numbers of which the largest finite |h| is top
TB_DEVI float up_scale(float top, float& back) {
  int e = 14 - ((int)(__float_as_uint(top) >> 23) - 127);
  if (!(top > 0.f)) e = 0;
  e = max(-126, min(126, e));
  back = __uint_as_float((uint32_t)(127 - e) << 23);
  return __uint_as_float((uint32_t)(127 + e) << 23);
}

// ---------------------------------------------------------------- down
// Parts of a tile's h, [PARTS][M][PITCH] in shared memory, summed in their order, then over the cluster's CTAs in theirs;
// each CTA has some of the rows, a warp one at a time.
template <int PARTS, int M, int N, int PITCH, int THREADS>
TB_DEVI void join_down(const AdapterArgs& a, const AdapterTile& t, float* part, int share, int r0, int live) {
  const int tid = threadIdx.x, lane = tid & 31;
  const float scale = a.scale[t.adapter];
  if constexpr (PARTS > 1) {
    __syncthreads();
    for (int e = tid; e < M * PITCH; e += THREADS) {
      float s = part[e];
#pragma unroll
      for (int w = 1; w < PARTS; ++w) s += part[w * M * PITCH + e];
      part[e] = s;
    }
  }
  cg::cluster_group cl = cg::this_cluster();
  if (a.cluster > 1) cl.sync();
  else __syncthreads();
  const int rows = M / a.cluster;
  for (int i = tid >> 5; i < rows; i += THREADS / 32) {
    const int row = share * rows + i;
    if (row >= t.count) break;
    constexpr int kCols = (N + 31) / 32;
    float v[kCols], top = 0.f;
#pragma unroll
    for (int j = 0; j < kCols; ++j) {
      const int col = lane + 32 * j;
      v[j] = 0.f;
      if (col < N && r0 + col < live) {
        float s = 0.f;
        for (int r = 0; r < a.cluster; ++r) s += a.cluster > 1 ? *cl.map_shared_rank(part + row * PITCH + col, r) : part[row * PITCH + col];
        v[j] = s * scale;
      }
      top = fmaxf(top, fabsf(v[j]) < INFINITY ? fabsf(v[j]) : 0.f);  // (what is not finite stays so at any scale)
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    float back;
    const float up = up_scale(top, back);
    const int64_t at = (int64_t)(t.first + row) * a.blocks + blockIdx.y;
    if (lane == 0) a.back[at] = back;
#pragma unroll
    for (int j = 0; j < kCols; ++j) {
      const int col = lane + 32 * j;
      const __half hi = __float2half_rn(v[j] * up);
      const float f = __half2float(hi);
      if (col < N) {
        a.terms[at * 2 * N + col] = hi;
        a.terms[at * 2 * N + N + col] = fabsf(f) < INFINITY ? __float2half_rn((v[j] * up - f) * kLowScale) : __half();
      }
    }
  }
  if (a.cluster > 1) cl.sync();  // the parts stay until they have been read
}

// Few tokens: a CTA takes 16 tokens by NT x 8 rows of A; its warps and those of its cluster share out K in steps of
// 32.  Thread (g, c) of a warp takes 8 neighbouring elements of rows g (and g + 8), which serve as the k's 2c, 2c + 1,
// 2c + 8 and 2c + 9 of two MMAs: a product over k does not mind their order, if both operands have the same.  They
// come by cp.async into a ring of the thread's own, so that several steps are in flight without registers, and no thread
// waits for another.  Bound by latency (first loads, join over the cluster): 64 tokens of K 5120, ranks up to 32 of 48
// adapters, 10 MB in 9.7 us; both launches, 47 MB, 19.2 us in a graph, 2.5 TB/s.
constexpr int kDownThreads = 256, kDownWarps = kDownThreads / 32;
constexpr int few_stages(int NT) { return NT == 2 ? 5 : NT == 4 ? 4 : 2; }
template <int NT>
constexpr int down_few_smem() {
  const int ring = few_stages(NT) * (2 + NT) * kDownThreads * 16, parts = kDownWarps * 16 * NT * 8 * 4;
  return ring > parts ? ring : parts;
}

template <int NT>
__global__ void __launch_bounds__(kDownThreads, 2) adapter_down_few_kernel(const AdapterArgs a) {
  constexpr int N = NT * 8, S = few_stages(NT);
  extern __shared__ __align__(128) unsigned char down_smem[];
  asm volatile("griddepcontrol.wait;" ::: "memory");  // what came before is over (see launch_early), for the second launch too
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tile = blockIdx.x / a.cluster, share = blockIdx.x - tile * a.cluster;
  if (!plan_fits(a)) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) set_status(a.status, TB_DEV_BAD_PLAN);
    return;
  }
  if (tile >= a.plan->tiles[a.kind]) return;  // (all CTAs of the cluster)
  const AdapterTile t = a.tiles[tile];  // (not before the plan is known to be one of T tokens)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const int r0 = blockIdx.y * N, live = live_rank(a, t.adapter);

  const __half* xr[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) xr[i] = i * 8 + g < t.count ? a.x + a.order[t.first + i * 8 + g] * a.ldx + c * 8 : nullptr;
  const __half* ar = a.a + ((int64_t)t.adapter * a.R + r0 + g) * a.K + c * 8;
  float acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
  const int steps = (a.K + 31) >> 5, stride = a.cluster * kDownWarps, s0 = share * kDownWarps + warp;
  const uint32_t ring = smem_u32(down_smem) + tid * 16;
  auto piece = [&](int stage, int i) { return ring + (stage * (2 + NT) + i) * kDownThreads * 16; };
  if (r0 < live) {
    auto fetch = [&](int s, int stage) {
      const int k = s * 32;
      const bool in = k + c * 8 < a.K;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (i == 0 || t.count > 8) {
          const bool have = in && xr[i];
          cp_async16(piece(stage, i), have ? xr[i] + k : a.x, have ? 16 : 0);
        }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const bool have = in && r0 + n * 8 + g < live;
        cp_async16(piece(stage, 2 + n), have ? ar + (int64_t)n * 8 * a.K + k : a.a, have ? 16 : 0);
      }
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) {
      if (s0 + i * stride < steps) fetch(s0 + i * stride, i);
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
    int stage = 0;
    for (int s = s0; s < steps; s += stride) {
      const int ahead = s + (S - 1) * stride;
      if (ahead < steps) fetch(ahead, stage == 0 ? S - 1 : stage - 1);
      asm volatile("cp.async.commit_group;" ::: "memory");
      asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
      const uint4 p = ld_shared_v4(piece(stage, 0)), q = t.count > 8 ? ld_shared_v4(piece(stage, 1)) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint4 w = ld_shared_v4(piece(stage, 2 + n));
        mma_16816(acc[n], p.x, q.x, p.y, q.y, w.x, w.y);
        mma_16816(acc[n], p.z, q.z, p.w, q.w, w.z, w.w);
      }
      stage = stage == S - 1 ? 0 : stage + 1;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();  // the ring's place is the parts' now
  }
  float* part = reinterpret_cast<float*>(down_smem) + warp * 16 * N;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    *reinterpret_cast<float2*>(part + g * N + n * 8 + 2 * c) = make_float2(acc[n][0], acc[n][1]);
    *reinterpret_cast<float2*>(part + (g + 8) * N + n * 8 + 2 * c) = make_float2(acc[n][2], acc[n][3]);
  }
  join_down<kDownWarps, 16, N, N, kDownThreads>(a, t, reinterpret_cast<float*>(down_smem), share, r0, live);
}

// Many tokens: a CTA takes 128 tokens by N rows of A, on tcgen05 with the sums in tensor memory.  Eight warps bring both
// operands to shared memory by cp.async (the tokens lie anywhere, and what is not there is zeroed), 64 of K a stage, in the
// 128-byte swizzle that the MMA's descriptors name (16-byte piece ^ row mod 8); when a thread's part of a stage has come it
// counts itself on the stage's barrier, two stages later than it asked for it.  The ninth warp's first lane issues the MMAs.
// With mma.sync instead (64 tokens a CTA), every warp took 100 instructions a stage at 11 clocks each: 28 us for 5935
// tokens of K 5120 and 64 ranks, 52 for 8192 of K 17408 and 16.  So 21.7 us for the first, 64 MB at 2.9 TB/s (0.43 of
// measured HBM): one wave of CTAs, of whose time first loads and join are a third and the MMAs a tenth.
constexpr int kManyThreads = kDownThreads + 32, kManyRows = 128, kManyLag = 2;
constexpr int many_stages(int N) { return N == 64 ? 4 : 5; }
template <int N>
constexpr int down_many_smem() {
  return 1024 + many_stages(N) * (kManyRows + N) * 128;
}

template <int N>
__global__ void __launch_bounds__(kManyThreads, 2) adapter_down_many_kernel(const AdapterArgs a) {
  constexpr int S = many_stages(N), kStageBytes = (kManyRows + N) * 128, kCols = N < 32 ? 32 : N, kPitch = N + 4;
  constexpr uint32_t kInstr = 1u << 4 | (uint32_t)(N / 8) << 17 | (uint32_t)(kManyRows / 16) << 24;  // fp16 operands, fp32 sums
  static_assert(kManyRows * kPitch * 4 <= S * kStageBytes, "the sums take the stages' place");
  extern __shared__ __align__(1024) unsigned char tile_smem[];
  __shared__ uint64_t full[S], empty[S], done;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int aborted;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // what came before is over (see launch_early), for the second launch too
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tile = blockIdx.x / a.cluster, share = blockIdx.x - tile * a.cluster;
  if (!plan_fits(a)) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) set_status(a.status, TB_DEV_BAD_PLAN);
    return;
  }
  if (tile >= a.plan->tiles[a.kind]) return;  // (all CTAs of the cluster)
  const AdapterTile t = a.tiles[tile];  // (not before the plan is known to be one of T tokens)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r0 = blockIdx.y * N, live = live_rank(a, t.adapter);
  unsigned char* const stages = tile_smem + ((1024 - (smem_u32(tile_smem) & 1023)) & 1023);
  const uint32_t base = smem_u32(stages);
  const int steps = (a.K + 63) >> 6, mine = r0 < live ? (steps - share + a.cluster - 1) / a.cluster : 0;
  if (tid == 0) {
    aborted = 0;
    for (int i = 0; i < S; ++i) {
      mbar_init(full + i, kDownThreads);
      mbar_init(empty + i, 1);
    }
    mbar_init(&done, 1);
    fence_barrier_init();
  }
  if (warp == kDownWarps) tmem_alloc(&tmem_slot, kCols);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t sums = tmem_slot;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity) || aborted) return;
    if (!mbar_wait(bar, parity)) {
      aborted = 1;
      set_status(a.status, TB_DEV_TIMEOUT);
    }
  };
  if (warp < kDownWarps) {
    // a thread's pieces of a stage: four of x, N / 32 of A
    const int row = tid >> 3, piece = tid & 7;
    const uint32_t at = row * 128 + ((piece ^ (row & 7)) << 4);
    const __half* xp[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) xp[i] = row + 32 * i < t.count ? a.x + a.order[t.first + row + 32 * i] * a.ldx + piece * 8 : nullptr;
    const __half* ap = a.a + ((int64_t)t.adapter * a.R + r0 + row) * a.K + piece * 8;
    int stage = 0, uses = 0, ready = 0;  // the stage asked for next, its uses before, the stage that has come next
    for (int i = 0; i < mine + kManyLag; ++i) {
      if (i < mine) {
        if (uses > 0) wait(empty + stage, (uses - 1) & 1);
        const int k = (share + i * a.cluster) * 64;
        const uint32_t dst = base + stage * kStageBytes + at;
        const bool in = k + piece * 8 < a.K;
#pragma unroll
        for (int j = 0; j < 4; ++j) cp_async16(dst + j * 32 * 128, xp[j] && in ? xp[j] + k : a.x, xp[j] && in ? 16 : 0);
#pragma unroll
        for (int j = 0; j < (N + 31) / 32; ++j)
          if (N >= 32 || row < N) {
            const bool have = in && r0 + row + j * 32 < live;
            cp_async16(dst + (kManyRows + j * 32) * 128, have ? ap + (int64_t)j * 32 * a.K + k : a.a, have ? 16 : 0);
          }
        if (++stage == S) stage = 0, ++uses;
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      if (i >= kManyLag) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kManyLag) : "memory");
        fence_proxy_async_smem();
        mbar_arrive(full + ready);
        ready = ready == S - 1 ? 0 : ready + 1;
      }
    }
  } else if (lane == 0) {
    for (int i = 0; i < mine; ++i) {
      const int stage = i % S;
      wait(full + stage, i / S & 1);
      tmem_fence_after();
      const uint64_t x = smem_desc_sw128(base + stage * kStageBytes, 1024), w = smem_desc_sw128(base + stage * kStageBytes + kManyRows * 128, 1024);
#pragma unroll
      for (int k = 0; k < 4; ++k) mma_f16_ss<1>(sums, x + 2 * k, w + 2 * k, kInstr, i > 0 || k > 0);
      mma_commit(empty + stage);
    }
    if (mine) mma_commit(&done);
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncwarp();
  if (mine) wait(&done, 0);
  tmem_fence_after();
  __syncthreads();  // the stages' place is the sums' now
  // warp w: tokens 32 w .. of the tile, a lane each
  float* const part = reinterpret_cast<float*>(stages);
  if (warp < 4) {
    float v[N];
    if (mine) {
      if constexpr (N == 16) {
        tmem_ld8(sums + ((uint32_t)(warp * 32) << 16), *reinterpret_cast<float (*)[8]>(v));
        tmem_ld8(sums + ((uint32_t)(warp * 32) << 16) + 8, *reinterpret_cast<float (*)[8]>(v + 8));
      } else {
#pragma unroll
        for (int i = 0; i < N; i += 32) tmem_ld32(sums + ((uint32_t)(warp * 32) << 16) + i, v + i);
      }
      tmem_wait_ld();
    }
#pragma unroll
    for (int i = 0; i < N; i += 4)
      *reinterpret_cast<float4*>(part + tid * kPitch + i) = mine ? make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]) : make_float4(0, 0, 0, 0);
  }
  tmem_fence_before();
  join_down<1, kManyRows, N, kPitch, kManyThreads>(a, t, part, share, r0, live);
  __syncthreads();
  if (warp == kDownWarps) tmem_dealloc(sums, kCols);
}

// ---------------------------------------------------------------- tokens without an adapter
// out = y for them, where out is not y: all threads of a launch, kCopy pieces of 16 bytes each in flight (one after
// another they would take a memory's latency each).
constexpr int kCopy = 4;

TB_DEVI void copy_bare(const AdapterArgs& a) {
  if (a.out == a.y) return;
  const int width = a.N / 8, bare = a.plan->bare;
  const int64_t pieces = (int64_t)(a.plan->rows - bare) * width, threads = (int64_t)gridDim.x * blockDim.x;
  for (int64_t e0 = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; e0 < pieces; e0 += threads * kCopy) {
    uint4 v[kCopy];
    uint4* to[kCopy];
#pragma unroll
    for (int i = 0; i < kCopy; ++i) {
      const int64_t e = e0 + i * threads, p = e / width;
      if (e < pieces) {
        const int64_t tok = a.order[bare + p];
        v[i] = __ldcs(reinterpret_cast<const uint4*>(a.y + tok * a.ldy) + (e - p * width));
        to[i] = reinterpret_cast<uint4*>(a.out + tok * a.ldo) + (e - p * width);
      }
    }
#pragma unroll
    for (int i = 0; i < kCopy; ++i)
      if (e0 + i * threads < pieces) __stcs(to[i], v[i]);
  }
}

// ---------------------------------------------------------------- up, few tokens
// The columns of out (rows of B) are the mma's 16 rows and the tokens its 8 columns, so that a weight is read once
// for a tile of 16 tokens and an idle token costs nothing but its place.  A warp takes 32 columns at a time, and
// every warp an equal run of all tiles' columns.  Thread (g, c) holds columns n0 + 4 g .. + 3: 8 bytes of y and out a
// token, and 8 neighbouring elements of each of their rows of B, as in `down`.  The next columns' rows of B and
// elements of y are on their way while the present ones are used.  64 tokens, N 17408, ranks up to 32 of 48 adapters:
// 56 MB in 15.2 us by itself, 3.7 TB/s (three CTAs an SM: 24.8 for both launches against 19.2).
constexpr int kUpFewThreads = 256, kUpFewWarps = kUpFewThreads / 32;

// They come by cp.async into a ring of the thread's own.
constexpr int up_few_stages(int W) { return W == 4 ? 6 : W == 8 ? 4 : 2; }
template <int W>
constexpr int up_few_smem() {
  return up_few_stages(W) * kUpFewThreads * (4 * W * 2 + 4 * 8);
}
TB_DEVI void cp_async8(uint32_t dst, const void* src, int bytes) {  // the rest of the 8 bytes is zeroed
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// W: elements of a row of B a thread loads at a time (16 as twice 8, so that four threads' are 64 bytes in a row), of
// blocks of 16, 32 or 64 ranks; MULTI: several blocks.  An item of the ring is a block of a unit, with the unit's y at its first block.
// 64 tokens of 40 adapters, N 17408: rank 16 15.0 us for both launches in a graph, 64 26.8 (floor 18), 128 51 (35); of 128 registers
// blocks of 64 ranks spill 8 bytes, several 120.
template <int W, bool MULTI>
__global__ void __launch_bounds__(kUpFewThreads, 2) adapter_up_few_kernel(const AdapterArgs a) {
  constexpr int kBlock = W * 4, kMma = W / 4, S = up_few_stages(W);  // ranks of a block, its MMAs of 16
  constexpr int kPieces = W == 16 ? 2 : 1, kBytes = W * 2 / kPieces;  // of a thread's elements of a row
  constexpr int kItem = kUpFewThreads * (4 * W * 2 + 4 * 8);
  extern __shared__ __align__(16) unsigned char up_few_smem_[];
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  if (!plan_fits(a)) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  copy_bare(a);
  const int units = (a.N + 31) / 32;
  const int64_t all = (int64_t)a.plan->tiles[a.kind] * units;
  const int64_t warps = (int64_t)gridDim.x * kUpFewWarps, warp = (int64_t)blockIdx.x * kUpFewWarps + (threadIdx.x >> 5);
  int64_t at = all * warp / warps;
  const int64_t stop = all * (warp + 1) / warps;
  const uint32_t ring = smem_u32(up_few_smem_);
  auto row_at = [&](int stage, int j, int i) { return ring + stage * kItem + (j * kPieces + i) * kUpFewThreads * kBytes + threadIdx.x * kBytes; };
  auto y_at = [&](int stage, int i) { return ring + stage * kItem + 4 * W * 2 * kUpFewThreads + (i * kUpFewThreads + threadIdx.x) * 8; };
  bool waited = false;
  while (at < stop) {
    const int tile = (int)(at / units), begin = (int)(at - (int64_t)tile * units);
    const int end = (int)(stop - at < units - begin ? begin + (stop - at) : units);
    at += end - begin;
    const AdapterTile t = a.tiles[tile];
    const int live = live_rank(a, t.adapter);
    const int half = t.count > 8 ? 4 : 2;  // tokens a thread has: 2 c, 2 c + 1 of each eight
    int64_t yo[4], oo[4];  // where they begin in y and out, -1: no token
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int p = (i >> 1) * 8 + 2 * c + (i & 1);
      yo[i] = oo[i] = -1;
      if (p < t.count) {
        const int64_t k = a.order[t.first + p];
        yo[i] = k * a.ldy + 4 * g, oo[i] = k * a.ldo + 4 * g;
      }
    }
    const __half* b = a.b + (int64_t)t.adapter * a.N * a.R + (int64_t)(4 * g) * a.R + c * (W / kPieces);
    const int blocks = MULTI ? max(1, (live + kBlock - 1) / kBlock) : 1;
    auto fetch = [&](int u, int blk, int stage) {  // rows 4 g .. + 3 of unit u; zeros behind the rank and the last row
      const bool in = u * 32 + 4 * g < a.N;  // (N is a multiple of 8)
      const int left = (live - blk * kBlock - c * (W / kPieces)) * 2;
      const __half* p = b + (int64_t)u * 32 * a.R + blk * kBlock;
#pragma unroll
      for (int j = 0; j < 4; ++j, p += a.R)
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          const int bytes = in ? min(kBytes, max(0, left - i * 64)) : 0;
          if constexpr (W == 4) cp_async8(row_at(stage, j, i), bytes ? p : a.b, bytes);
          else cp_async16(row_at(stage, j, i), bytes ? p + i * 32 : a.b, bytes);
        }
      if (!MULTI || blk == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < half && yo[i] >= 0 && in) cp_async8(y_at(stage, i), a.y + yo[i] + u * 32, 8);
      }
    };
    int fu = begin, fb = 0;  // the next item to fetch
    auto next = [&](int stage) {
      if (fu < end) {
        fetch(fu, fb, stage);
        if (!MULTI || ++fb == blocks) fb = 0, ++fu;
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) next(i);
    if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");  // h is written
    waited = true;
    // the terms of token g of each eight, as the mma's right operand
    auto term = [&](uint32_t (&h)[W / 2], int n, int lo, int blk) {
      const int p = n * 8 + g;
      const __half* q = a.terms + (((int64_t)(t.first + p) * a.blocks + blk) * 2 + lo) * kBlock + c * (W / kPieces);
      if constexpr (W == 4) {
        const uint2 v = p < t.count ? *reinterpret_cast<const uint2*>(q) : make_uint2(0, 0);
        h[0] = v.x, h[1] = v.y;
      } else {
#pragma unroll
        for (int i = 0; i < W / 2; i += 4) {
          const uint4 v = p < t.count ? *reinterpret_cast<const uint4*>(q + i * 8) : make_uint4(0, 0, 0, 0);
          h[i] = v.x, h[i + 1] = v.y, h[i + 2] = v.z, h[i + 3] = v.w;
        }
      }
    };
    auto back = [&](int i, int blk) {
      const int p = (i >> 1) * 8 + 2 * c + (i & 1);
      return p < t.count ? a.back[(int64_t)(t.first + p) * a.blocks + blk] : 0.f;
    };
    uint32_t hi[2][W / 2], lo[2][W / 2];
    float bk[4];
    auto terms = [&](int blk) {
#pragma unroll
      for (int n = 0; n < 2; ++n)
        if (2 * n < half) {
          term(hi[n], n, 0, blk);
          term(lo[n], n, 1, blk);
        }
#pragma unroll
      for (int i = 0; i < 4; ++i) bk[i] = back(i, blk);
    };
    if (!MULTI) terms(0);
    int stage = 0;
    for (int u = begin; u < end; ++u) {
      float sum[4][4];  // [token][column]
      uint2 y[4];
      for (int blk = 0; blk < blocks; ++blk) {
        next(stage == 0 ? S - 1 : stage - 1);
        if (MULTI) terms(blk);
        asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
        uint32_t w[4][W / 2];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (W == 4) {
            const uint2 v = ld_shared_v2(row_at(stage, j, 0));
            w[j][0] = v.x, w[j][1] = v.y;
          } else {
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
              const uint4 v = ld_shared_v4(row_at(stage, j, i));
              w[j][4 * i] = v.x, w[j][4 * i + 1] = v.y, w[j][4 * i + 2] = v.z, w[j][4 * i + 3] = v.w;
            }
          }
        }
        if (!MULTI || blk == 0) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i < half) y[i] = ld_shared_v2(y_at(stage, i));
        }
        stage = stage == S - 1 ? 0 : stage + 1;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          if (2 * n >= half) break;
          float acc[2][4];  // [rows 4 g, 4 g + 1 or 4 g + 2, 4 g + 3]
#pragma unroll
          for (int i = 0; i < 8; ++i) (&acc[0][0])[i] = 0.f;
#pragma unroll
          for (int m = 0; m < kMma; ++m)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              mma_16816(acc[q], w[2 * q][2 * m], w[2 * q + 1][2 * m], w[2 * q][2 * m + 1], w[2 * q + 1][2 * m + 1], lo[n][2 * m], lo[n][2 * m + 1]);
            }
#pragma unroll
          for (int i = 0; i < 8; ++i) (&acc[0][0])[i] *= 1 / kLowScale;
#pragma unroll
          for (int m = 0; m < kMma; ++m)
#pragma unroll
            for (int q = 0; q < 2; ++q)
              mma_16816(acc[q], w[2 * q][2 * m], w[2 * q + 1][2 * m], w[2 * q][2 * m + 1], w[2 * q + 1][2 * m + 1], hi[n][2 * m], hi[n][2 * m + 1]);
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float v = acc[e >> 1][(e & 1) * 2 + k], f = bk[2 * n + k];
              float& s = sum[2 * n + k][e];
              s = MULTI && blk ? fmaf(v, f, s) : v * f;
            }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < half && yo[i] >= 0 && u * 32 + 4 * g < a.N) {
          const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&y[i].x)), q = __half22float2(*reinterpret_cast<const __half2*>(&y[i].y));
          *reinterpret_cast<uint2*>(a.out + oo[i] + u * 32) = make_uint2(pack_half2(p.x + sum[i][0], p.y + sum[i][1]), pack_half2(q.x + sum[i][2], q.y + sum[i][3]));
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  }
  if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");  // no launch is over before the one it began beside
}

// ---------------------------------------------------------------- up, many tokens
// Every CTA takes equal runs of all row tiles' (at most 128 tokens) column tiles of 64, back and forth over them, as tiles
// of few tokens take less time (packed prompts 115 us; 120 with one run a CTA and with four); a warp takes 16 of the tokens.  A
// thread keeps its tokens' terms as the mma's left operand (of up to 64 ranks; above, they are read again); B's rows come
// by cp.async three column tiles ahead, and y into a ring of the thread's own with them.  Which column of out is which of the MMAs' columns is free: thread
// (g, c) has twice 8 neighbouring ones of tokens g and g + 8, so that four threads' y and out are 64 bytes in a row.
// The two terms' sums in registers of their own: packed prompts 121 us in a graph, 115 with one sum for both (see above);
// other orders 122 to 132 (B read twice and one sum scaled between the terms, columns two MMAs at a time).  This launch by
// itself 102 us of them, 387 MB at 3.8 TB/s, the tensor pipe busy 28 % and a thread issuing in 42 % of the cycles.  8192 tokens of one
// adapter, K 5120, N 17408: rank 32 127 us, 64 169, 128 388 (floors 97); ranks of 256, N 5120, four adapters: 322 (40).
constexpr int kUpThreads = 256, kUpCols = 64, kUpRuns = 2;
constexpr int up_stages(bool multi) { return multi ? 3 : 4; }

// bytes of a row of B in shared memory: whole blocks of 16, 32 or 64 ranks, without gaps.  In rows of 128 bytes and more
// the 16-byte pieces of odd rows are exchanged in fours, so that two rows' 64 bytes lie in different banks
__host__ __device__ constexpr int up_pitch(int block, int blocks) { return block * blocks * 2; }
constexpr int kUpY = kUpThreads * 4 * 16;  // bytes of a stage's y

// KS: steps of 16 ranks of a block; MULTI: several blocks
template <int KS, bool MULTI>
__global__ void __launch_bounds__(kUpThreads, 2) adapter_up_many_kernel(const AdapterArgs a) {
  constexpr int S = up_stages(MULTI);
  extern __shared__ __align__(128) unsigned char up_smem[];
  if (!plan_fits(a)) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  copy_bare(a);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const int pitch = up_pitch(KS * 16, MULTI ? a.blocks : 1);
  const uint32_t base = smem_u32(up_smem), y_ring = base + tid * 16, b_ring = base + S * kUpY, stage_bytes = kUpCols * pitch;
  const int cols = (a.N + kUpCols - 1) / kUpCols;
  const int64_t all = (int64_t)a.plan->tiles[a.kind] * cols;
  bool waited = false;
  int64_t at = 0, stop = 0;
  for (int side = 0;;) {
    if (at >= stop) {
      if (side == kUpRuns) break;
      const int64_t run = (int64_t)side * gridDim.x + (side & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x), runs = (int64_t)kUpRuns * gridDim.x;
      at = all * run / runs;
      stop = all * (run + 1) / runs;
      ++side;
      continue;
    }
    const int tile = (int)(at / cols), begin = (int)(at - (int64_t)tile * cols);
    const int end = (int)(stop - at < cols - begin ? begin + (stop - at) : cols);
    at += end - begin;
    const AdapterTile t = a.tiles[tile];
    const int live = live_rank(a, t.adapter), blocks = MULTI ? max(1, (live + KS * 16 - 1) / (KS * 16)) : 1;
    const int p0 = warp * 16 + g;  // the thread's tokens: p0 and p0 + 8 of the tile
    const __half* yp[2];
    __half* op[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int k = p0 + 8 * i < t.count ? a.order[t.first + p0 + 8 * i] : -1;
      yp[i] = k >= 0 ? a.y + k * a.ldy + 8 * c : nullptr;
      op[i] = a.out + (k >= 0 ? k : 0) * a.ldo + begin * kUpCols + 8 * c;
    }
    // Column 32 q + 8 c + 2 j + i of a tile is column 2 c + i of MMA 4 q + j: its row of B lies at 8 (4 q + j) + 2 c + i.
    // Zeros behind the rank up to whole blocks
    const __half* bg = a.b + (int64_t)t.adapter * a.N * a.R;
    const int pieces = 2 * KS * blocks, more = kUpThreads / pieces, rest = kUpThreads - more * pieces;
    const int col0 = tid / pieces, piece0 = tid - col0 * pieces;
    auto fetch = [&](int nt, int stage) {
      const int n0 = nt * kUpCols, have = min(kUpCols, a.N - n0);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int q = 0; q < 2; ++q)
          if (yp[i] && 8 * c + 32 * q < have) cp_async16(y_ring + stage * kUpY + (2 * i + q) * kUpThreads * 16, yp[i] + n0 + 32 * q, 16);
      const uint32_t st = b_ring + stage * stage_bytes;
      const __half* src = bg + (int64_t)n0 * a.R;
      auto one = [&](int col, int p) {
        const int bytes = col < have ? min(16, max(0, (live - p * 8) * 2)) : 0;
        const int at = (col & 32) + (col >> 1 & 3) * 8 + (col >> 3 & 3) * 2 + (col & 1);
        cp_async16(st + at * pitch + (KS == 4 ? p ^ (at & 1) << 2 : p) * 16, bytes ? src + col * a.R + p * 8 : a.b, bytes);
      };
      if constexpr (MULTI) {
        for (int col = col0, p = piece0; col < kUpCols;) {
          one(col, p);
          col += more, p += rest;
          if (p >= pieces) p -= pieces, ++col;
        }
      } else if constexpr (KS >= 2) {
#pragma unroll
        for (int i = 0; i < kUpCols * 2 * KS / kUpThreads; ++i) one(col0 + i * (kUpThreads / (2 * KS)), piece0);
      } else {
        if (col0 < kUpCols) one(col0, piece0);
      }
    };
    __syncthreads();  // the stages of the run before have been used
#pragma unroll
    for (int i = 0; i < S - 1; ++i) {
      if (begin + i < end) fetch(begin + i, i);
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
    if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");  // h is written
    waited = true;
    // 8 neighbouring ranks of 32 (of 16: 4) are a thread's k's of two MMAs (of one), as in `down`; B's are read below alike
    uint32_t hi[KS][4], lo[KS][4];
    float back[2];
    auto terms = [&](int blk) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int p = p0 + 8 * i;
        const int64_t q = ((int64_t)(t.first + p) * a.blocks + blk);
        back[i] = p < t.count ? a.back[q] : 0.f;
        auto load = [&](uint32_t (&w)[KS][4], const __half* h) {
          if constexpr (KS == 1) {
            const uint2 v = p < t.count ? *reinterpret_cast<const uint2*>(h + 4 * c) : make_uint2(0, 0);
            w[0][i] = v.x, w[0][i + 2] = v.y;
          } else {
#pragma unroll
            for (int k = 0; k < KS; k += 2) {
              const uint4 v = p < t.count ? *reinterpret_cast<const uint4*>(h + 16 * k + 8 * c) : make_uint4(0, 0, 0, 0);
              w[k][i] = v.x, w[k][i + 2] = v.y;
              w[k + 1][i] = v.z, w[k + 1][i + 2] = v.w;
            }
          }
        };
        load(hi, a.terms + q * 2 * (KS * 16));
        load(lo, a.terms + q * 2 * (KS * 16) + KS * 16);
      }
    };
    if (!MULTI) terms(0);
    int stage = 0;
    for (int nt = begin; nt < end; ++nt) {
      asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
      __syncthreads();  // tile nt is there, and tile nt - 1 has been used
      if (nt + S - 1 < end) fetch(nt + S - 1, stage == 0 ? S - 1 : stage - 1);
      asm volatile("cp.async.commit_group;" ::: "memory");
      const uint32_t st = b_ring + stage * stage_bytes + g * pitch, swap = KS == 4 ? (g & 1) << 6 : 0;
      const int left = a.N - nt * kUpCols - 8 * c;
      if (warp * 16 < t.count) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {  // MMAs 4 q .. + 3: columns 32 q + 8 c .. + 7
          float sum[4][4];
          for (int blk = 0; blk < blocks; ++blk) {
            if (MULTI) terms(blk);
            float acc[4][4];
            const uint32_t row = st + 4 * q * 8 * pitch + blk * KS * 32;
            const bool more = KS == 4 && (blk * KS + 2) * 16 < live;
            // sums with lo and with hi apart, by the B of two steps and two MMAs' columns at a time
            float low[4][4];
            constexpr int kAtOnce = KS == 1 ? 1 : 2, kSteps = 2 * (KS == 4 ? 2 : 1);
            uint2 b[2][kAtOnce][2];
            auto load = [&](int i) {
              const int k0 = (i >> 1) * 2, j0 = (i & 1) * 2;
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                if constexpr (KS == 1) {
                  b[i & 1][0][j] = ld_shared_v2(row + (j0 + j) * 8 * pitch + c * 8);
                } else {
                  const uint4 v = ld_shared_v4(row + (j0 + j) * 8 * pitch + ((k0 * 32 + c * 16) ^ swap));
                  b[i & 1][0][j] = make_uint2(v.x, v.y), b[i & 1][kAtOnce - 1][j] = make_uint2(v.z, v.w);
                }
              }
            };
            // (the next B ahead: of ranks 65 to 128 388 us against 405, of up to 64 123.4 against 122.4)
            if (MULTI) load(0);
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
              if (i == 2 && !more) break;
              if (!MULTI) load(i);
              else if (i + 1 < kSteps) load(i + 1);
#pragma unroll
              for (int h = 0; h < kAtOnce; ++h)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                  const int k = (i >> 1) * 2 + h, jj = (i & 1) * 2 + j;
                  const uint2 w = b[i & 1][h][j];
                  if (k == 0) {
                    mma_16816_first(low[jj], lo[k][0], lo[k][1], lo[k][2], lo[k][3], w.x, w.y);
                    mma_16816_first(acc[jj], hi[k][0], hi[k][1], hi[k][2], hi[k][3], w.x, w.y);
                  } else {
                    mma_16816(low[jj], lo[k][0], lo[k][1], lo[k][2], lo[k][3], w.x, w.y);
                    mma_16816(acc[jj], hi[k][0], hi[k][1], hi[k][2], hi[k][3], w.x, w.y);
                  }
                }
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) (&acc[0][0])[j] = fmaf((&low[0][0])[j], 1 / kLowScale, (&acc[0][0])[j]);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              float& s = (&sum[0][0])[j];
              const float v = (&acc[0][0])[j];
              s = !MULTI ? v : blk == 0 ? v * back[j >> 1 & 1] : fmaf(v, back[j >> 1 & 1], s);
            }
          }
          if (32 * q < left) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (!yp[i]) continue;
              uint4 o = ld_shared_v4(y_ring + stage * kUpY + (2 * i + q) * kUpThreads * 16);
              uint32_t* w = reinterpret_cast<uint32_t*>(&o);
              const float f = MULTI ? 1.f : back[i];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
                w[j] = pack_half2(fmaf(sum[j][2 * i], f, v.x), fmaf(sum[j][2 * i + 1], f, v.y));
              }
              __stcs(reinterpret_cast<uint4*>(op[i]) + 4 * q, o);
            }
          }
        }
      }
      op[0] += kUpCols;
      op[1] += kUpCols;
      stage = stage == S - 1 ? 0 : stage + 1;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  }
  if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");  // no launch is over before the one it began beside
}

template <typename... Args>
static cudaError_t launch(void (*fn)(Args...), dim3 grid, int threads, size_t smem, cudaStream_t s, int cluster, Args... args) {
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
  at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[n].val.programmaticStreamSerializationAllowed = 1;
  ++n;
  cfg.attrs = at;
  cfg.numAttrs = (unsigned)n;
  return cudaLaunchKernelEx(&cfg, fn, args...);
}

// ranks that share a power of two, and a launch of `down`'s part of A
static int rank_block(int64_t R) { return R <= 16 ? 16 : R <= 32 ? 32 : 64; }

// Up to this many tokens of a step the tiles are of 16.  In a graph, K 5120, N 17408, rank 16, tiles of 16 against those of 128:
//   tokens   one adapter       10 adapters in turn   100 in turn
//      64     7.7 / 10.6 us       8.5 / 15.5 us        17.9 / 45.7 us
//     256    12.9 / 15.5         14.8 / 19.2           25.8 / 69.1
//     512    17.7 / 18.9         20.8 / 20.7           28.8 / 69.2
//    1024    27.1 / 24.4         30.0 / 25.6           38.1 / 77.0
// rank 64: 17.2 / 20.5, 20.3 / 27.3 and 56.5 / 116 at 256 tokens, 35.7 / 35.1, 39.6 / 39.1 and 67.8 / 124 at 1024.  The two
// cross between 512 and 1024 tokens where adapters are few, and later than 1024 where they are many: up to there a higher
// number than 256, and one that goes by the adapters, would be the faster one.
constexpr int kFewTokens = 256;

}  // namespace tb

extern "C" size_t tb_adapter_linear_workspace_size(int64_t T, int64_t n, int64_t K, int64_t N, int64_t R) {
  using namespace tb;
  if (T < 0 || T > INT_MAX / 2 || n < 1 || K < 8 || N < 8 || R < 8 || R > kAdapterMaxR) return 0;
  const int64_t block = rank_block(R), blocks = (R + block - 1) / block;
  return (size_t)T * blocks * (block * 4 + 4);
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
  g.kind = few ? 0 : 1;
  const char* base = static_cast<const char*>(plan);
  g.plan = static_cast<const AdapterPlan*>(plan);
  g.order = reinterpret_cast<const int32_t*>(base + adapter_order_at());
  g.tiles = reinterpret_cast<const AdapterTile*>(base + adapter_tiles_at(T, n, g.kind));
  g.block = rank_block(R);
  g.blocks = (int)((R + g.block - 1) / g.block);
  g.terms = static_cast<__half*>(workspace);
  g.back = reinterpret_cast<float*>(g.terms + (size_t)T * g.blocks * g.block * 2);
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
  const int64_t tiles = adapter_max_tiles(T, n, g.kind);
  // K is split over a cluster, as long as two CTAs an SM are enough for all (64 tiles by eight, as more than fit at once:
  // 22 us for 64 tokens; by four: 19): few tokens, of at least four steps a warp; many, of at least 16 stages
  g.cluster = 1;
  if (few)
    while (g.cluster < 8 && tiles * g.cluster * 2 <= 2 * f.sms && K / 32 >= g.cluster * 2 * kDownWarps) g.cluster *= 2;
  else
    while (g.cluster < 8 && tiles * g.cluster * 2 <= 2 * f.sms && K / 64 >= g.cluster * 16) g.cluster *= 2;
  const int nt = g.block / 8;
  const dim3 grid((unsigned)(tiles * g.cluster), (unsigned)g.blocks);
  cudaError_t e;
#define TB_DOWN_FEW(NT)                                                                                                         \
  ((rc = ensure_dynamic_smem(reinterpret_cast<const void*>(adapter_down_few_kernel<NT>), f.device, down_few_smem<NT>())) != TB_OK \
       ? cudaErrorUnknown                                                                                                       \
       : launch(adapter_down_few_kernel<NT>, grid, kDownThreads, (size_t)down_few_smem<NT>(), s, g.cluster, g))
#define TB_DOWN_MANY(N)                                                                                                        \
  ((rc = ensure_dynamic_smem(reinterpret_cast<const void*>(adapter_down_many_kernel<N>), f.device, down_many_smem<N>())) != TB_OK \
       ? cudaErrorUnknown                                                                                                      \
       : launch(adapter_down_many_kernel<N>, grid, kManyThreads, (size_t)down_many_smem<N>(), s, g.cluster, g))
  if (few)
    e = nt == 2 ? TB_DOWN_FEW(2) : nt == 4 ? TB_DOWN_FEW(4) : TB_DOWN_FEW(8);
  else
    e = nt == 2 ? TB_DOWN_MANY(16) : nt == 4 ? TB_DOWN_MANY(32) : TB_DOWN_MANY(64);
#undef TB_DOWN_FEW
#undef TB_DOWN_MANY
  if (rc != TB_OK) return rc;
  if (e == cudaSuccess) {
    if (few) {
      // two CTAs an SM share all tiles' columns; at least 32 columns a warp
      int64_t ctas = (tiles * ((N + 31) / 32) + kUpFewWarps - 1) / kUpFewWarps;
      const dim3 some((unsigned)(ctas < 2 * f.sms ? ctas : 2 * f.sms));
#define TB_UP(W, MULTI)                                                                                                            \
  ((rc = ensure_dynamic_smem(reinterpret_cast<const void*>(adapter_up_few_kernel<W, MULTI>), f.device, up_few_smem<W>())) != TB_OK \
       ? cudaErrorUnknown                                                                                                          \
       : launch(adapter_up_few_kernel<W, MULTI>, some, kUpFewThreads, (size_t)up_few_smem<W>(), s, 1, g))
      e = R <= 16 ? TB_UP(4, false) : R <= 32 ? TB_UP(8, false) : R <= 64 ? TB_UP(16, false) : TB_UP(16, true);
#undef TB_UP
      if (rc != TB_OK) return rc;
    } else {
      const size_t smem = (size_t)up_stages(R > 64) * (kUpY + kUpCols * up_pitch(g.block, g.blocks));
      const int64_t ctas = tiles * ((N + kUpCols - 1) / kUpCols);
      const dim3 some((unsigned)(ctas < 2 * f.sms ? ctas : 2 * f.sms));
#define TB_UP(KS, MULTI)                                                                                                           \
  ((rc = ensure_dynamic_smem(reinterpret_cast<const void*>(adapter_up_many_kernel<KS, MULTI>), f.device, (int)smem)) != TB_OK \
       ? cudaErrorUnknown                                                                                                          \
       : launch(adapter_up_many_kernel<KS, MULTI>, some, kUpThreads, smem, s, 1, g))
      e = R <= 16 ? TB_UP(1, false) : R <= 32 ? TB_UP(2, false) : R <= 64 ? TB_UP(4, false) : TB_UP(4, true);
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
