// Causal attention over packed prompts on tcgen05 (csrc/tb_attention.cu has the entry point's checks,
// csrc/tb_attention.cuh the row-by-row form).
//
// A tile is up to 128 rows of one KV head, a row being one (token, query head) pair: the query heads
// that share the KV head lie next to each other in q, so a tile of 128 / G tokens by G heads is one
// box of a 3-D tensor map.  Short requests fill a tile with few tokens, and the causal edge wastes
// G times less than tiles of 128 tokens would.
//
// Per tile of 128 keys:  S = Q K^T (tensor memory, 128 x 128 fp32, two buffers), softmax with the
// running maximum and sum in registers (one thread per row), P in fp16 back into S's columns, and
// O += P V (tensor memory, 128 x D fp32).  A tile's softmax takes about 2100 clocks from S to P with one
// warp per SM sub-partition, as long as its MMAs (D = 256: 16.8 MFLOP are 2048 clocks at 8192 a clock),
// so two groups of four warps take turns at the tiles: while one is in the softmax of a tile, the
// tensor cores run P V of the tile before and S of the next.  The groups pass the rows' maxima on in
// tile order, as O has one scale.
// CG = 2: a CTA pair (cta_group::2) runs 256 rows on the same keys; each CTA loads half of K (its 64
// keys) and half of V (its half of the columns) and the tensor cores read both halves.  One CTA alone
// reads Q, K and V at 128 bytes a clock, all that shared memory gives, and loads 64 bytes a clock
// from L2; the pair halves the K and V part of both.
//
// Precision: S, maxima, sums and O in fp32; P is rounded to fp16, O once at the end.  O is rescaled
// only when a row's maximum has grown by more than 2^8 since the last time (P stays within 2^15,
// kPTop, and the sum carries the same factor).
//
// One prompt of 12289 tokens, 24/4 heads of 256: 1.09 to 1.13 ms in a replayed graph (1640 to 1700 TFLOP/s, 0.87 to
// 0.90 of measured), 1.20 to 1.23 ms a call in a row of calls (0.81; under the power cap); one of 4096: 0.15 ms; of
// 1024: 24 us.  Bound by the tensor cores from a few thousand tokens on, below by what each tile has beside its MMAs
// (first loads, first softmax, output).  Heads of 128 and 64: 0.82 and 0.76 ms, bound by the exponentials (16384 a
// tile, 1024 clocks of their pipe).
//
// Keys a row does not see get P = 0, which keeps them out as long as V is finite.  Rows that are not finite are
// looked at by all warps of their CTA once it has no item left, when nothing waits for anything under a limit: one
// pass over V per tile finds, column by column, what is not finite among the keys a row sees and makes its output
// so; a row that sees nothing of the kind there is computed again from its own keys (attend_keys).  A prompt of
// 12289 tokens whose first value is NaN takes 2.5 ms instead of 1.1.
#include <cuda.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>

#include "tb_attention.cuh"
#include "tb_attn_tc.cuh"
#include "tb_host.h"

namespace tb {

constexpr int kPaThreads = 320;  // warps 0-3 and 4-7: softmax of even and odd key tiles; 8: loads; 9: MMAs
constexpr int kPaKeys = 128;     // keys per tile

template <int D, int CG>
struct PaCfg {
  static constexpr int kChunks = D / 64;             // 128-byte wide pieces of a row
  static constexpr int kQBytes = kChunks * 16384;    // 128 rows
  // of a tile's keys a CTA loads 128 / CG rows of K, and D / CG columns of V
  static constexpr int kKRows = kPaKeys / CG;
  static constexpr int kVChunks = kChunks / CG;
  static_assert(kVChunks >= 1, "D = 64 has no pair form");
  static constexpr int kTileBytes = kPaKeys * D * 2 / CG;  // of K, or of V
  static constexpr int kK = kQBytes, kV = kK + 2 * kTileBytes, kStage = kV + 2 * kTileBytes;  // two of each
  static constexpr int kBars = kStage + 8 * 2048;  // a warp's 32 rows of output, 64 bytes of each at a time
  static constexpr int kSmem = 1024 + kBars + 256;
  static constexpr uint32_t kIdescQK = (1u << 4) | ((uint32_t)(kPaKeys >> 3) << 17) | ((uint32_t)(128 * CG >> 4) << 24);
  static constexpr uint32_t kIdescPV =
      (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | ((uint32_t)(128 * CG >> 4) << 24);
  static constexpr uint32_t kTmemO = 2 * kPaKeys;  // columns: S0 | S1 | O
};

struct PaArgs {
  AttnArgs a;
  int gp, tok;      // query heads per tile, tokens per CTA's tile
  int head_parts;   // tiles side by side over the heads: Hkv * (G / gp)
  int64_t room;     // 0, or tiles of a head part that are to be counted and not to be exceeded
  unsigned magic;   // for divisions by the tokens of a tile
};

// a tile of 128 CG rows and what it needs; n < 0: no more of them
struct PaItem {
  int n, hp;            // key tiles; which heads
  int q0, lq, k0, lk;   // the request's rows
  int first;            // the tile's first token in the request
  int pad;
};

// Item k of the schedule: all requests' tiles by falling number of key tiles, the heads side by side, so
// that clusters which take turns at them, back and forth, end together.  Nothing is sorted: the number
// of tiles with more than c key tiles is a sum over the requests, and a bisection over c finds item
// k's; whole warps call this, each lane with its share of the requests.
TB_DEVI bool pa_rows(const AttnArgs& a, int b, int& q0, int& lq, int& k0, int& lk) {
  const int64_t x = __ldg(a.q_start + b), y = __ldg(a.q_start + b + 1);
  const int64_t u = __ldg(a.k_start + b), w = __ldg(a.k_start + b + 1);
  const bool q_ok = x >= 0 && y >= x && y <= a.T, k_ok = u >= 0 && w >= u && w <= a.Tk;
  q0 = (int)x;
  lq = q_ok ? (int)(y - x) : 0;
  k0 = k_ok ? (int)u : 0;
  lk = k_ok ? (int)(w - u) : 0;
  return q_ok && k_ok;
}
struct PaSpan {
  unsigned tokens, magic;  // of a tile, and 2^32 / tokens rounded up (0 for one token)
};
TB_DEVI int pa_div(int x, const PaSpan& s) {  // x >= 0
  if (s.tokens == 1) return x;
  unsigned q = __umulhi((unsigned)x, s.magic);  // at most one too large
  if (q * s.tokens > (unsigned)x) --q;
  return (int)q;
}
// tiles of a request with more than c key tiles (c = -1: all)
TB_DEVI int pa_longer(int lq, int lk, const PaSpan& span, int c) {
  const int tiles = pa_div(lq + (int)span.tokens - 1, span);
  const int64_t x = c < 0 ? -1 : (int64_t)c * kPaKeys - ((int64_t)lk - lq);  // tokens that see at most c tiles of keys
  return x < 0 ? tiles : (x >= lq ? 0 : tiles - pa_div((int)x, span));
}
// (Counts of tiles fit 32 bits: requests in order, one after another, have no more than T / span tokens + B together.
// Where row starts go back they can have up to B times T / span; calls for which that is too much are counted in 64
// bits first, pa_in_order.)
//
// With more than kPaSorted requests a lane the bisection would cost more than a tile of them; they
// then go in the order they come in, each one's longest tile first.
constexpr int kPaSorted = 4;
struct PaShare {
  int per, lq, lk;  // a lane's requests, and the first one's lengths
  int own, upto;    // its tiles, and those up to it
};
TB_DEVI PaShare pa_share(const AttnArgs& a, const PaSpan& span, int lane) {
  PaShare s;
  s.per = (a.B + 31) / 32;
  s.lq = s.lk = s.own = 0;
  int q0, k0, lq, lk;
  if (lane * s.per < a.B) pa_rows(a, lane * s.per, q0, s.lq, k0, s.lk);
  for (int b = lane * s.per; b < (lane + 1) * s.per && b < a.B; ++b) {
    pa_rows(a, b, q0, lq, k0, lk);
    s.own += pa_longer(lq, lk, span, -1);
  }
  s.upto = s.own;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, s.upto, d);
    if (lane >= d) s.upto += x;
  }
  return s;
}
// do the requests make no more tiles than `room`?
TB_DEVI bool pa_in_order(const AttnArgs& a, const PaSpan& span, int64_t room, int lane) {
  int64_t sum = 0;
  int q0, k0, lq, lk;
  for (int b = lane; b < a.B; b += 32) {
    pa_rows(a, b, q0, lq, k0, lk);
    sum += pa_longer(lq, lk, span, -1);
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  return sum <= room;
}
TB_DEVI PaItem pa_item(const PaArgs& p, const PaShare& sh, const PaSpan& span, unsigned k, int lane) {
  const AttnArgs& a = p.a;
  PaItem it;
  it.n = -1;
  const int place = (int)(k / (unsigned)p.head_parts);
  it.hp = (int)(k - (unsigned)place * (unsigned)p.head_parts);
  int q0, lq, k0, lk;
  auto own = [&](int c) {
    int n = pa_longer(sh.lq, sh.lk, span, c);
    for (int b = lane * sh.per + 1; b < (lane + 1) * sh.per && b < a.B; ++b) {
      pa_rows(a, b, q0, lq, k0, lk);
      n += pa_longer(lq, lk, span, c);
    }
    return n;
  };
  auto total = [&](int n) { return (int)__reduce_add_sync(0xffffffffu, (unsigned)n); };
  if (place >= __shfl_sync(0xffffffffu, sh.upto, 31)) return it;
  if (sh.per > kPaSorted) {
    const int src = __ffs(__ballot_sync(0xffffffffu, place < sh.upto)) - 1;
    int b = lane * sh.per, r = place - (sh.upto - sh.own), tile = 0;
    if (lane == src) {
      for (;; ++b) {
        pa_rows(a, b, q0, lq, k0, lk);
        const int tiles = pa_longer(lq, lk, span, -1);
        if (r < tiles) {
          tile = tiles - 1 - r;
          break;
        }
        r -= tiles;
      }
    }
    b = __shfl_sync(0xffffffffu, b, src);
    it.first = __shfl_sync(0xffffffffu, tile, src) * (int)span.tokens;
    pa_rows(a, b, it.q0, it.lq, it.k0, it.lk);
    const int64_t end = it.first + (int64_t)span.tokens, keys = (end < it.lq ? end : it.lq) + (int64_t)it.lk - it.lq;
    it.n = keys > 0 ? (int)((keys + kPaKeys - 1) / kPaKeys) : 0;
    return it;
  }
  int lo = 0, hi = (int)((a.Tk + kPaKeys - 1) / kPaKeys);  // the least c with at most `place` longer tiles
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (total(own(mid)) <= place) hi = mid;
    else lo = mid + 1;
  }
  const int longer = own(lo), as_long = own(lo - 1) - longer;
  int upto = as_long;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += x;
  }
  int r = place - total(longer);
  const int src = __ffs(__ballot_sync(0xffffffffu, r < upto)) - 1;
  r -= upto - as_long;  // among the lane's own
  int b = lane * sh.per, first = 0;
  if (lane == src) {
    for (;; ++b) {
      pa_rows(a, b, q0, lq, k0, lk);
      const int more = pa_longer(lq, lk, span, lo), same = pa_longer(lq, lk, span, lo - 1) - more;
      if (r < same) {
        first = (pa_div(lq + (int)span.tokens - 1, span) - 1 - more - r) * (int)span.tokens;  // the longest such tile first
        break;
      }
      r -= same;
    }
  }
  b = __shfl_sync(0xffffffffu, b, src);
  it.first = __shfl_sync(0xffffffffu, first, src);
  pa_rows(a, b, it.q0, it.lq, it.k0, it.lk);
  it.n = lo;
  return it;
}

template <int D, int CG>
__global__ void __launch_bounds__(kPaThreads, 1)
    prompt_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const PaArgs p) {
  using C = PaCfg<D, CG>;
  const AttnArgs& a = p.a;
  extern __shared__ uint8_t pa_raw[];
  const uint32_t raw = smem_u32(pa_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = pa_raw + (base - raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBars);
  // per key tile, two of each in turn: K and V have landed; S is computed (and K read); P is written;
  // P V is added (and V read)
  uint64_t *k_full = bars, *v_full = bars + 2, *s_full = bars + 4, *p_full = bars + 6, *o_done = bars + 8;
  uint64_t* m_full = bars + 10;  // [2][4]: a warp's row maxima after its tile, for the other group's warp
  // per item: Q has landed, has been read; O is complete, has been read; the item's words are there, read
  uint64_t *q_full = bars + 18, *q_empty = bars + 19, *o_last = bars + 20, *o_free = bars + 21;
  uint64_t *item_full = bars + 22, *item_empty = bars + 24;  // [2] each
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 26);
  __shared__ volatile int aborted, redo;  // redo: a row of this CTA's is not finite
  __shared__ float maxima[2][128];
  __shared__ float2 sums[2][128];  // (sum, the maximum it refers to) of each group's rows
  __shared__ PaItem items[2];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = CG > 1 ? cta_rank_in_cluster() : 0;

  if (tid == 0) {
    aborted = redo = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(k_full + i, 1);
      mbar_init(v_full + i, 1);
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, 4 * CG);  // lane 0 of each warp of the group, of both CTAs
      mbar_init(o_done + i, 1);
      mbar_init(item_full + i, 1);
      mbar_init(item_empty + i, 9);  // the MMA warp and the softmax warps
    }
    for (int i = 0; i < 8; ++i) mbar_init(m_full + i, 1);
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(o_last, 1);
    mbar_init(o_free, 8 * CG);
    fence_barrier_init();
  }
  if (p.room && !pa_in_order(a, PaSpan{(unsigned)(p.tok * CG), p.magic}, p.room, lane)) {
    if (blockIdx.x == 0 && tid == 0) set_status(a.status, TB_DEV_BAD_LEN);
    return;  // every thread of every CTA
  }
  if (warp == 9) tmem_alloc_cg<CG>(tmem_slot, 512);
  if (blockIdx.x == 0 && a.status) {  // one CTA looks at every request's row starts
    int x, y, z, w;
    for (int b = tid; b < a.B; b += kPaThreads)
      if (!pa_rows(a, b, x, y, z, w)) set_status(a.status, TB_DEV_BAD_LEN);
  }
  tmem_fence_before();
  __syncthreads();
  if constexpr (CG > 1) cluster_barrier();  // the peer's barriers exist
  tmem_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int G = a.Hq / a.Hkv, parts = G / p.gp;

  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity) || aborted) return;
    if (!mbar_wait(bar, parity)) {
      aborted = 1;
      set_status(a.status, TB_DEV_TIMEOUT);
    }
  };
  auto wait_cluster = [&](uint64_t* bar, uint32_t parity) {  // arrivals from both CTAs
    if (CG == 1) {
      wait(bar, parity);
      return;
    }
    if (mbar_try_wait_cluster(bar, parity) || aborted) return;
    const uint64_t t = globaltimer_ns();
    while (!mbar_try_wait_cluster(bar, parity)) {
      if (aborted || globaltimer_ns() - t > TB_WAIT_NS) {
        aborted = 1;
        set_status(a.status, TB_DEV_TIMEOUT);
        return;
      }
    }
  };
  const unsigned clusters = gridDim.x / CG, me = blockIdx.x / CG;
  const PaSpan span = {(unsigned)(p.tok * CG), p.magic};
  const PaShare share = pa_share(a, span, lane);
  auto my_item = [&](unsigned i) {  // back and forth over the clusters
    return pa_item(p, share, span, i * clusters + ((i & 1) ? clusters - 1 - me : me), lane);
  };
  // the words of this CTA's item number i, handed back when the warp has them
  auto next_item = [&](int i) {
    PaItem it;
    wait(item_full + (i & 1), (i >> 1) & 1);
    // a wait somewhere gave up: the words may not be there, but every warp still takes the same items,
    // so that none is left alone at a barrier
    if (aborted) return my_item(i);
    const volatile int* w = reinterpret_cast<const volatile int*>(&items[i & 1]);
    it.n = w[0];
    it.hp = w[1];
    it.q0 = w[2];
    it.lq = w[3];
    it.k0 = w[4];
    it.lk = w[5];
    it.first = w[6];
    __syncwarp();
    if (lane == 0) mbar_arrive(item_empty + (i & 1));
    return it;
  };

  if (warp == 8) {
    const uint32_t qbar = CG > 1 ? cluster_addr(q_full, 0) : smem_u32(q_full);
    const uint32_t kbar = CG > 1 ? cluster_addr(k_full, 0) : smem_u32(k_full);
    const uint32_t vbar = CG > 1 ? cluster_addr(v_full, 0) : smem_u32(v_full);
    int gt = 0, seg = 0;  // key tiles and items with keys so far
    PaItem it = my_item(0);
    for (int i = 0;; ++i) {
      if (i >= 2) wait(item_empty + (i & 1), ((i >> 1) - 1) & 1);
      if (lane == 0) {
        items[i & 1] = it;
        mbar_arrive(item_full + (i & 1));
      }
      __syncwarp();
      if (it.n < 0 || aborted) break;
      PaItem next;
      if (it.n == 0) {
        it = my_item(i + 1);
        continue;
      }
      const int hk = it.hp / parts, h0 = hk * G + (it.hp % parts) * p.gp;
      if (lane == 0) {
        if (seg > 0) wait(q_empty, (seg - 1) & 1);
        if (rank == 0) mbar_arrive_expect_tx(q_full, CG * C::kChunks * 128 * p.gp * p.tok);
#pragma unroll
        for (int c = 0; c < C::kChunks; ++c)
          tma_load_3d<CG>(base + c * 16384, &tmQ, c * 64, h0, it.q0 + it.first + (int)rank * p.tok, qbar);
      }
      auto load_k = [&](int j) {
        const int g = gt + j, x = g & 1, row = it.k0 + j * kPaKeys + (int)rank * C::kKRows;
        if (g >= 2) wait(s_full + x, ((g >> 1) - 1) & 1);  // S of two tiles ago has read its K
        if (rank == 0) mbar_arrive_expect_tx(k_full + x, CG * C::kTileBytes);
#pragma unroll
        for (int c = 0; c < C::kChunks; ++c)
          tma_load_3d<CG>(base + C::kK + x * C::kTileBytes + c * (C::kKRows * 128), &tmK, c * 64, hk, row, kbar + 8u * x);
      };
      auto load_v = [&](int j) {
        const int g = gt + j, x = g & 1, row = it.k0 + j * kPaKeys;
        if (g >= 2) wait(o_done + x, ((g >> 1) - 1) & 1);
        if (rank == 0) mbar_arrive_expect_tx(v_full + x, CG * C::kTileBytes);
#pragma unroll
        for (int c = 0; c < C::kVChunks; ++c)
          tma_load_3d<CG>(base + C::kV + x * C::kTileBytes + c * (kPaKeys * 128), &tmV, ((int)rank * C::kVChunks + c) * 64, hk,
                          row, vbar + 8u * x);
      };
      if (lane == 0) {
        load_k(0);
        if (it.n > 1) load_k(1);
        load_v(0);
      }
      __syncwarp();
      next = my_item(i + 1);  // while the tensor cores have something to do
      if (lane == 0) {
        for (int j = 1; j < it.n; ++j) {
          if (j + 1 < it.n) load_k(j + 1);
          load_v(j);
        }
      }
      __syncwarp();
      gt += it.n;
      ++seg;
      it = next;
    }
    if (aborted) {  // a wait gave up: leave the copies in flight time to land before the CTA ends
      const uint64_t t = globaltimer_ns();
      while (globaltimer_ns() - t < 1000000) {
      }
    }
  } else if (warp == 9) {
    // An MMA is issued about when its predecessor starts, so what this thread does between two of them
    // is idle time of the tensor cores: a tile costs it three waits and two commits.
    // descriptors of place 0; the address field counts 16 bytes, and no sum carries out of it
    const uint64_t qdesc = smem_desc_sw128(base, 1024), kdesc = smem_desc_sw128(base + C::kK, 1024);
    const uint64_t vdesc = smem_desc_mn128(base + C::kV, kPaKeys * 128, 1024);
    int gt = 0, seg = 0;
    for (int i = 0;; ++i) {
      const PaItem it = next_item(i);
      if (it.n < 0) break;
      if (it.n == 0) continue;
      if (lane == 0 && rank == 0) {
        wait(q_full, seg & 1);
        auto qk = [&](int j) {
          const int x = (gt + j) & 1;
          const uint32_t d = tmem + (uint32_t)x * kPaKeys;
          const uint64_t kd = kdesc + x * (C::kTileBytes >> 4);
          wait(k_full + x, ((gt + j) >> 1) & 1);
          tmem_fence_after();
#pragma unroll
          for (int c = 0; c < C::kChunks; ++c)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_f16_ss<CG>(d, qdesc + c * (16384 >> 4) + kk * 2, kd + c * (C::kKRows * 128 >> 4) + kk * 2, C::kIdescQK,
                             (c | kk) != 0);
          mma_commit_cg<CG>(s_full + x);
          if (j + 1 == it.n) mma_commit_cg<CG>(q_empty);
        };
        qk(0);
        if (it.n > 1) qk(1);
        if (seg > 0) wait_cluster(o_free, (seg - 1) & 1);  // the last item's O has been read
        for (int j = 0; j < it.n; ++j) {
          const int x = (gt + j) & 1;
          const uint32_t pa = tmem + (uint32_t)x * kPaKeys;
          const uint64_t vd = vdesc + x * (C::kTileBytes >> 4);
          wait(v_full + x, ((gt + j) >> 1) & 1);
          wait_cluster(p_full + x, ((gt + j) >> 1) & 1);
          tmem_fence_after();
#pragma unroll
          for (int kk = 0; kk < kPaKeys / 16; ++kk)
            mma_f16_ts<CG>(tmem + C::kTmemO, pa + kk * 8, vd + kk * (2048 >> 4), C::kIdescPV, (j | kk) != 0);
          mma_commit_cg<CG>(o_done + x);
          if (j + 2 < it.n) qk(j + 2);  // over P of this tile, which the MMAs before it have read
        }
        mma_commit_cg<CG>(o_last);
      }
      __syncwarp();
      gt += it.n;
      ++seg;
    }
  } else {
    // ---- softmax: thread = row; two groups of four warps take turns at the key tiles
    const int group = warp >> 2, row = tid & 127;
    const int tr = row / p.gp;
    const uint32_t mine = tmem + ((uint32_t)(warp & 3) << 21);  // lane quarter: 32 lanes, in bits 16..
    const float sc = a.scale_log2;
    const uint32_t pbar = (CG > 1 ? cluster_addr(p_full, 0) : smem_u32(p_full)) + 8u * (uint32_t)group;
    const uint32_t obar = CG > 1 ? cluster_addr(o_free, 0) : smem_u32(o_free);
    auto sync256 = []() { asm volatile("bar.sync 1, 256;" ::: "memory"); };
    int gt = 0, seg = 0;
    for (int i = 0;; ++i) {
      const PaItem it = next_item(i);
      if (it.n < 0) break;
      const int hk = it.hp / parts, head = hk * G + (it.hp % parts) * p.gp + row - tr * p.gp;
      const int tok = it.first + (int)rank * p.tok + tr;
      const bool live = tr < p.tok && tok < it.lq;
      const int lim = live && tok + it.lk - it.lq + 1 > 0 ? tok + it.lk - it.lq + 1 : 0;  // keys [0, lim) are visible
      __half* dst = a.o + (((int64_t)it.q0 + tok) * a.Hq + head) * D;
      if (it.n == 0) {  // no row of the tile sees a key
        if (live)
          for (int c = group * (D / 2); c < (group + 1) * (D / 2); c += 8)
            *reinterpret_cast<uint4*>(dst + c) = make_uint4(0, 0, 0, 0);
        continue;
      }
      float m = -INFINITY, l = 0.f;  // the group's reference (log2 units after scaling), and its sum
      for (int j = (gt ^ group) & 1; j < it.n; j += 2) {
        const int g = gt + j;
        wait(s_full + group, (g >> 1) & 1);
        tmem_fence_after();
        float s[kPaKeys];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(mine + group * kPaKeys + c * 32, s + 32 * c);
        tmem_wait_ld();
        const int left = lim - j * kPaKeys;
        if (__any_sync(0xffffffffu, left < kPaKeys)) {
#pragma unroll
          for (int c = 0; c < kPaKeys; ++c) s[c] = c < left ? s[c] : -INFINITY;
        }
        float mx[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) mx[c] = s[c];
#pragma unroll
        for (int c = 8; c < kPaKeys - 8; c += 16)
#pragma unroll
          for (int e = 0; e < 8; ++e) mx[e] = max3(mx[e], s[c + e], s[c + 8 + e]);
#pragma unroll
        for (int e = 0; e < 8; ++e) mx[e] = fmaxf(mx[e], s[kPaKeys - 8 + e]);
        const float tmax = max3(max3(mx[0], mx[1], mx[2]), max3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7])) * sc;
        // the reference of the tile before, from the other group
        float before = -INFINITY;
        if (j > 0) {
          wait(m_full + (group ^ 1) * 4 + (warp & 3), ((g - 1) >> 1) & 1);
          before = *reinterpret_cast<volatile float*>(&maxima[group ^ 1][row]);
        }
        // a new reference only when the old one is 2^8 too small (or there is none yet)
        const bool grow = tmax > before + 8.f || (before == -INFINITY && tmax > -INFINITY);
        const float now = grow ? tmax : before;
        maxima[group][row] = now;
        __syncwarp();
        if (lane == 0) mbar_arrive(m_full + group * 4 + (warp & 3));
        if (__any_sync(0xffffffffu, grow && j > 0)) {
          const float f = grow ? (before == -INFINITY ? 0.f : ex2(before - now)) : 1.f;
          // a parity tells only neighbouring phases apart: tile g - 3's is over, as S of tile g came after
          // it, and tile g + 1's cannot be over before this warp's part of P is there
          wait(o_done + (group ^ 1), ((g - 1) >> 1) & 1);
          tmem_fence_after();
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float o[32];
            tmem_ld32(mine + C::kTmemO + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 r = mul_f32x2(make_float2(o[e], o[e + 1]), make_float2(f, f));
              o[e] = r.x;
              o[e + 1] = r.y;
            }
            tmem_st32(mine + C::kTmemO + c, reinterpret_cast<uint32_t(&)[32]>(o));
          }
          tmem_wait_st();
        }
        if (now != m) l *= m == -INFINITY ? 0.f : ex2(m - now);
        m = now;
        const float ms = m == -INFINITY ? 0.f : kPTop - m;
        float2 acc0 = make_float2(0.f, 0.f), acc1 = acc0;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t pk[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const int c = half * 64 + e * 2;
            float2 x = fma_f32x2(make_float2(s[c], s[c + 1]), make_float2(sc, sc), make_float2(ms, ms));
            x.x = ex2(x.x);
            x.y = ex2(x.y);
            if (e & 1) acc1 = add_f32x2(acc1, x);
            else acc0 = add_f32x2(acc0, x);
            pk[e] = pack_half2(x.x, x.y);
          }
          tmem_st32(mine + group * kPaKeys + half * 32, pk);
        }
        acc0 = add_f32x2(acc0, acc1);
        l += acc0.x + acc0.y;
        tmem_wait_st();
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (CG > 1) mbar_arrive_cluster(pbar);
          else mbar_arrive(p_full + group);
        }
      }
      gt += it.n;
      // ---- O / l -> fp16, half of the columns per group
      sums[group][row] = make_float2(l, m);
      sync256();
      {
        const float2 other = sums[group ^ 1][row];
        const float M = fmaxf(m, other.y);  // the last reference: references only grow
        l = (m == -INFINITY ? l : l * ex2(m - M)) + (other.y == -INFINITY ? other.x : other.x * ex2(other.y - M));
      }
      wait(o_last, seg & 1);
      ++seg;
      tmem_fence_after();
      const float inv = inverse_sum(l);
      bool odd = false;
      // through shared memory, so that a store instruction covers eight rows (a thread's own row at a time it
      // touches 32: 3 us an item)
      int64_t out[4];  // where the rows that this lane stores begin
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int rr = (warp & 3) * 32 + x * 8 + (lane >> 2), rt = rr / p.gp, rtok = it.first + (int)rank * p.tok + rt;
        out[x] = rt < p.tok && rtok < it.lq
                     ? (((int64_t)it.q0 + rtok) * a.Hq + hk * G + (it.hp % parts) * p.gp + rr - rt * p.gp) * D
                     : -1;
      }
      const uint32_t stage = base + C::kStage + (uint32_t)warp * 2048u;
#pragma unroll 1
      for (int c = group * (D / 2); c < (group + 1) * (D / 2); c += 32) {
        float o[32];
        tmem_ld32(mine + C::kTmemO + c, o);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // (the pieces of neighbouring rows in turn, so that banks differ)
          uint32_t w[4] = {0, 0, 0, 0};
          if (lim > 0) {
#pragma unroll
            for (int y = 0; y < 8; ++y) odd |= !(fabsf(o[e * 8 + y]) < INFINITY);
#pragma unroll
            for (int y = 0; y < 4; ++y) w[y] = pack_half2(o[e * 8 + 2 * y] * inv, o[e * 8 + 2 * y + 1] * inv);
          }
          asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(stage + (uint32_t)lane * 64u +
                                                                     (((uint32_t)e ^ (((uint32_t)lane >> 1) & 3u)) << 4)),
                       "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                       : "memory");
        }
        __syncwarp();
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int r = x * 8 + (lane >> 2), pc = lane & 3;
          const uint4 w = ld_shared_v4(stage + (uint32_t)r * 64u + (((uint32_t)pc ^ (((uint32_t)r >> 1) & 3u)) << 4));
          if (out[x] >= 0) *reinterpret_cast<uint4*>(a.o + out[x] + c + pc * 8) = w;
        }
        __syncwarp();
      }
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (CG > 1) mbar_arrive_cluster(obar);
        else mbar_arrive(o_free);
      }
      for (unsigned lost = __ballot_sync(0xffffffffu, live && lim > 0 && !(l < INFINITY)); lost; lost &= lost - 1) {
        const int64_t to = __shfl_sync(0xffffffffu, (int64_t)(dst - a.o), __ffs(lost) - 1) + group * (D / 2);
        for (int c = lane; c < D / 2; c += 32) a.o[to + c] = __ushort_as_half((unsigned short)kNanRow);
      }
      if (live && lim > 0 && odd && l < INFINITY) redo = 1;
      sync256();  // the sums have been read
    }
  }

  tmem_fence_before();
  __syncthreads();
  if constexpr (CG > 1) cluster_barrier();  // no CTA leaves while its peer may still signal it or read it
  if (warp == 9) tmem_dealloc_cg<CG>(tmem, 512);
  if (!redo || aborted) return;
  // ---- the CTA's rows that are not finite, found by their output
  constexpr int E = D / 32, kWarps = kPaThreads / 32, kAhead = 4;
  // per column of V: the first key of the request whose value is NaN; infinity; minus infinity; infinite under a
  // key that is not finite itself, so that its weight may be zero
  int* first = reinterpret_cast<int*>(smem);  // [4][D], over Q
  for (int i = 0;; ++i) {
    const PaItem it = my_item(i);
    if (it.n < 0) break;
    if (it.n == 0) continue;
    const int hk = it.hp / parts, h0 = hk * G + (it.hp % parts) * p.gp;
    const int tok0 = it.first + (int)rank * p.tok, toks = min(p.tok, it.lq - tok0);
    auto keys_of = [&](int tr) { return tok0 + tr + it.lk - it.lq + 1; };
    auto out_of = [&](int row) { return a.o + (((int64_t)it.q0 + tok0 + row / p.gp) * a.Hq + h0 + row % p.gp) * D; };
    bool any = false;
    for (int row = warp; row < p.gp * toks; row += kWarps) {
      if (keys_of(row / p.gp) <= 0) continue;
      uint32_t w[E / 2];
      load_bits<E>(out_of(row), lane, w);
      any |= any_to_mend(w);
    }
    if (!__syncthreads_or(any)) continue;
    for (int x = tid; x < 4 * D; x += kPaThreads) first[x] = INT_MAX;
    __syncthreads();
    const int end = keys_of(toks - 1);
    for (int j0 = warp; j0 < end; j0 += kAhead * kWarps) {
      uint32_t v[kAhead][E / 2];
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        load_bits<E>(a.v + ((int64_t)it.k0 + min(j0 + u * kWarps, end - 1)) * a.ldv + hk * D, lane, v[u]);
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int j = min(j0 + u * kWarps, end - 1);
        bool odd = false, inf = false;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const uint32_t h = v[u][e / 2] >> (e & 1) * 16;
          odd |= not_finite_h(h);
          inf |= (h & 0x7fffu) == 0x7c00u;
        }
        if (!__any_sync(0xffffffffu, odd)) continue;
        bool key = false;
        if (__any_sync(0xffffffffu, inf)) {
          uint32_t k[E / 2];
          load_bits<E>(a.k + ((int64_t)it.k0 + j) * a.ldk + hk * D, lane, k);
#pragma unroll
          for (int e = 0; e < E / 2; ++e) key |= not_finite_h(k[e]) || not_finite_h(k[e] >> 16);
          key = __any_sync(0xffffffffu, key);
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const uint32_t h = v[u][e / 2] >> (e & 1) * 16;
          if (!not_finite_h(h)) continue;
          int* at = first + ((h & 0x3ffu) ? 0 : (key ? 3 : (h & 0x8000u ? 2 : 1))) * D + lane * E + e;
          if (*reinterpret_cast<volatile int*>(at) > j) atomicMin(at, j);
        }
      }
    }
    __syncthreads();
    for (int row = warp; row < p.gp * toks; row += kWarps) {
      const int lim = keys_of(row / p.gp);
      if (lim <= 0) continue;
      __half* dst = out_of(row);
      uint32_t w[E / 2];
      load_bits<E>(dst, lane, w);
      if (!__any_sync(0xffffffffu, any_to_mend(w))) continue;
      bool again = false;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const uint32_t h = (w[e / 2] >> (e & 1) * 16) & 0xffffu;
        if (!not_finite_h(h) || h == kNanRow) continue;
        const int* at = first + lane * E + e;
        const bool up = at[D] < lim, down = at[2 * D] < lim;
        uint32_t is = 0x7fffu;
        if (at[0] >= lim) {
          if (at[3 * D] < lim || !(up || down)) again = true;
          else if (up != down) is = up ? 0x7c00u : 0xfc00u;
        }
        w[e / 2] = (w[e / 2] & (0xffff0000u >> (e & 1) * 16)) | is << (e & 1) * 16;
      }
      if (__any_sync(0xffffffffu, again)) {
        float m, l, x[E];
        attend_keys<D, false>(a, (int64_t)it.q0 + tok0 + row / p.gp, h0 + row % p.gp, 0, it.k0, 0, 1, lim, lim, 0, lane, m, l, x);
        const float inv = inverse_sum(l);
#pragma unroll
        for (int e = 0; e < E / 2; ++e) w[e] = l == 0.f ? 0u : pack_half2(x[2 * e] * inv, x[2 * e + 1] * inv);
      }
#pragma unroll
      for (int e = 0; e < E / 2; ++e) reinterpret_cast<uint32_t*>(dst)[lane * (E / 2) + e] = w[e];
    }
  }
}

// 3-D map [tokens, heads, D] with `ld` elements between tokens; box 64 x heads x tokens
int token_map(CUtensorMap* m, const __half* p, int64_t tokens, int64_t heads, int64_t D, int64_t ld, int box_heads,
                     int box_tokens) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return TB_ERR_CUDA;
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)tokens};
  cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)ld * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_tokens};
  cuuint32_t es[3] = {1, 1, 1};
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<__half*>(p), dims, strides, box, es,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? TB_OK : TB_ERR_CUDA;
}

template <int D, int CG>
static int launch_tiles(PaArgs& p, int device, int sms, cudaStream_t s) {
  using C = PaCfg<D, CG>;
  const AttnArgs& a = p.a;
  CUtensorMap tq, tk, tv;
  int rc = token_map(&tq, a.q, a.T, a.Hq, D, a.ldq, p.gp, p.tok);
  // without any keys the maps of K and V are never used, but have to be maps
  const int64_t Tk = a.Tk ? a.Tk : 1;
  if (rc == TB_OK) rc = token_map(&tk, a.Tk ? a.k : a.q, Tk, a.Hkv, D, a.ldk, 1, C::kKRows);
  if (rc == TB_OK) rc = token_map(&tv, a.Tk ? a.v : a.q, Tk, a.Hkv, D, a.ldv, 1, kPaKeys);
  if (rc != TB_OK) return rc;
  auto* fn = prompt_attn_kernel<D, CG>;
  rc = ensure_dynamic_smem(reinterpret_cast<const void*>(fn), device, C::kSmem);
  if (rc != TB_OK) return rc;
  const int64_t span = (int64_t)p.tok * CG;
  p.magic = (unsigned)(((1ull << 32) + span - 1) / span);  // (of one token: overflows, and is not used)
  // at most: ceil(x) <= floor(x) + 1 per request
  const int64_t tiles = a.T / span + a.B, most = tiles * p.head_parts, clusters = sms / CG < most ? sms / CG : most;
  p.room = (double)a.B * (double)(a.T / span + 1) * p.head_parts > INT_MAX ? tiles : 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(clusters * CG));
  cfg.blockDim = dim3(kPaThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = CG;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, fn, tq, tk, tv, p);
  if (e != cudaSuccess) {
    record_cuda_error(e);
    return TB_ERR_CUDA;
  }
  return check_launch();
}

int launch_prompt_tiles(const AttnArgs& a, int64_t D, cudaStream_t s) {
  DeviceFacts f;
  const int rc = device_facts(&f);
  if (rc != TB_OK) return rc;
  PaArgs p;
  p.a = a;
  const int G = a.Hq / a.Hkv;
  p.gp = heads_per_tile(G);
  p.tok = 128 / p.gp;
  p.magic = 0;  // set with the tile's tokens
  p.head_parts = a.Hkv * (G / p.gp);
  if (D == 64) return launch_tiles<64, 1>(p, f.device, f.sms, s);
  if (D == 128) return launch_tiles<128, 2>(p, f.device, f.sms, s);
  return launch_tiles<256, 2>(p, f.device, f.sms, s);
}

}  // namespace tb
