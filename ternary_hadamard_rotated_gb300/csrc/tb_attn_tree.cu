// Attention of the newest tokens over the paged cache, on tcgen05: one token per request (decode), a
// run, or a tree of drafted tokens (csrc/tb_attention.cu has the entry point's checks).
//
// A tile is up to 128 rows of one KV head (row = token of the request x query head of the group) by
// 128 keys, as in the prompt kernel.  With the few rows of decode most of the MMA's 128 rows are
// idle, and that costs nothing: a tile's K and V are 512 D bytes, which at 6.8 TB/s over 152 SMs
// arrive in 5600 clocks for D = 256, its two MMA passes take 2048, its softmax about 2000.  So one
// kernel serves one row to 384, bound by the cache's bytes until several row tiles share them.
//
// Work: units of (request, head part, row tile, key tile), key tiles fastest, are cut into one equal
// contiguous range per SM, so the longest request is spread over as many SMs as its bytes call for.
// A CTA walks its range as segments (runs of key tiles of one item).  An item inside one range is
// written at once; one cut between CTAs leaves fp32 parts (O, maximum, sum) in the workspace, which a
// second kernel joins, all rows at once (with the last CTA of an item joining them alone, the calls
// below took at that time 26.6 us instead of 23.6 for the one context, 92 instead of 38 for the drafts).
//
// 64 contexts of 2000 to 30000 tokens, one token each (2.65 GB): 392 us, 0.99 of measured HBM.  One context of
// 4097: 16.6 us in a replayed graph, 18.5 a call, a chain of latencies (schedule, a tile's data, its products and
// softmax, parts, join).  9 requests of 5 to 16 drafts (53 MB): 26.0 and 30.9 us.
//
// Warps 0-3: softmax (thread = row) and epilogue; 4: TMA loads (pages by the block table); 5: MMAs.
// V rows past the request's last token are zeroed in shared memory before the MMAs read them (what
// lies there may be anything); a row whose output is not finite is computed again from the keys it
// sees alone (attend_keys), by the joining kernel, where nothing waits under a limit: a CTA a row, the keys shared
// out among its warps (one token over 131072 keys, one value of them NaN: 9.5 ms, without it 0.1).
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>

#include "tb_attention.cuh"
#include "tb_attn_tc.cuh"
#include "tb_host.h"

namespace tb {

constexpr int kTaThreads = 192;
constexpr int kTaKeys = 128;
constexpr int kTaSlot = 16384;
constexpr int kTaRing = 208 * 1024;  // Q and the ring
constexpr int kTaStage = 4 * 4096;   // a warp's 32 rows of output, 32 columns at a time
constexpr int kTaMaxCtas = 160;  // CTAs the workspace has room for

template <int D>
struct TaCfg {
  static constexpr int kChunks = D / 64;
  static constexpr int kKSlots = kChunks;                     // a slot: 64 elements of 128 keys
  static constexpr int kVKeys = kTaSlot / (D * 2);            // a slot: all elements of 128 / kChunks keys
  static constexpr int kVSlots = kTaKeys / kVKeys;
  // Q, then the ring: each row of Q that the tile has is there once (in eights), and the MMA's idle
  // rows read on into what follows, so that the ring gets what a full tile of Q would take
  static constexpr int kSmem = 1024 + kTaRing + kTaStage + 1024;
  static int slots(int rows) { return (kTaRing - kChunks * ((rows + 7) / 8 * 1024)) / kTaSlot; }
  static constexpr uint32_t kIdescQK = (1u << 4) | ((uint32_t)(kTaKeys >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
  static constexpr uint32_t kIdescPV = (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
  static constexpr uint32_t kTmemO = 2 * kTaKeys;
};

struct TaArgs {
  AttnArgs a;
  int gp, tok, head_parts, row_tiles;  // query heads and tokens per tile; row tiles at max_q tokens
  int rows;                            // rows of a part in the workspace: gp * tok
  int kbox, vbox;                      // keys per box of the K and V maps
  int slots;                           // slots of the ring
  float* part_o;                       // [2 * grid][rows][D]
  float* part_ml;                      // [2 * grid][rows][2]
  int2* meta;                          // [B * head_parts * row_tiles]: an item's first CTA, and how many
};

// Do a request's rows and length fit the arguments?  One that does not has no units and no entry in meta, which
// has room for max_q rows a request; the joining kernel writes its zeros.
TB_DEVI bool ta_fits(const AttnArgs& a, int64_t n, int64_t len) {
  return n <= a.max_q && len >= n && len <= a.max_pages << a.page_log2;
}

// a run of key tiles of one item
struct TaSegment {
  int b, hp, rt;
  int tile0, tiles, item_tiles;
  int64_t q0, n, len;            // the request's first row, rows, and cached tokens
  unsigned item_unit;            // the item's first unit
};

template <int D>
__global__ void __launch_bounds__(kTaThreads, 1)
    tree_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const TaArgs p) {
  using C = TaCfg<D>;
  const AttnArgs& a = p.a;
  extern __shared__ uint8_t ta_raw[];
  const uint32_t raw = smem_u32(ta_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = ta_raw + (base - raw);
  const int S = p.slots;
  const uint32_t qchunk = (uint32_t)(p.rows + 7) / 8 * 1024;  // bytes of 64 elements of Q's rows
  const uint32_t ring = base + C::kChunks * qchunk;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kTaRing + kTaStage);
  uint64_t* full = bars;
  uint64_t* empty = bars + S;
  uint64_t* q_full = bars + 2 * S;
  uint64_t* q_empty = q_full + 1;
  uint64_t* s_full = q_full + 2;  // [2]
  uint64_t* p_full = q_full + 4;  // [2]
  uint64_t* o_done = q_full + 6;
  uint64_t* o_free = q_full + 7;
  uint64_t* o_last = q_full + 8;  // the segment's last P V is done
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(q_full + 9);
  __shared__ volatile int aborted;
  __shared__ uint32_t granules[16];  // per key tile: which runs of 16 keys lie in a page of the cache

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    aborted = 0;
    for (int i = 0; i < S; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, 4);  // lane 0 of each softmax warp
    }
    mbar_init(o_done, 1);
    mbar_init(o_last, 1);
    mbar_init(o_free, 4);
    fence_barrier_init();
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (warp == 4 && lane < 3)
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(lane == 0 ? &tmQ : (lane == 1 ? &tmK : &tmV)))
                 : "memory");
  if (warp == 5) tmem_alloc(tmem_slot, 512);

  // ---- the schedule: every warp adds up the units of all requests itself
  struct Req {
    int64_t q0, n, len;
    int items, tiles;  // items 0: no rows, or not to be computed
    int bad;
  };
  auto request = [&](int b) {
    Req r;
    r.q0 = __ldg(a.q_start + b);
    r.n = __ldg(a.q_start + b + 1) - r.q0;
    r.len = __ldg(a.total + b);
    r.bad = 0;
    if (r.q0 < 0 || r.n < 0 || r.q0 + r.n > a.T) {
      r.bad = 1;
      r.n = 0;
    }
    if (r.n > 0 && !ta_fits(a, r.n, r.len)) {
      r.bad = 1;
      r.n = 0;
    }
    r.items = ((int)r.n + p.tok - 1) / p.tok * p.head_parts;  // (at most row_tiles * head_parts)
    const int64_t t = (r.len + kTaKeys - 1) / kTaKeys;
    r.tiles = t > 0 ? (int)t : 1;
    return r;
  };
  // (units fit 32 bits: the entry point checks that they do at max_q tokens and max_pages a request)
  const int per = (a.B + 31) / 32;
  unsigned upto = 0, own = 0;
  int any_bad = 0;
  for (int i = lane * per; i < (lane + 1) * per && i < a.B; ++i) {
    const Req r = request(i);
    own += (unsigned)r.items * (unsigned)r.tiles;
    any_bad |= r.bad;
  }
  upto = own;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const unsigned x = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += x;
  }
  const unsigned units = __shfl_sync(0xffffffffu, upto, 31);
  if (blockIdx.x == 0 && warp == 0 && any_bad) set_status(a.status, TB_DEV_BAD_LEN);
  // equal ranges: the first `more` CTAs have one unit more than the others (and no CTA of an item is
  // without a unit)
  const unsigned grid = units < gridDim.x ? units : gridDim.x;
  const unsigned share = grid ? units / grid : 0, more = units - share * grid, big = more * (share + 1);
  auto lo_of = [&](unsigned c) { return c * share + (c < more ? c : more); };
  auto owner = [&](unsigned u) { return u < big ? u / (share + 1) : more + (u - big) / share; };
  const bool works = blockIdx.x < grid;
  const unsigned lo = works ? lo_of(blockIdx.x) : 0, hi = works ? lo_of(blockIdx.x + 1) : 0;
  // the segment that starts at unit u (whole warps call this)
  auto segment = [&](unsigned u) {
    TaSegment s;
    const unsigned who = __ballot_sync(0xffffffffu, u < upto);
    const int src = __ffs(who) - 1;
    unsigned before = upto - own;
    int b = 0;
    if (lane == src) {
      for (b = lane * per;; ++b) {
        const Req r = request(b);
        const unsigned n = (unsigned)r.items * (unsigned)r.tiles;
        if (u < before + n) break;
        before += n;
      }
    }
    b = __shfl_sync(0xffffffffu, b, src);
    before = __shfl_sync(0xffffffffu, before, src);
    const Req r = request(b);
    const unsigned item = (u - before) / (unsigned)r.tiles;
    s.b = b;
    s.rt = (int)(item / (unsigned)p.head_parts);
    s.hp = (int)item - s.rt * p.head_parts;
    s.item_unit = before + item * (unsigned)r.tiles;
    s.tile0 = (int)(u - s.item_unit);
    s.item_tiles = r.tiles;
    s.tiles = hi - u < (unsigned)(r.tiles - s.tile0) ? (int)(hi - u) : r.tiles - s.tile0;
    s.q0 = r.q0;
    s.n = r.n;
    s.len = r.len;
    return s;
  };
  const int G = a.Hq / a.Hkv, parts = G / p.gp;

  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity) || aborted) return;
    if (!mbar_wait(bar, parity)) {
      aborted = 1;
      set_status(a.status, TB_DEV_TIMEOUT);
    }
  };

  // a place in the ring: slot, and the parity of the phase its next use completes
  struct Ring {
    int r = 0;
    uint32_t ph = 0;
  };
  auto advance = [&](Ring& x, int n) {
    x.r += n;
    if (x.r >= S) {
      x.r -= S;
      x.ph ^= 1;
    }
  };

  if (warp == 4) {
    // Each lane owns one box of a K tile and one of a V tile (at most 32 of each), waits for its slot
    // and issues it; the page numbers of a tile are fetched two tiles ahead of its use.
    int seg = 0, gt = 0;
    Ring at;
    int used = 0;  // slots handed out so far, up to S: a slot's first use waits for nobody
    const int page = 1 << a.page_log2;
    const int kb = kTaKeys / p.kbox, vb = C::kVKeys / p.vbox;
    // K: slot (chunk) lane / kb, box lane % kb of it
    const bool k_on = lane < C::kKSlots * kb;
    const int k_slot = lane / kb, k_key = (lane - k_slot * kb) * p.kbox;
    // V: slot lane / (vb * chunks), keys and chunk within it
    const bool v_on = lane < C::kVSlots * vb * C::kChunks;
    const int v_slot = lane / (vb * C::kChunks), v_rest = lane - v_slot * (vb * C::kChunks);
    const int v_in = v_rest / C::kChunks * p.vbox, v_c = v_rest % C::kChunks;
    const int v_key = v_slot * C::kVKeys + v_in;
    for (unsigned u = lo; u < hi;) {
      const TaSegment s = segment(u);
      u += s.tiles;
      const int hk = s.hp / parts, h0 = hk * G + (s.hp % parts) * p.gp;
      const int32_t* row = a.table + (int64_t)s.b * a.max_pages;
      // page of the 16-key run that this lane (0-7) looks up; -1 past the last token or the segment
      auto look = [&](int i) -> int {
        const int64_t j = (int64_t)(s.tile0 + i) * kTaKeys + (lane & 7) * 16;
        return i < s.tiles && j < s.len ? __ldg(row + (j >> a.page_log2)) : -1;
      };
      // its row of the cache's map; out of the map, where boxes are filled with zeros, for no page
      auto coord = [&](int i, int pg) -> int {
        const int64_t j = (int64_t)(s.tile0 + i) * kTaKeys + (lane & 7) * 16;
        const bool ok = pg >= 0 && pg < a.pages;
        if (!ok && i < s.tiles && j < s.len && lane < 8) set_status(a.status, TB_DEV_BAD_SLOT);
        return ok ? (int)(pg * a.Hkv + hk) : -1;
      };
      const int none = (int)(a.pages * a.Hkv);
      auto acquire = [&](int slot, bool first) -> int {  // this lane's slot, its bytes announced by one lane
        Ring x = at;
        advance(x, slot);
        if (used + slot >= S) wait(empty + x.r, x.ph ^ 1);
        if (first) mbar_arrive_expect_tx(full + x.r, kTaSlot);
        return x.r;
      };
      auto load_k = [&](int i, int z) {
        const unsigned ok = __ballot_sync(0xffffffffu, z >= 0) & 0xffu;
        if (lane == 0) *reinterpret_cast<volatile uint32_t*>(granules + ((gt + i) & 15)) = ok;
        __syncwarp();
        const int zz = __shfl_sync(0xffffffffu, z, k_key / 16);
        if (k_on) {
          const int r = acquire(k_slot, k_key == 0);
          tma_load_3d<1>(ring + r * kTaSlot + k_key * 128, &tmK, k_slot * 64,
                         ((s.tile0 + i) * kTaKeys + k_key) & (page - 1), zz < 0 ? none : zz, smem_u32(full + r));
        }
        __syncwarp();
        advance(at, C::kKSlots);
        used += C::kKSlots;
      };
      auto load_v = [&](int i, int z) {
        const int zz = __shfl_sync(0xffffffffu, z, (v_key / 16) & 7);
        if (v_on) {
          const int r = acquire(v_slot, v_rest == 0);
          tma_load_3d<1>(ring + r * kTaSlot + v_c * (C::kVKeys * 128) + v_in * 128, &tmV, v_c * 64,
                         ((s.tile0 + i) * kTaKeys + v_key) & (page - 1), zz < 0 ? none : zz, smem_u32(full + r));
        }
        __syncwarp();
        advance(at, C::kVSlots);
        used += C::kVSlots;
      };
      int z0 = coord(0, look(0)), ahead = look(1);
      load_k(0, z0);
      if (lane == 0) {
        if (seg > 0) wait(q_empty, (seg - 1) & 1);
        mbar_arrive_expect_tx(q_full, C::kChunks * 128 * p.gp * p.tok);
        for (int c = 0; c < C::kChunks; ++c)
          tma_load_3d<1>(base + c * qchunk, &tmQ, c * 64, h0, (int)(s.q0 + (int64_t)s.rt * p.tok), smem_u32(q_full));
      }
      __syncwarp();
      for (int i = 0; i < s.tiles; ++i) {
        const int z1 = coord(i + 1, ahead);
        ahead = look(i + 2);
        if (i + 1 < s.tiles) load_k(i + 1, z1);
        load_v(i, z0);
        z0 = z1;
      }
      gt += s.tiles;
      ++seg;
    }
    if (aborted) {  // a wait gave up: leave the copies in flight time to land before the CTA ends
      const uint64_t t = globaltimer_ns();
      while (globaltimer_ns() - t < 1000000) {
      }
    }
  } else if (warp == 5) {
    int seg = 0, gt = 0;
    Ring at;
    for (unsigned u = lo; u < hi;) {
      const TaSegment s = segment(u);
      u += s.tiles;
      if (lane == 0) {
        // descriptors of place 0; the address field counts 16 bytes, and no sum carries out of it
        const uint64_t qdesc = smem_desc_sw128(base, 1024), kdesc = smem_desc_sw128(ring, 1024);
        const uint64_t vdesc = smem_desc_mn128(ring, C::kVKeys * 128, 1024);
        wait(q_full, seg & 1);
        tmem_fence_after();
        auto qk = [&](int i) {
          const uint32_t d = tmem + (uint32_t)((gt + i) & 1) * kTaKeys;
#pragma unroll
          for (int c = 0; c < C::kChunks; ++c) {
            const int r = at.r;
            wait(full + r, at.ph);
            tmem_fence_after();
            const uint64_t qd = qdesc + c * (qchunk >> 4), kd = kdesc + r * (kTaSlot >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) mma_f16_ss<1>(d, qd + kk * 2, kd + kk * 2, C::kIdescQK, (c | kk) != 0);
            mma_commit(empty + r);
            advance(at, 1);
          }
          mma_commit(s_full + ((gt + i) & 1));
        };
        qk(0);
        for (int i = 0; i < s.tiles; ++i) {
          if (i + 1 < s.tiles) qk(i + 1);
          else mma_commit(q_empty);
          if (i == 0 && seg > 0) wait(o_free, (seg - 1) & 1);  // the last segment's O has been read
          wait(p_full + ((gt + i) & 1), ((gt + i) >> 1) & 1);
          tmem_fence_after();
#pragma unroll
          for (int v = 0; v < C::kVSlots; ++v) {
            const int r = at.r;
            wait(full + r, at.ph);
            tmem_fence_after();
            const uint64_t vd = vdesc + r * (kTaSlot >> 4);
#pragma unroll
            for (int kk = 0; kk < C::kVKeys / 16; ++kk)
              mma_f16_ts<1>(tmem + C::kTmemO, tmem + (uint32_t)((gt + i) & 1) * kTaKeys + (v * (C::kVKeys / 16) + kk) * 8,
                            vd + kk * (2048 >> 4), C::kIdescPV, (i | v | kk) != 0);
            mma_commit(empty + r);
            advance(at, 1);
          }
          mma_commit(o_done);
        }
        mma_commit(o_last);
      }
      __syncwarp();
      gt += s.tiles;
      ++seg;
    }
  } else {
    const int row = warp * 32 + lane;
    const uint32_t mine = tmem + ((uint32_t)warp << 21);
    const float sc = a.scale_log2;
    const int tr = row / p.gp;
    int gt = 0, seg = 0;
    int64_t it = 0;  // slots used before this segment
    for (unsigned u = lo; u < hi;) {
      const TaSegment s = segment(u);
      u += s.tiles;
      if (row == 0 && s.tile0 == 0)  // where the item's parts are, for the joining kernel
        p.meta[((int64_t)s.b * p.head_parts + s.hp) * p.row_tiles + s.rt] =
            make_int2((int)blockIdx.x, (int)(owner(s.item_unit + (unsigned)s.item_tiles - 1) - blockIdx.x) + 1);
      const int hk = s.hp / parts;
      const int head = hk * G + (s.hp % parts) * p.gp + row - tr * p.gp;
      const int64_t tq = (int64_t)s.rt * p.tok + tr;  // token of the request
      const bool live = tr < p.tok && tq < s.n;
      __half* dst = a.o + ((s.q0 + tq) * a.Hq + head) * D;
      const int64_t prefix = s.len - s.n;
      uint64_t word = 0;
      if (live) {
        word = a.tree ? (uint64_t)__ldg(reinterpret_cast<const long long*>(a.tree) + s.q0 + tq)
                      : ~0ull >> (63 - (int)tq);
        if (s.n < 64) word &= (1ull << s.n) - 1;
      }
      float m = -INFINITY, l = 0.f;
      for (int i = 0; i < s.tiles; ++i) {
        const int g = gt + i, buf = g & 1;
        const int64_t j0 = (int64_t)(s.tile0 + i) * kTaKeys;
        wait(s_full + buf, (g >> 1) & 1);
        tmem_fence_after();
        float x[kTaKeys];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(mine + buf * kTaKeys + c * 32, x + 32 * c);
        tmem_wait_ld();
        const uint32_t pages_ok = *reinterpret_cast<volatile uint32_t*>(granules + (g & 15));
        if (j0 + kTaKeys > prefix || pages_ok != 0xffu) {
          // which of the tile's keys the row sees: the prefix, then the word's bits
          const int64_t d = prefix - j0;
          uint64_t low, high;
          if (d >= 128) low = high = ~0ull;
          else if (d >= 64) {
            low = ~0ull;
            high = d == 64 ? word : ((1ull << (d - 64)) - 1) | (word << (d - 64));
          } else if (d > 0) {
            low = ((1ull << d) - 1) | (word << d);
            high = word >> (64 - d);
          } else {
            low = d > -64 ? word >> (-d) : 0;
            high = 0;
          }
          uint32_t seen[4] = {(uint32_t)low, (uint32_t)(low >> 32), (uint32_t)high, (uint32_t)(high >> 32)};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            seen[w] &= ((pages_ok >> (2 * w)) & 1 ? 0xffffu : 0u) | ((pages_ok >> (2 * w + 1)) & 1 ? 0xffff0000u : 0u);
#pragma unroll
            for (int c = 0; c < 32; ++c) x[w * 32 + c] = (seen[w] >> c) & 1 ? x[w * 32 + c] : -INFINITY;
          }
        }
        float mx[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) mx[c] = fmaxf(x[c], x[c + 4]);
#pragma unroll
        for (int c = 8; c < kTaKeys; c += 4)
#pragma unroll
          for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], x[c + e]);
        const float tmax = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;
        const bool grow = tmax > m + 8.f || (m == -INFINITY && tmax > -INFINITY);
        if (__any_sync(0xffffffffu, grow && i > 0 && live)) {
          const float f = grow ? (m == -INFINITY ? 0.f : ex2(m - tmax)) : 1.f;
          l *= f;
          // a parity tells only neighbouring phases apart: tile i - 2's is over, as S of tile i came after
          // it, and tile i's cannot be over before this warp's part of P is there
          wait(o_done, (g - 1) & 1);
          tmem_fence_after();
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float o[32];
            tmem_ld32(mine + C::kTmemO + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= f;
            tmem_st32(mine + C::kTmemO + c, reinterpret_cast<uint32_t(&)[32]>(o));
          }
          tmem_wait_st();
        }
        if (grow) m = tmax;
        const float ms = m == -INFINITY ? 0.f : kPTop - m;
        float2 acc0 = make_float2(0.f, 0.f), acc1 = acc0;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t pk[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const int c = half * 64 + e * 2;
            float2 y = fma_f32x2(make_float2(x[c], x[c + 1]), make_float2(sc, sc), make_float2(ms, ms));
            y.x = ex2(y.x);
            y.y = ex2(y.y);
            if (e & 1) acc1 = add_f32x2(acc1, y);
            else acc0 = add_f32x2(acc0, y);
            pk[e] = pack_half2(y.x, y.y);
          }
          tmem_st32(mine + buf * kTaKeys + half * 32, pk);
        }
        acc0 = add_f32x2(acc0, acc1);
        l += acc0.x + acc0.y;
        tmem_wait_st();
        tmem_fence_before();
        const int64_t tail = s.len - j0;  // keys of this tile that exist
        if (tail < kTaKeys) {
          // V's rows past the last token: zeroed once the tile's V is here.  Its slots follow the
          // segment's K tiles and earlier V tiles in the ring; every earlier use of them is over,
          // since S of this tile came after it, so one phase's parity cannot be taken for another's.
          const int64_t first = it + (int64_t)s.tiles * C::kKSlots + (int64_t)i * C::kVSlots;
          for (int v = (int)(tail / C::kVKeys); v < C::kVSlots; ++v) {
            const int r = (int)((first + v) % S);
            wait(full + r, (uint32_t)((first + v) / S) & 1);
            const int k0 = tail > v * C::kVKeys ? (int)tail - v * C::kVKeys : 0;
            for (int e = row; e < (C::kVKeys - k0) * C::kChunks * 8; e += 128) {
              const int c = e / ((C::kVKeys - k0) * 8), w = e - c * ((C::kVKeys - k0) * 8);
              asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(ring + r * kTaSlot + c * (C::kVKeys * 128) +
                                                                         k0 * 128 + w * 16),
                           "r"(0)
                           : "memory");
            }
          }
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + buf);
      }
      gt += s.tiles;
      it += (int64_t)s.tiles * (C::kKSlots + C::kVSlots);
      // ---- the segment's O: the output, or a part
      wait(o_last, seg & 1);
      ++seg;
      tmem_fence_after();
      const bool whole = s.tiles == s.item_tiles;
      const int64_t slot = (int64_t)blockIdx.x * 2 + (s.tile0 == 0);
      const float inv = whole ? inverse_sum(l) : 1.f;
      const bool none = l == 0.f;  // the row saw nothing here: what the MMAs left is 0 times V
      // through shared memory, so that a store instruction covers whole runs of a few rows (a thread's own
      // row at a time it touches 32: the drafts above took 28.0 us instead of 25.5 then)
      const uint32_t stage = base + kTaRing + (uint32_t)warp * 4096u;
      const unsigned rows = __ballot_sync(0xffffffffu, live);
      const int64_t begin = dst - a.o;
      float* part = p.part_o + (slot * p.rows + warp * 32) * D;
      auto piece = [&](int r, int pc) { return stage + (uint32_t)r * 128u + (((uint32_t)pc ^ ((uint32_t)r & 7u)) << 4); };
#pragma unroll 1
      for (int c = 0; rows && c < D; c += 32) {
        float o[32];
        tmem_ld32(mine + C::kTmemO + c, o);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = none ? 0.f : o[e];
        if (whole) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t w[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) w[y] = pack_half2(o[e * 8 + 2 * y] * inv, o[e * 8 + 2 * y + 1] * inv);
            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(piece(lane, e)), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                         : "memory");
          }
          __syncwarp();
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int r = x * 8 + (lane >> 2), pc = lane & 3;
            const uint4 w = ld_shared_v4(piece(r, pc));
            const int64_t to = __shfl_sync(0xffffffffu, begin, r);
            if (rows >> r & 1) *reinterpret_cast<uint4*>(a.o + to + c + pc * 8) = w;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(piece(lane, e)), "f"(o[e * 4]), "f"(o[e * 4 + 1]),
                         "f"(o[e * 4 + 2]), "f"(o[e * 4 + 3])
                         : "memory");
          __syncwarp();
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            const int r = x * 4 + (lane >> 3), pc = lane & 7;
            const uint4 w = ld_shared_v4(piece(r, pc));
            if (rows >> r & 1) *reinterpret_cast<uint4*>(part + r * D + c + pc * 4) = w;
          }
        }
        __syncwarp();
      }
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_free);
      if (whole)
        for (unsigned lost = __ballot_sync(0xffffffffu, live && !(l < INFINITY)); lost; lost &= lost - 1) {
          const int64_t to = __shfl_sync(0xffffffffu, begin, __ffs(lost) - 1);
          for (int c = lane; c < D; c += 32) a.o[to + c] = __ushort_as_half((unsigned short)kNanRow);
        }
      else if (live) *reinterpret_cast<float2*>(p.part_ml + (slot * p.rows + row) * 2) = make_float2(m, l);
    }
  }

  tmem_fence_before();
  __syncthreads();
  if (warp == 5) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- parts -> output
// One CTA of W warps per (row, head): the warps share the parts of the row's item, the lanes the columns;
// rows of items that one CTA finished are done already.  The order of the sums is fixed by the schedule.  A row that
// is not finite, of parts or done, is made again from its keys.
template <int D, int W>
__global__ void __launch_bounds__(W * 32, 32 / W) tree_join_kernel(const TaArgs p) {
  const AttnArgs& a = p.a;
  constexpr int E = D / 32;  // columns of a lane: lane * 2 + 64 i (+ 1)
  __shared__ float acc_s[W][D];
  __shared__ float ml_s[W][2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = blockIdx.x / a.Hq;
  const int h = (int)(blockIdx.x - t * a.Hq);
  int b = 0;
  {
    int hi = a.B - 1;  // the last request that begins at or before row t
    while (b < hi) {
      const int mid = (b + hi + 1) >> 1;
      if (__ldg(a.q_start + mid) <= t) b = mid;
      else hi = mid - 1;
    }
  }
  const int64_t q0 = __ldg(a.q_start + b), n = __ldg(a.q_start + b + 1) - q0, len = __ldg(a.total + b);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the parts are written
  if (q0 < 0 || t < q0 || t >= q0 + n || q0 + n > a.T) return;
  if (!ta_fits(a, n, len)) {
    for (int c = threadIdx.x * 2; c < D; c += W * 64) *reinterpret_cast<__half2*>(a.o + (t * a.Hq + h) * D + c) = __floats2half2_rn(0.f, 0.f);
    return;
  }
  const int G = a.Hq / a.Hkv, parts = G / p.gp, hk = h / G;
  const int hp = hk * parts + (h - hk * G) / p.gp;
  const int tq = (int)(t - q0), rt = tq / p.tok;
  const int2 meta = p.meta[((int64_t)b * p.head_parts + hp) * p.row_tiles + rt];
  __half* out = a.o + (t * a.Hq + h) * D;
  bool redo = false;
  if (meta.y < 2) {
    bool bad = false;
    for (int c = threadIdx.x * 2; c < D; c += W * 64) {
      const uint32_t x[1] = {__ldcg(reinterpret_cast<const unsigned*>(out + c))};
      bad |= any_to_mend(x);
    }
    redo = __syncthreads_or(bad);
    if (!redo) return;
  }
  const int row = (tq - rt * p.tok) * p.gp + (h - hk * G) % p.gp;
  // part i is CTA meta.x + i's: its first segment (0), or for the item's first CTA its last (1)
  auto at = [&](int i) { return (int64_t)(2 * (meta.x + i) + (i == 0)) * p.rows + row; };
  for (;; redo = true) {
    // each warp takes every W-th part, or key, with a running maximum; parts without a key have a sum of 0 and
    // zeros, whatever their weight
    float acc[E], M = -INFINITY, L = 0.f;
    if (!redo) {
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 4
      for (int i = warp; i < meta.y; i += W) {
        const float2 ml = __ldcg(reinterpret_cast<const float2*>(p.part_ml + at(i) * 2));
        const float* src = p.part_o + at(i) * D + lane * 2;
        float2 y[E / 2];
#pragma unroll
        for (int e = 0; e < E / 2; ++e) y[e] = __ldcg(reinterpret_cast<const float2*>(src + e * 64));
        const float m2 = fmaxf(M, ml.x);
        const float c = M == m2 ? 1.f : ex2(M - m2), w = ml.x == m2 ? 1.f : ex2(ml.x - m2);
        L = fmaf(w, ml.y, L * c);
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
          acc[2 * e] = fmaf(w, y[e].x, acc[2 * e] * c);
          acc[2 * e + 1] = fmaf(w, y[e].y, acc[2 * e + 1] * c);
        }
        M = m2;
      }
#pragma unroll
      for (int e = 0; e < E; e += 2)
        *reinterpret_cast<float2*>(&acc_s[warp][e * 32 + lane * 2]) = make_float2(acc[e], acc[e + 1]);
    } else {
      uint64_t word = a.tree ? (uint64_t)__ldg(reinterpret_cast<const long long*>(a.tree) + t) : ~0ull >> (63 - tq);
      if (n < 64) word &= (1ull << n) - 1;
      attend_keys<D, true>(a, t, h, b, 0, warp, W, len, len - n, word, lane, M, L, acc);
#pragma unroll
      for (int e = 0; e < E; e += 2) *reinterpret_cast<float2*>(&acc_s[warp][lane * E + e]) = make_float2(acc[e], acc[e + 1]);
    }
    if (lane == 0) {
      ml_s[warp][0] = L;
      ml_s[warp][1] = M;
    }
    __syncthreads();
    M = -INFINITY;
#pragma unroll
    for (int w = 0; w < W; ++w) M = fmaxf(M, ml_s[w][1]);
    float f[W];
    L = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      f[w] = ml_s[w][1] == M ? 1.f : ex2(ml_s[w][1] - M);
      L = fmaf(f[w], ml_s[w][0], L);
    }
    const float inv = inverse_sum(L);
    bool bad = false;  // (a sum that is not finite leaves NaN, and that is right)
    for (int c = threadIdx.x * 2; c < D; c += W * 64) {
      float x = 0.f, y = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        x = fmaf(f[w], acc_s[w][c], x);
        y = fmaf(f[w], acc_s[w][c + 1], y);
      }
      bad |= L < INFINITY && (!(fabsf(x) < INFINITY) || !(fabsf(y) < INFINITY));
      *reinterpret_cast<__half2*>(out + c) = L == 0.f ? __floats2half2_rn(0.f, 0.f) : __floats2half2_rn(x * inv, y * inv);
    }
    if (redo || !__syncthreads_or(bad)) break;
  }
}

static void tile_shape(int64_t Hq, int64_t Hkv, int64_t max_q, int* gp, int* tok) {
  *gp = heads_per_tile((int)(Hq / Hkv));
  *tok = 128 / *gp;
  if (*tok > max_q) *tok = (int)max_q;
}

int64_t tree_items(int64_t B, int64_t max_q, int64_t Hq, int64_t Hkv) {
  int gp, tok;
  tile_shape(Hq, Hkv, max_q, &gp, &tok);
  return B * Hkv * (Hq / Hkv / gp) * ((max_q + tok - 1) / tok);
}

size_t tree_workspace(int64_t B, int64_t max_q, int64_t Hq, int64_t Hkv, int64_t D) {
  int gp, tok;
  tile_shape(Hq, Hkv, max_q, &gp, &tok);
  const int64_t items = tree_items(B, max_q, Hq, Hkv);
  const int64_t rows = 2 * kTaMaxCtas * (int64_t)gp * tok;
  return (size_t)((items * 8 + 255) / 256 * 256 + rows * 2 * 4 + rows * D * 4);
}

template <int D>
static int launch_tree(TaArgs& p, const DeviceFacts& f, cudaStream_t s) {
  using C = TaCfg<D>;
  const AttnArgs& a = p.a;
  const int page = 1 << a.page_log2;
  p.kbox = page < kTaKeys ? page : kTaKeys;
  p.vbox = page < C::kVKeys ? page : C::kVKeys;
  CUtensorMap tq, tk, tv;
  int rc = token_map(&tq, a.q, a.T, a.Hq, D, a.ldq, p.gp, p.tok);
  // the cache as [pages * Hkv, page, D]
  if (rc == TB_OK) rc = token_map(&tk, a.k, a.pages * a.Hkv, page, D, (int64_t)page * D, p.kbox, 1);
  if (rc == TB_OK) rc = token_map(&tv, a.v, a.pages * a.Hkv, page, D, (int64_t)page * D, p.vbox, 1);
  if (rc != TB_OK) return rc;
  rc = ensure_dynamic_smem(reinterpret_cast<const void*>(tree_attn_kernel<D>), f.device, C::kSmem);
  if (rc != TB_OK) return rc;
  const int grid = f.sms < kTaMaxCtas ? f.sms : kTaMaxCtas;
  p.slots = C::slots(p.rows) < 16 ? C::slots(p.rows) : 16;
  tree_attn_kernel<D><<<grid, kTaThreads, C::kSmem, s>>>(tq, tk, tv, p);
  rc = check_launch();
  if (rc != TB_OK) return rc;
  // the joining kernel starts while the last CTAs still run and waits for them on the device.  Sixteen warps
  // a row while every row has an SM of its own, else four.  Contexts of 4097, 24 rows each, both kernels, with
  // sixteen and with four: 24 rows 16.8 and 18.1 us, 48 21.5 and 22.1, 144 28.4 and 28.4, 192 36.1 and 36.1, 384 56.7
  // and 53.4, 768 98.7 and 92.2; contexts of 1000 the same way round.
  const bool few = a.T * a.Hq <= f.sms;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.T * a.Hq));
  cfg.blockDim = dim3(few ? 512 : 128);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = few ? cudaLaunchKernelEx(&cfg, tree_join_kernel<D, 16>, p) : cudaLaunchKernelEx(&cfg, tree_join_kernel<D, 4>, p);
  if (e != cudaSuccess) {
    record_cuda_error(e);
    return TB_ERR_CUDA;
  }
  return check_launch();
}

int launch_tree_tiles(const AttnArgs& a, int64_t D, void* workspace, cudaStream_t s) {
  DeviceFacts f;
  const int rc = device_facts(&f);
  if (rc != TB_OK) return rc;
  TaArgs p;
  p.a = a;
  tile_shape(a.Hq, a.Hkv, a.max_q, &p.gp, &p.tok);
  p.head_parts = a.Hkv * (a.Hq / a.Hkv / p.gp);
  p.row_tiles = (a.max_q + p.tok - 1) / p.tok;
  p.rows = p.gp * p.tok;
  const int64_t items = tree_items(a.B, a.max_q, a.Hq, a.Hkv);
  uint8_t* w = static_cast<uint8_t*>(workspace);
  p.meta = reinterpret_cast<int2*>(w);
  p.part_ml = reinterpret_cast<float*>(w + (items * 8 + 255) / 256 * 256);
  p.part_o = p.part_ml + 2 * kTaMaxCtas * (int64_t)p.rows * 2;
  if (D == 64) return launch_tree<64>(p, f, s);
  if (D == 128) return launch_tree<128>(p, f, s);
  return launch_tree<256>(p, f, s);
}

}  // namespace tb
