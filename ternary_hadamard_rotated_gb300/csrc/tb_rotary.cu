// Rotary positions: q and k turned by their tokens' positions, k and v written to the paged cache on the way.
//
// The pair (a, b) = (x_i, x_{i + R/2}) or (x_2i, x_{2i+1}), i < R/2, of a head becomes
//   amplitude * (a cos - b sin, a sin + b cos)  of the angle pos * f_i;
// a head's elements from R on stay as they are.
//
// Angles are kept in turns (of 2 pi) as 64-bit fractions: turns_i = f_i / 2 pi mod 1 times 2^64, so that
// pos * turns_i mod 2^64 is the angle without its whole turns, exactly, however far the position (an fp32
// product pos * f_i of 262144 radians is off by 0.016; the fraction by 2^-33 turns for positions up to 2^31,
// beside the 53 bits of f_i itself).  Its signed value goes to fp32 with 24 bits of its own and from there into
// sincospif.
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>

#include "tb_common.cuh"
#include "tb_host.h"

namespace tb {

constexpr int32_t kRotaryMagic = 0x52544f52;
constexpr int kRotaryMaxR = 1024;

struct RotaryPlan {  // in device memory; the pairs' turns follow, uint64 [R/2]
  int32_t magic, R;
  float amplitude;
  int32_t pad;
};
static_assert(sizeof(RotaryPlan) == 16, "the turns follow the head of the plan on a 16-byte boundary");

// ---------------------------------------------------------------- plan
struct RotaryPlanArgs {
  double base, factor, original, beta_fast, beta_slow, amplitude;
  const double* freqs;
  int scaling, R;
};

__global__ void rotary_plan_kernel(const RotaryPlanArgs a, RotaryPlan* __restrict__ plan, int32_t* __restrict__ status) {
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  const int i = threadIdx.x;
  const double R = a.R;
  if (i == 0) {
    plan->magic = kRotaryMagic;
    plan->R = a.R;
    double amp = a.amplitude;
    if (amp == 0.0) amp = a.scaling == TB_ROTARY_PARTS && a.factor > 1.0 ? 0.1 * log(a.factor) + 1.0 : 1.0;
    plan->amplitude = (float)amp;
    plan->pad = 0;
  }
  if (i >= a.R / 2) return;
  double f;
  if (a.freqs) {
    f = a.freqs[i];
  } else {
    const double base = a.scaling == TB_ROTARY_BASE ? a.base * pow(a.factor, R / (R - 2.0)) : a.base;
    f = pow(base, -2.0 * i / R);
    if (a.scaling == TB_ROTARY_LINEAR) f /= a.factor;
    if (a.scaling == TB_ROTARY_PARTS) {
      // the (fractional) pair that turns beta times over the original context: base^(2 i / R) = original / (2 pi beta)
      const double low = floor(R * log(a.original / (a.beta_fast * kTwoPi)) / (2.0 * log(a.base)));
      const double high = ceil(R * log(a.original / (a.beta_slow * kTwoPi)) / (2.0 * log(a.base)));
      const double lo = fmax(low, 0.0), hi = fmin(high, R - 1.0);
      const double ramp = fmin(fmax((i - lo) / fmax(hi - lo, 1e-3), 0.0), 1.0);
      f = f / a.factor * ramp + f * (1.0 - ramp);
    }
  }
  double t = f / kTwoPi;
  t -= floor(t);
  unsigned long long turns = 0;
  if (isfinite(f)) {
    if (t < 1.0) turns = (unsigned long long)(t * 18446744073709551616.0);  // (a tiny negative f leaves 1.0: a whole turn)
  } else {
    set_status(status, TB_DEV_BAD_PLAN);
  }
  reinterpret_cast<unsigned long long*>(plan + 1)[i] = turns;
}

// ---------------------------------------------------------------- rotation, any head
struct RotaryArgs {
  const __half *q, *k, *v;
  __half *q_out, *k_out, *k_cache, *v_cache;
  int64_t ldq, ldk, ldv, ldqo, ldko, T, n_slots;
  const int32_t* pos;
  const int64_t* slots;
  const RotaryPlan* plan;
  int32_t* status;
  int Hq, Hk, D, R, pairs, inverse, page_log2;
  int q_copy, k_copy;   // 16-byte pieces of a head (pairs of elements in the narrow form) that are only copied
  int rot;              // rotations of a head: of 8 pairs each (of one in the narrow form)
  int per_token, tile;  // pieces of work of a token, tokens of a CTA
  int split;            // CTAs that share a tile's pieces
};

struct Eight {
  float v[8];
};

TB_DEVI Eight unpack8(uint4 x) {
  Eight r;
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    r.v[2 * i] = f.x;
    r.v[2 * i + 1] = f.y;
  }
  return r;
}
TB_DEVI uint4 pack8(const Eight& e) {
  return make_uint4(pack_half2(e.v[0], e.v[1]), pack_half2(e.v[2], e.v[3]), pack_half2(e.v[4], e.v[5]), pack_half2(e.v[6], e.v[7]));
}

constexpr int kRotaryThreads = 256;
constexpr int kRotaryAngles = 2048;  // (token, pair) angles a CTA holds: 16 KB

// WIDE: R a multiple of 16, rotations of 8 pairs by two 16-byte loads; otherwise pair by pair, 2 bytes an access.
// 20000 tokens of 32/8 heads of 80 and 96, all turned: 53 and 60 us in a graph (floors 38 and 45); 12000 of 24/4 heads of 192:
// 48 (38).  Of 34 turned elements, pair by pair: 251 us for 12000 tokens of 24/4 heads of 256 (floor 51), 267 for 20000 of 32/8
// heads of 128 (60).  64 tokens: 2.6 us for heads of 80, 4.6 with 34 turned of 128 (rows of 128, all turned: 3.5).
template <bool WIDE>
__global__ void __launch_bounds__(kRotaryThreads) rotary_kernel(const RotaryArgs a) {
  __shared__ __align__(16) float cosines[kRotaryAngles], sines[kRotaryAngles];
  asm volatile("griddepcontrol.wait;" ::: "memory");  // what came before is over (see launch_early)
  if (a.plan->magic != kRotaryMagic || a.plan->R != a.R) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) set_status(a.status, TB_DEV_BAD_PLAN);
    return;
  }
  const int half = a.R / 2;
  const float amp = a.plan->amplitude;
  const unsigned long long* turns = reinterpret_cast<const unsigned long long*>(a.plan + 1);
  const unsigned row_q = a.Hq * (a.rot + a.q_copy), row_k = a.Hk * (a.rot + a.k_copy);
  const int64_t head = (int64_t)a.D << a.page_log2;  // of the cache: elements from one head to the next
  for (int64_t t0 = (int64_t)blockIdx.x * a.tile; t0 < a.T; t0 += (int64_t)gridDim.x * a.tile) {
    const int n = (int)(a.T - t0 < a.tile ? a.T - t0 : a.tile);
    __syncthreads();  // the tile before has been read
    for (int i = threadIdx.x; i < n * half; i += kRotaryThreads) {
      const int t = i / half;
      const unsigned long long at = (unsigned long long)(long long)a.pos[t0 + t] * turns[i - t * half];
      float s, c;
      sincospif(__ll2float_rn((long long)at) * 0x1p-63f, &s, &c);
      cosines[i] = amp * c;
      sines[i] = a.inverse ? -amp * s : amp * s;
    }
    __syncthreads();
    const unsigned work = (unsigned)n * a.per_token;
    for (unsigned i = blockIdx.y * kRotaryThreads + threadIdx.x; i < work; i += a.split * kRotaryThreads) {
      const unsigned t = i / a.per_token;
      unsigned r = i - t * a.per_token;
      const int64_t tok = t0 + t;
      int64_t slot = -1;
      if (a.slots && r >= row_q) {
        slot = a.slots[tok];
        if (slot >= a.n_slots) {
          set_status(a.status, TB_DEV_BAD_SLOT);
          slot = -1;
        }
      }
      const int64_t place = slot < 0 ? 0 : (((slot >> a.page_log2) * a.Hk << a.page_log2) + (slot & ((1ll << a.page_log2) - 1))) * a.D;
      if (r >= row_q + row_k) {  // v: copied
        if (slot < 0) continue;
        r -= row_q + row_k;
        const unsigned h = r / (a.D / 8), c = r - h * (a.D / 8);
        *reinterpret_cast<uint4*>(a.v_cache + place + h * head + c * 8) = __ldcs(reinterpret_cast<const uint4*>(a.v + tok * a.ldv + h * a.D + c * 8));
        continue;
      }
      const bool is_q = r < row_q;
      if (!is_q) r -= row_q;
      const unsigned per = a.rot + (is_q ? a.q_copy : a.k_copy), h = r / per, c = r - h * per;
      const __half* src = is_q ? a.q + tok * a.ldq + h * a.D : a.k + tok * a.ldk + h * a.D;
      __half* dst = is_q ? a.q_out + tok * a.ldqo + h * a.D : a.k_out ? a.k_out + tok * a.ldko + h * a.D : nullptr;
      __half* cached = slot < 0 ? nullptr : a.k_cache + place + h * head;
      if (!dst && !cached) continue;
      if (c < (unsigned)a.rot) {
        if constexpr (WIDE) {
          const unsigned p = c * 8;
          const unsigned lo = a.pairs ? 2 * p : p, hi = a.pairs ? 2 * p + 8 : p + half;
          const Eight x = unpack8(*reinterpret_cast<const uint4*>(src + lo)), y = unpack8(*reinterpret_cast<const uint4*>(src + hi));
          Eight u, w;
          const float *cs = cosines + t * half + p, *sn = sines + t * half + p;
          if (a.pairs) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              u.v[2 * j] = x.v[2 * j] * cs[j] - x.v[2 * j + 1] * sn[j];
              u.v[2 * j + 1] = x.v[2 * j] * sn[j] + x.v[2 * j + 1] * cs[j];
              w.v[2 * j] = y.v[2 * j] * cs[4 + j] - y.v[2 * j + 1] * sn[4 + j];
              w.v[2 * j + 1] = y.v[2 * j] * sn[4 + j] + y.v[2 * j + 1] * cs[4 + j];
            }
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              u.v[j] = x.v[j] * cs[j] - y.v[j] * sn[j];
              w.v[j] = x.v[j] * sn[j] + y.v[j] * cs[j];
            }
          }
          const uint4 pu = pack8(u), pw = pack8(w);
          if (dst) {
            *reinterpret_cast<uint4*>(dst + lo) = pu;
            *reinterpret_cast<uint4*>(dst + hi) = pw;
          }
          if (cached) {
            *reinterpret_cast<uint4*>(cached + lo) = pu;
            *reinterpret_cast<uint4*>(cached + hi) = pw;
          }
        } else {
          const unsigned lo = a.pairs ? 2 * c : c, hi = a.pairs ? 2 * c + 1 : c + half;
          const float x = __half2float(src[lo]), y = __half2float(src[hi]);
          const float cs = cosines[t * half + c], sn = sines[t * half + c];
          const __half u = __float2half_rn(x * cs - y * sn), w = __float2half_rn(x * sn + y * cs);
          if (dst) {
            dst[lo] = u;
            dst[hi] = w;
          }
          if (cached) {
            cached[lo] = u;
            cached[hi] = w;
          }
        }
      } else if constexpr (WIDE) {
        const unsigned e = a.R + (c - a.rot) * 8;
        const uint4 x = *reinterpret_cast<const uint4*>(src + e);
        if (dst && dst != src) *reinterpret_cast<uint4*>(dst + e) = x;
        if (cached) *reinterpret_cast<uint4*>(cached + e) = x;
      } else {
        const unsigned e = a.R + (c - a.rot) * 2;
        const uint32_t x = *reinterpret_cast<const uint32_t*>(src + e);
        if (dst && dst != src) *reinterpret_cast<uint32_t*>(dst + e) = x;
        if (cached) *reinterpret_cast<uint32_t*>(cached + e) = x;
      }
    }
  }
}

// ---------------------------------------------------------------- heads of 64, 128 and 256
// L lanes hold a head's row, 16 bytes each, so that every access is a whole row; the row's other half of a pair comes
// from the lane that holds it (neighbours in pairs are in one lane anyway).  A warp takes a token, or a part of its rows
// where tokens are few: kAhead rows of loads on their way before the angles are made, by all lanes together, a pair at a
// time, and kept in registers for all of the token's heads.  Bound by the bytes: 12289 tokens of 24/4 heads of 256, 64 of
// them turned, with the cache's write, 428 MB in 71.8 us, 0.88 of measured HBM; 40001 tokens of 32/8 heads of 128, 819 MB
// in 125 us, 0.97 (the form for any head: 137 and 147).  Four CTAs an SM, 64 registers a thread: halves spill 40 bytes,
// pairs of neighbours none; with five CTAs 88 and 137 us.
constexpr int kRowsThreads = 256, kRowsWarps = kRowsThreads / 32;

template <int L, bool PAIRS>
__global__ void __launch_bounds__(kRowsThreads, 4) rotary_rows_kernel(const RotaryArgs a) {
  constexpr int D = L * 8, kRows = 32 / L, kAhead = 4;
  extern __shared__ __align__(16) float row_angles[];  // of each warp: cosines [R/2], sines [R/2]
  asm volatile("griddepcontrol.wait;" ::: "memory");  // what came before is over (see launch_early)
  if (a.plan->magic != kRotaryMagic || a.plan->R != a.R) {
    if (blockIdx.x == 0 && threadIdx.x == 0) set_status(a.status, TB_DEV_BAD_PLAN);
    return;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = lane % L, half = a.R / 2;
  const float amp = a.plan->amplitude;
  const unsigned long long* turns = reinterpret_cast<const unsigned long long*>(a.plan + 1);
  float *cosines = row_angles + warp * a.R, *sines = cosines + half;
  // the lane's elements: turned or not, and as the first or second of their pairs
  const bool turned = c * 8 < a.R;
  const int hop = half / 8;  // lanes from the first half of the pairs to the second
  const bool second = !PAIRS && turned && c >= hop;
  const int pair = PAIRS ? c * 4 : (second ? c - hop : c) * 8;
  const int other = PAIRS || !turned ? lane : second ? lane - hop : lane + hop;
  const int rows = a.Hq + a.Hk + (a.v_cache ? a.Hk : 0);
  const int64_t head = (int64_t)D << a.page_log2;  // of the cache: elements from one head to the next
  const int64_t units = a.T * a.split;
  for (int64_t u = (int64_t)blockIdx.x * kRowsWarps + warp; u < units; u += (int64_t)gridDim.x * kRowsWarps) {
    const int64_t t = u / a.split;
    const int part = (int)(u - t * a.split);
    const int begin = rows * part / a.split, end = rows * (part + 1) / a.split;
    const __half *q = a.q + t * a.ldq + c * 8, *k = a.k + t * a.ldk + c * 8, *v = a.v + t * a.ldv + c * 8;
    auto load = [&](int row) {
      const __half* p = row < a.Hq ? q + row * D : row < a.Hq + a.Hk ? k + (row - a.Hq) * D : v + (row - a.Hq - a.Hk) * D;
      return row < end ? *reinterpret_cast<const uint4*>(p) : make_uint4(0, 0, 0, 0);
    };
    uint4 x[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) x[i] = load(begin + i * kRows + lane / L);
    int64_t slot = -1;
    if (a.slots) {
      slot = a.slots[t];
      if (slot >= a.n_slots) {
        if (lane == 0) set_status(a.status, TB_DEV_BAD_SLOT);
        slot = -1;
      }
    }
    const int64_t place = slot < 0 ? 0 : (((slot >> a.page_log2) * a.Hk << a.page_log2) + (slot & ((1ll << a.page_log2) - 1))) * D + c * 8;
    const unsigned long long pos = (unsigned long long)(long long)a.pos[t];
    __syncwarp();
    for (int i = lane; i < half; i += 32) {
      float sn, cs;
      sincospif(__ll2float_rn((long long)(pos * turns[i])) * 0x1p-63f, &sn, &cs);
      cosines[i] = amp * cs;
      sines[i] = a.inverse ? -amp * sn : amp * sn;
    }
    __syncwarp();
    float cs[PAIRS ? 4 : 8], sn[PAIRS ? 4 : 8];
    if (turned) {
#pragma unroll
      for (int i = 0; i < (PAIRS ? 4 : 8); i += 4) {
        const float4 p = *reinterpret_cast<const float4*>(cosines + pair + i), r = *reinterpret_cast<const float4*>(sines + pair + i);
        cs[i] = p.x, cs[i + 1] = p.y, cs[i + 2] = p.z, cs[i + 3] = p.w;
        sn[i] = r.x, sn[i + 1] = r.y, sn[i + 2] = r.z, sn[i + 3] = r.w;
      }
      if (second) {  // b cos + a sin, as a cos - b sin with the sine turned round
#pragma unroll
        for (int i = 0; i < (PAIRS ? 4 : 8); ++i) sn[i] = -sn[i];
      }
    }
    for (int row0 = begin; row0 < end; row0 += kAhead * kRows) {
      if (row0 > begin) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) x[i] = load(row0 + i * kRows + lane / L);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int row = row0 + i * kRows + lane / L;
        uint4 y = x[i];
        if (row0 + i * kRows < a.Hq + a.Hk) {  // (all lanes: some of its rows may be v's)
          if constexpr (PAIRS) {
            if (turned) {
              const Eight e = unpack8(x[i]);
              Eight o;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                o.v[2 * j] = e.v[2 * j] * cs[j] - e.v[2 * j + 1] * sn[j];
                o.v[2 * j + 1] = e.v[2 * j] * sn[j] + e.v[2 * j + 1] * cs[j];
              }
              y = pack8(o);
            }
          } else {
            uint4 z;
            z.x = __shfl_sync(0xffffffffu, x[i].x, other);
            z.y = __shfl_sync(0xffffffffu, x[i].y, other);
            z.z = __shfl_sync(0xffffffffu, x[i].z, other);
            z.w = __shfl_sync(0xffffffffu, x[i].w, other);
            if (turned) {
              const Eight e = unpack8(x[i]), f = unpack8(z);
              Eight o;
#pragma unroll
              for (int j = 0; j < 8; ++j) o.v[j] = e.v[j] * cs[j] - f.v[j] * sn[j];
              y = pack8(o);
            }
          }
        }
        if (row < end) {
          if (row < a.Hq) {
            __half* o = a.q_out + t * a.ldqo + row * D + c * 8;
            if (turned || a.q_copy) *reinterpret_cast<uint4*>(o) = y;
          } else if (row < a.Hq + a.Hk) {
            const int h = row - a.Hq;
            if (a.k_out && (turned || a.k_out != a.k)) *reinterpret_cast<uint4*>(a.k_out + t * a.ldko + h * D + c * 8) = y;
            if (slot >= 0) *reinterpret_cast<uint4*>(a.k_cache + place + h * head) = y;
          } else if (slot >= 0) {
            *reinterpret_cast<uint4*>(a.v_cache + place + (row - a.Hq - a.Hk) * head) = x[i];
          }
        }
      }
    }
  }
}

static int launch_rotary(RotaryArgs a, cudaStream_t stream) {
  DeviceFacts f;
  const int rc = device_facts(&f);
  if (rc != TB_OK) return rc;
  const bool wide = a.R % 16 == 0;
  a.rot = wide ? a.R / 16 : a.R / 2;
  const int copy = wide ? (a.D - a.R) / 8 : (a.D - a.R) / 2;
  a.q_copy = a.q_out != a.q ? copy : 0;
  a.k_copy = a.k_cache || (a.k_out && a.k_out != a.k) ? copy : 0;
  a.per_token = a.Hq * (a.rot + a.q_copy) + a.Hk * (a.rot + a.k_copy) + (a.v_cache ? a.Hk * (a.D / 8) : 0);
  if (wide && (a.D == 64 || a.D == 128 || a.D == 256)) {
    const int per = a.D / 8, step = 32 / per, rows = a.Hq + a.Hk + (a.v_cache ? a.Hk : 0), steps = (rows + step - 1) / step;
    // a token's rows are shared out while tokens are few, down to four rows a lane
    const int64_t enough = (int64_t)f.sms * 32;
    int64_t split = (enough + a.T - 1) / a.T;
    if (split > (steps + 3) / 4) split = (steps + 3) / 4;
    a.split = (int)split;
    int64_t ctas = (a.T * split + kRowsWarps - 1) / kRowsWarps;
    if (ctas > (int64_t)f.sms * 16) ctas = (int64_t)f.sms * 16;
    const int smem = kRowsWarps * a.R * 4;
    void (*fn)(const RotaryArgs) = a.pairs ? (per == 8 ? rotary_rows_kernel<8, true> : per == 16 ? rotary_rows_kernel<16, true> : rotary_rows_kernel<32, true>)
                                           : (per == 8 ? rotary_rows_kernel<8, false> : per == 16 ? rotary_rows_kernel<16, false> : rotary_rows_kernel<32, false>);
    return launch_early(fn, dim3((unsigned)ctas), kRowsThreads, smem, stream, a);
  }
  a.tile = kRotaryAngles / (a.R / 2);
  if (a.tile > 8) a.tile = 8;
  const int64_t ctas = (int64_t)f.sms * 8;
  while (a.tile > 1 && (a.T + a.tile - 1) / a.tile < ctas) a.tile /= 2;
  int64_t tiles = (a.T + a.tile - 1) / a.tile;
  // a token's pieces are shared out while tokens are few: a CTA keeps one piece a thread
  const int most = (a.tile * a.per_token + kRotaryThreads - 1) / kRotaryThreads;
  a.split = tiles < f.sms ? (int)((f.sms + tiles - 1) / tiles) : 1;
  if (a.split > most) a.split = most;
  if (tiles > ctas) tiles = ctas;
  const dim3 grid((unsigned)tiles, (unsigned)a.split);
  return launch_early(wide ? rotary_kernel<true> : rotary_kernel<false>, grid, kRotaryThreads, 0, stream, a);
}

// q, k and the plan, as both entry points take them
static int check_rotary(const RotaryArgs& a, int64_t Hq, int64_t Hk, int64_t D, int64_t R, int layout) {
  if (a.T < 0 || a.T > INT_MAX || Hq < 1 || Hq > 1024 || Hk < 0 || Hk > 1024 || D < 8 || D > 1024 || D % 8 || R < 2 || R > D || R % 2) return TB_ERR_SHAPE;
  if (a.ldq < Hq * D || a.ldq % 8 || a.ldqo < Hq * D || a.ldqo % 8) return TB_ERR_SHAPE;
  if (Hk && (a.ldk < Hk * D || a.ldk % 8)) return TB_ERR_SHAPE;
  if (a.k_out && (a.ldko < Hk * D || a.ldko % 8)) return TB_ERR_SHAPE;
  if (layout != TB_ROTARY_HALF && layout != TB_ROTARY_PAIRS) return TB_ERR_UNSUPPORTED;
  return TB_OK;
}

static int check_rotary_pointers(const RotaryArgs& a, int Hk) {
  if (!a.q || !a.q_out || (Hk && !a.k) || !a.pos || !a.plan) return TB_ERR_NULL;
  if (!aligned16(a.q) || !aligned16(a.k) || !aligned16(a.q_out) || !aligned16(a.k_out) || !aligned16(a.plan) || !aligned_to(a.pos, 4))
    return TB_ERR_ALIGN;
  // in place only element for element
  if ((a.q_out == a.q && a.ldqo != a.ldq && a.T > 1) || (a.k_out && a.k_out == a.k && a.ldko != a.ldk && a.T > 1)) return TB_ERR_SHAPE;
  return TB_OK;
}

}  // namespace tb

extern "C" size_t tb_rotary_plan_size(int64_t R) {
  if (R < 2 || R > tb::kRotaryMaxR || R % 2) return 0;
  return (sizeof(tb::RotaryPlan) + (size_t)R / 2 * 8 + 15) / 16 * 16;
}

extern "C" int tb_rotary_plan(void* plan, size_t plan_bytes, int64_t R, double base, int scaling, double factor, double original,
                              double beta_fast, double beta_slow, double amplitude, const double* freqs, int32_t* dev_status,
                              void* stream) {
  using namespace tb;
  const size_t need = tb_rotary_plan_size(R);
  if (!need) return TB_ERR_SHAPE;
  if (scaling != TB_ROTARY_NONE && scaling != TB_ROTARY_LINEAR && scaling != TB_ROTARY_BASE && scaling != TB_ROTARY_PARTS)
    return TB_ERR_UNSUPPORTED;
  if (!plan) return TB_ERR_NULL;
  if (!aligned16(plan) || !aligned_to(freqs, 8)) return TB_ERR_ALIGN;
  if (plan_bytes < need) return TB_ERR_WORKSPACE;
  if (!(amplitude >= 0.0) || !isfinite((float)amplitude)) return TB_ERR_VALUE;
  if (freqs) {
    if (scaling != TB_ROTARY_NONE) return TB_ERR_VALUE;
  } else {
    if (!(base > 1.0) || !isfinite(base)) return TB_ERR_VALUE;
    if (scaling != TB_ROTARY_NONE && (!(factor > 0.0) || !isfinite(factor))) return TB_ERR_VALUE;
    if (scaling == TB_ROTARY_BASE && R == 2) return TB_ERR_VALUE;
    if (scaling == TB_ROTARY_PARTS &&
        (!(original > 0.0) || !isfinite(original) || !(beta_slow > 0.0) || !(beta_fast > beta_slow) || !isfinite(beta_fast)))
      return TB_ERR_VALUE;
  }
  RotaryPlanArgs a;
  a.base = base;
  a.factor = factor;
  a.original = original;
  a.beta_fast = beta_fast;
  a.beta_slow = beta_slow;
  a.amplitude = amplitude;
  a.freqs = freqs;
  a.scaling = scaling;
  a.R = (int)R;
  rotary_plan_kernel<<<1, (unsigned)((R / 2 + 31) / 32 * 32), 0, static_cast<cudaStream_t>(stream)>>>(a, static_cast<RotaryPlan*>(plan), dev_status);
  return check_launch();
}

extern "C" int tb_rotary(const uint16_t* q, int64_t ldq, int64_t Hq, const uint16_t* k, int64_t ldk, int64_t Hk, int64_t T, int64_t D,
                         const int32_t* pos, const void* plan, int64_t R, int layout, int inverse, uint16_t* q_out, int64_t ldqo,
                         uint16_t* k_out, int64_t ldko, int32_t* dev_status, void* stream) {
  using namespace tb;
  RotaryArgs a = {};
  a.q = reinterpret_cast<const __half*>(q);
  a.k = reinterpret_cast<const __half*>(k);
  a.q_out = reinterpret_cast<__half*>(q_out);
  a.k_out = reinterpret_cast<__half*>(k_out);
  a.ldq = ldq;
  a.ldk = ldk;
  a.ldqo = ldqo;
  a.ldko = ldko;
  a.T = T;
  a.pos = pos;
  a.plan = static_cast<const RotaryPlan*>(plan);
  a.status = dev_status;
  int rc = check_rotary(a, Hq, Hk, D, R, layout);
  if (rc != TB_OK) return rc;
  if (T == 0) return TB_OK;
  rc = check_rotary_pointers(a, (int)Hk);
  if (rc != TB_OK) return rc;
  if (Hk && !k_out) return TB_ERR_NULL;
  a.Hq = (int)Hq;
  a.Hk = (int)Hk;
  a.D = (int)D;
  a.R = (int)R;
  a.pairs = layout == TB_ROTARY_PAIRS;
  a.inverse = inverse != 0;
  return launch_rotary(a, static_cast<cudaStream_t>(stream));
}

extern "C" int tb_rotary_cache_write(const uint16_t* q, int64_t ldq, int64_t Hq, const uint16_t* k, int64_t ldk, const uint16_t* v,
                                     int64_t ldv, int64_t Hkv, int64_t T, int64_t D, const int32_t* pos, const int64_t* slots,
                                     const void* plan, int64_t R, int layout, int inverse, uint16_t* q_out, int64_t ldqo,
                                     uint16_t* k_out, int64_t ldko, uint16_t* k_cache, uint16_t* v_cache, int64_t pages, int64_t page,
                                     int32_t* dev_status, void* stream) {
  using namespace tb;
  RotaryArgs a = {};
  a.q = reinterpret_cast<const __half*>(q);
  a.k = reinterpret_cast<const __half*>(k);
  a.v = reinterpret_cast<const __half*>(v);
  a.q_out = reinterpret_cast<__half*>(q_out);
  a.k_out = reinterpret_cast<__half*>(k_out);
  a.k_cache = reinterpret_cast<__half*>(k_cache);
  a.v_cache = reinterpret_cast<__half*>(v_cache);
  a.ldq = ldq;
  a.ldk = ldk;
  a.ldv = ldv;
  a.ldqo = ldqo;
  a.ldko = ldko;
  a.T = T;
  a.pos = pos;
  a.slots = slots;
  a.plan = static_cast<const RotaryPlan*>(plan);
  a.status = dev_status;
  int rc = check_rotary(a, Hq, Hkv, D, R, layout);
  if (rc != TB_OK) return rc;
  if (Hkv < 1 || ldv < Hkv * D || ldv % 8 || pages < 1 || pages > INT_MAX) return TB_ERR_SHAPE;
  if (!supported_page(page)) return TB_ERR_UNSUPPORTED;
  if (T == 0) return TB_OK;
  rc = check_rotary_pointers(a, (int)Hkv);
  if (rc != TB_OK) return rc;
  if (!v || !slots || !k_cache || !v_cache) return TB_ERR_NULL;
  if (!aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned_to(slots, 8)) return TB_ERR_ALIGN;
  a.n_slots = pages * page;
  a.page_log2 = log2_of(page);
  a.Hq = (int)Hq;
  a.Hk = (int)Hkv;
  a.D = (int)D;
  a.R = (int)R;
  a.pairs = layout == TB_ROTARY_PAIRS;
  a.inverse = inverse != 0;
  return launch_rotary(a, static_cast<cudaStream_t>(stream));
}
