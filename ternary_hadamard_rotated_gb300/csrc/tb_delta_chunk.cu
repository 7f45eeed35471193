// The gated delta rule over prompts, in chunks of 64 tokens (csrc/tb_delta.cu has the recurrent form
// and the entry point).
//
// Inside a chunk, with gamma_i the decays' running sum, D_ij = exp(gamma_i - gamma_j) for j <= i, S the
// state before the chunk, and q, k already divided by their norms:
//   A_ij = beta_i (k_i . k_j) D_ij  (j < i),     T = (I + A)^-1 diag(beta)
//   R_i  = v_i - exp(gamma_i) S^T k_i,           U = T R
//   o_i  = scale (exp(gamma_i) S^T q_i + sum_{j <= i} (q_i . k_j) D_ij u_j)
//   S   <- exp(gamma_C) S + sum_j exp(gamma_C - gamma_j) k_j u_j^T
// T does not depend on the state, so one kernel computes it for all chunks at once, and with it
// P T, P_ij = scale (q_i . k_j) D_ij: the second kernel then gets U and the chunk's own part of o from
// one product [T; P T] R.
//
// Kernel 1, a CTA per (chunk, key head), which its value heads share: K K^T and Q K^T by mma.sync (fp16
// inputs, exact products), per value head the triangular system by substitution in fp32 (a thread
// per column, the column in registers), P T by mma.sync.  It writes T (fp16, high and low part) and
// P T (fp16) as the shared-memory image that kernel 2's MMAs read, and each token's factors.
//
// Kernel 2 walks the chunks, a warp per 16 columns of v, which no other warp's columns depend on: S^T
// stays in the warp's registers as fp32 accumulators of mma.sync, and every product's left factor (S^T,
// R^T, (w U)^T, 16 rows) comes out of the product before it in the layout that the next one wants, so
// a chunk has no exchange between warps at all.  K, Q, V and kernel 1's results come by TMA, three
// chunks deep.  An fp32 factor goes in as two fp16 terms, x 2^e = hi + lo with the warp's largest |x|
// at 2^14: 22 bits, and K and Q are fp16 already.  T has two terms too; what goes into o alone has one.
// About 400 MMAs a warp and chunk, at one per 7.8 clocks and SM sub-partition 1.6 us: what bounds it.
// (The same walk on tcgen05, 32 columns a CTA, took 2.7 us a chunk alone on its SM and 3.4 with a
// second CTA: 20 MMAs of 44 to 60 clocks, and three trips through registers, shared memory and a
// barrier of 800 to 1000 each.)
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>

#include "tb_attention.cuh"
#include "tb_attn_tc.cuh"
#include "tb_common.cuh"
#include "tb_delta.cuh"
#include "tb_host.h"

namespace tb {

constexpr int kDcTok = 64;    // tokens per chunk
constexpr int kDcBlock = kDcTok * 128;  // bytes of a 64 x 64 fp16 image
// a (chunk, value head) in the workspace: T, P T, T's low part, factors
constexpr int kDcItem = 3 * kDcBlock + 1024;
constexpr int kDcFactors = 3 * kDcBlock;  // floats: c [64], w [64], q [64], exp(gamma_C)

struct ChunkArgs {
  DeltaArgs a;
  uint8_t* ws;  // [chunks][Hv] items
};

// ---- which request a chunk belongs to; every warp adds up all requests' chunks itself
struct ChunkScan {
  int64_t upto, own;
  int per;
};
TB_DEVI int64_t chunks_of(const DeltaArgs& a, int b) {
  int64_t t0, n;
  return delta_rows(a, b, t0, n) ? (n + kDcTok - 1) / kDcTok : 0;
}
TB_DEVI ChunkScan chunk_scan(const DeltaArgs& a, int lane) {
  ChunkScan s;
  s.per = (a.B + 31) / 32;
  s.own = 0;
  for (int i = lane * s.per; i < (lane + 1) * s.per && i < a.B; ++i) s.own += chunks_of(a, i);
  s.upto = s.own;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, s.upto, d);
    if (lane >= d) s.upto += x;
  }
  return s;
}

// (volatile keeps them in order with barriers and waits, which are volatile too and clobber memory)
TB_DEVI void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
TB_DEVI void ldsm4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
TB_DEVI void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// ---------------------------------------------------------------- kernel 1
constexpr int kD1Threads = 256;
constexpr int kD1Pitch = 136;   // halves per row of K and Q in shared memory
constexpr int kD1Dots = 65;     // floats per row of K K^T and Q K^T
constexpr int kD1At = 68;       // floats per row of A^T
constexpr int kD1Region = 64 * kD1At * 4;  // 17408 bytes: K, or Q, or one head's A^T, or its T
constexpr int kD1Smem = 4 * kD1Region + 2 * 64 * kD1Dots * 4;

__global__ void __launch_bounds__(kD1Threads, 2) delta_prep_kernel(const ChunkArgs p) {
  const DeltaArgs& a = p.a;
  extern __shared__ __align__(16) uint8_t d1_smem[];
  __shared__ float rk[64], rq[64];
  __shared__ float2 gam[4][64];  // running sums of the decays, high and low part
  __shared__ float bet[4][64];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int hk = (int)(blockIdx.x % a.Hk);
  const int64_t chunk = blockIdx.x / a.Hk;
  const ChunkScan sc = chunk_scan(a, lane);
  const unsigned who = __ballot_sync(0xffffffffu, chunk < sc.upto);
  if (!who) return;  // past the last chunk
  int b = 0;
  int64_t before = sc.upto - sc.own;
  const int src = __ffs(who) - 1;
  if (lane == src) {
    for (b = lane * sc.per;; ++b) {
      const int64_t n = chunks_of(a, b);
      if (chunk < before + n) break;
      before += n;
    }
  }
  b = __shfl_sync(0xffffffffu, b, src);
  before = __shfl_sync(0xffffffffu, before, src);
  int64_t t0, len;
  delta_rows(a, b, t0, len);
  const int64_t c = chunk - before;
  t0 += c * kDcTok;
  const int n = (int)(len - c * kDcTok < kDcTok ? len - c * kDcTok : kDcTok);

  // K and Q: four threads a row, 32 elements each; rows past the request's end are zeros
  __half* Ks = reinterpret_cast<__half*>(d1_smem);
  __half* Qs = reinterpret_cast<__half*>(d1_smem + kD1Region);
  {
    const int row = tid >> 2, part = (tid & 3) * 32;
    float sk = 0.f, sq = 0.f;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const __half* g = (m ? a.q + (t0 + row) * a.ldq : a.k + (t0 + row) * a.ldk) + hk * kDeltaD + part;
      __half* d = (m ? Qs : Ks) + row * kD1Pitch + part;
      float& s = m ? sq : sk;
#pragma unroll
      for (int e = 0; e < 32; e += 8) {
        uint4 w = make_uint4(0, 0, 0, 0);
        if (row < n) w = __ldg(reinterpret_cast<const uint4*>(g + e));
        *reinterpret_cast<uint4*>(d + e) = w;
        const __half2* h = reinterpret_cast<const __half2*>(&w);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float2 f = __half22float2(h[x]);
          s = fmaf(f.x, f.x, fmaf(f.y, f.y, s));
        }
      }
    }
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
      sk += __shfl_xor_sync(0xffffffffu, sk, d);
      sq += __shfl_xor_sync(0xffffffffu, sq, d);
    }
    if ((tid & 3) == 0) {
      rk[row] = a.normalise ? 1.f / sqrtf(sk + kDeltaEps) : 1.f;
      rq[row] = (a.normalise ? 1.f / sqrtf(sq + kDeltaEps) : 1.f) * a.scale;
    }
  }
  __syncthreads();

  // K K^T (warps 0-3) and Q K^T (4-7), 16 rows a warp, the lower triangle's tiles
  float* dots = reinterpret_cast<float*>(d1_smem + 4 * kD1Region);
  float* qdots = dots + 64 * kD1Dots;
  {
    const int r0 = (warp & 3) * 16;
    const __half* A = warp < 4 ? Ks : Qs;
    float acc[8][4];
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
    for (int k = 0; k < kDeltaD; k += 16) {
      uint32_t af[4];
      ldsm4(smem_u32(A + (r0 + (lane & 15)) * kD1Pitch + k + (lane >> 4) * 8), af);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j * 16 > r0) break;
        uint32_t bf[4];  // keys j*16 + 0..7 (k, k+8), then 8..15
        ldsm4(smem_u32(Ks + (j * 16 + (lane & 7) + (lane >> 4) * 8) * kD1Pitch + k + ((lane >> 3) & 1) * 8), bf);
        mma_16816(acc[2 * j], af, bf[0], bf[1]);
        mma_16816(acc[2 * j + 1], af, bf[2], bf[3]);
      }
    }
    float* out = warp < 4 ? dots : qdots;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j * 8 > r0 + 15) break;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        out[(r0 + (lane >> 2) + (e >> 1) * 8) * kD1Dots + j * 8 + (lane & 3) * 2 + (e & 1)] = acc[j][e];
    }
  }
  __syncthreads();

  // the value heads of this key head, four at a time, a pair of warps each
  const int group = a.Hv / a.Hk, pair = warp >> 1, l64 = tid & 63;
  float* At = reinterpret_cast<float*>(d1_smem + pair * kD1Region);
  auto sync_pair = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(pair + 1) : "memory"); };
  for (int h0 = 0; h0 < group; h0 += 4) {
    if (h0 + pair >= group) continue;
    const int h = hk * group + h0 + pair;
    if ((warp & 1) == 0) {  // the decays' sums in double: differences of large sums stay exact enough
      double x[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = lane * 2 + e;
        float g = i < n ? __ldg(a.g + (t0 + i) * a.Hv + h) : 0.f;
        if (g < -200.f) g = -200.f;  // e^-200 is 0 in fp32 already
        x[e] = g;
        bet[pair][i] = i < n ? __ldg(a.beta + (t0 + i) * a.Hv + h) : 0.f;
      }
      double s = x[0] + x[1];
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, s, d);
        if (lane >= d) s += y;
      }
      const double s0 = s - x[1];
      gam[pair][lane * 2] = make_float2((float)s0, (float)(s0 - (double)(float)s0));
      gam[pair][lane * 2 + 1] = make_float2((float)s, (float)(s - (double)(float)s));
    }
    sync_pair();
    uint8_t* item = p.ws + (chunk * a.Hv + h) * (int64_t)kDcItem;
    const float2 mine = gam[pair][l64], last = gam[pair][63];
    {
      float* f = reinterpret_cast<float*>(item + kDcFactors);
      const float eg = expf(mine.x) * (1.f + mine.y);
      f[l64] = eg * rk[l64];
      f[64 + l64] = expf((last.x - mine.x) + (last.y - mine.y)) * rk[l64];
      f[128 + l64] = eg * rq[l64];
      if (l64 == 0) f[192] = expf(last.x) * (1.f + last.y);
    }
    // A^T: thread = row i of A
    {
      const float bi = bet[pair][l64] * rk[l64];
      for (int k = 0; k < 63; ++k) {
        const float2 gk = gam[pair][k];
        const float d = expf((mine.x - gk.x) + (mine.y - gk.y));
        At[k * kD1At + l64] = l64 > k ? bi * rk[k] * dots[l64 * kD1Dots + k] * d : 0.f;
      }
    }
    sync_pair();
    // column l64 of (I + A)^-1 by substitution; the upper half's warp starts at its first column
    float x[64];
#pragma unroll
    for (int i = 0; i < 64; ++i) x[i] = i == l64 ? 1.f : 0.f;
    if ((warp & 1) == 0) {
#pragma unroll
      for (int k = 0; k < 32; ++k) {
#pragma unroll
        for (int i4 = (k + 1) / 4; i4 < 16; ++i4) {
          const float4 w = *reinterpret_cast<const float4*>(At + k * kD1At + i4 * 4);
          if (i4 * 4 > k) x[i4 * 4] = fmaf(-w.x, x[k], x[i4 * 4]);
          if (i4 * 4 + 1 > k) x[i4 * 4 + 1] = fmaf(-w.y, x[k], x[i4 * 4 + 1]);
          if (i4 * 4 + 2 > k) x[i4 * 4 + 2] = fmaf(-w.z, x[k], x[i4 * 4 + 2]);
          x[i4 * 4 + 3] = fmaf(-w.w, x[k], x[i4 * 4 + 3]);
        }
      }
    }
#pragma unroll
    for (int k = 32; k < 63; ++k) {
#pragma unroll
      for (int i4 = (k + 1) / 4; i4 < 16; ++i4) {
        const float4 w = *reinterpret_cast<const float4*>(At + k * kD1At + i4 * 4);
        if (i4 * 4 > k) x[i4 * 4] = fmaf(-w.x, x[k], x[i4 * 4]);
        if (i4 * 4 + 1 > k) x[i4 * 4 + 1] = fmaf(-w.y, x[k], x[i4 * 4 + 1]);
        if (i4 * 4 + 2 > k) x[i4 * 4 + 2] = fmaf(-w.z, x[k], x[i4 * 4 + 2]);
        x[i4 * 4 + 3] = fmaf(-w.w, x[k], x[i4 * 4 + 3]);
      }
    }
    sync_pair();  // A^T has been read: its room takes T's image (high part, then low)
    uint8_t* img = d1_smem + pair * kD1Region;
    {
      const float bj = bet[pair][l64];
#pragma unroll
      for (int i = 0; i < 64; ++i) {
        const float v = x[i] * bj;
        const __half hi = __float2half_rn(v);
        const int at = i * 128 + (((l64 >> 3) ^ (i & 7)) << 4) + (l64 & 7) * 2;
        *reinterpret_cast<__half*>(img + at) = hi;
        *reinterpret_cast<__half*>(img + kDcBlock + at) = __float2half_rn(v - __half2float(hi));
      }
    }
    sync_pair();
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int o = (e * 64 + l64) * 16;
      *reinterpret_cast<uint4*>(item + o) = *reinterpret_cast<const uint4*>(img + o);
      *reinterpret_cast<uint4*>(item + 2 * kDcBlock + o) = *reinterpret_cast<const uint4*>(img + kDcBlock + o);
    }
    // P T: 32 rows a warp, P made from Q K^T as the A fragments
#pragma unroll 1
    for (int m = 0; m < 2; ++m) {
      const int r0 = (warp & 1) * 16 + m * 32;  // the pair's warps share the longer rows
      float acc[8][4];
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
      const int i0 = r0 + (lane >> 2);
      const float2 g0 = gam[pair][i0], g1 = gam[pair][i0 + 8];
      const float f0 = rq[i0], f1 = rq[i0 + 8];
      for (int k = 0; k <= r0; k += 16) {
        uint32_t af[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {  // rows i0, i0 + 8; columns k + 2 (lane % 4) (+ 8)
          const int i = i0 + (q & 1) * 8, j = k + (lane & 3) * 2 + (q >> 1) * 8;
          const float2 gi = (q & 1) ? g1 : g0;
          float v[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float2 gj = gam[pair][j + e];
            v[e] = j + e <= i ? qdots[i * kD1Dots + j + e] * ((q & 1) ? f1 : f0) * rk[j + e] *
                                    expf((gi.x - gj.x) + (gi.y - gj.y))
                              : 0.f;
          }
          af[q] = pack_half2(v[0], v[1]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int kr = k + (lane & 15), ch = j * 2 + (lane >> 4);
          uint32_t bf[4];  // columns j*16 + 0..7 (k, k+8), then 8..15
          ldsm4_trans(smem_u32(img + kr * 128 + ((ch ^ (kr & 7)) << 4)), bf);
          mma_16816(acc[2 * j], af, bf[0], bf[1]);
          mma_16816(acc[2 * j + 1], af, bf[2], bf[3]);
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int i = i0 + e * 8;
          *reinterpret_cast<uint32_t*>(item + kDcBlock + i * 128 + ((j ^ (i & 7)) << 4) + (lane & 3) * 4) =
              pack_half2(acc[j][2 * e], acc[j][2 * e + 1]);
        }
    }
    sync_pair();  // the image has been read before the next head's A^T takes its place
  }
}

// ---------------------------------------------------------------- kernel 2
constexpr int kD2Stages = 3;
constexpr int kD2Q = 2 * kDcBlock, kD2Item = 4 * kDcBlock, kD2V = kD2Item + 26624;  // places in a stage

template <int W>
struct ScanCfg {
  // a warp of its own for the loads, unless that makes a third warp in an SM sub-partition, whose
  // registers two warps of 255 fill
  static constexpr bool kLoader = W == 4;
  static constexpr int kThreads = (W + kLoader) * 32;
  static constexpr int kStage = kD2V + W / 4 * kDcBlock;
  static constexpr int kBytes = 4 * kDcBlock + kDcItem + W / 4 * kDcBlock;  // loaded per chunk
  static constexpr int kSmem = 1024 + kD2Stages * kStage + 128;
};

// a power of two that takes magnitudes up to `bits` (an fp32's) to 2^14, and its inverse
TB_DEVI float operand_scale(uint32_t bits, float& inverse) {
  int e = 268 - (int)(bits >> 23);
  e = e < 127 - 100 ? 127 - 100 : (e > 127 + 100 ? 127 + 100 : e);
  inverse = __int_as_float((254 - e) << 23);
  return __int_as_float(e << 23);
}
TB_DEVI uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }  // orders as the values do, NaN last
// x, y -> fp16 pair and the fp16 pair of what it leaves
TB_DEVI void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x, y);
  const float2 f = __half22float2(h);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = pack_half2(x - f.x, y - f.y);
}
TB_DEVI uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// Arrival that hands a place back after reads whose values have been used: nothing to release (a release
// waits for the warp's global stores too, 400 clocks a chunk).
TB_DEVI void mbar_arrive_reads(uint64_t* bar) {
  asm volatile("mbarrier.arrive.relaxed.cta.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// W warps per CTA, 16 columns of v each.
template <int W>
__global__ void __launch_bounds__(ScanCfg<W>::kThreads, 1)
    delta_scan_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmQ,
                      const __grid_constant__ CUtensorMap tmV, const ChunkArgs p) {
  using C = ScanCfg<W>;
  const DeltaArgs& a = p.a;
  extern __shared__ uint8_t d2_raw[];
  const uint32_t raw = smem_u32(d2_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = d2_raw + (base - raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kD2Stages * C::kStage);
  uint64_t* empty = full + kD2Stages;
  volatile int* aborted = reinterpret_cast<volatile int*>(full + 2 * kD2Stages);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kSlices = 8 / W;
  const int slice = (int)(blockIdx.x % kSlices);
  const int64_t bh = blockIdx.x / kSlices;
  const int h = (int)(bh % a.Hv), b = (int)(bh / a.Hv), hk = h / (a.Hv / a.Hk);
  if (tid == 0) {
    *aborted = 0;
    for (int i = 0; i < kD2Stages; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, W);
    }
    fence_barrier_init();
  }
  int64_t t0, len;
  if (!delta_rows(a, b, t0, len)) {
    if (tid == 0 && h == 0 && slice == 0) set_status(a.status, TB_DEV_BAD_LEN);
    len = 0;
  }
  const int nc = (int)((len + kDcTok - 1) / kDcTok);
  __syncthreads();
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity) || *aborted) return;
    if (!mbar_wait(bar, parity)) {
      *aborted = 1;
      set_status(a.status, TB_DEV_TIMEOUT);
    }
  };

  int64_t first = 0;  // the request's first chunk
  constexpr int kLoads = C::kLoader ? W : 0;  // the warp that loads
  if (warp == kLoads) {
    const ChunkScan sc = chunk_scan(a, lane);
    first = sc.upto - sc.own;
    const int src = b / sc.per;
    if (lane == src)
      for (int i = lane * sc.per; i < b; ++i) first += chunks_of(a, i);
    first = __shfl_sync(0xffffffffu, first, src);
  }
  // a lane per copy
  constexpr int kCopies = 5 + W / 4;
  auto load = [&](int c) {
    const int s = c % kD2Stages, row = (int)t0 + c * kDcTok;
    const uint32_t sa = base + s * C::kStage, bar = smem_u32(full + s);
    if (c >= kD2Stages) wait(empty + s, (c / kD2Stages - 1) & 1);
    if (lane == 0) {
      mbar_arrive_expect_tx(full + s, C::kBytes);
      if (c == 0) asm volatile("griddepcontrol.wait;" ::: "memory");  // kernel 1's results
      bulk_g2s(smem + s * C::kStage + kD2Item, p.ws + ((first + c) * a.Hv + h) * (int64_t)kDcItem, kDcItem, full + s);
    } else if (lane < kCopies) {
      const int d = (lane - 1) & 1;
      const bool v = lane >= 5;
      const CUtensorMap* tm = v ? &tmV : (lane >= 3 ? &tmQ : &tmK);
      const uint32_t dst = sa + (v ? kD2V : (lane >= 3 ? kD2Q : 0)) + d * kDcBlock;
      tma_load_3d<1>(dst, tm, v ? (slice * (W / 4) + d) * 64 : d * 64, v ? h : hk, row, bar);
    }
    __syncwarp();
  };
  if (warp == kLoads)
    for (int c = 0; c < (C::kLoader ? nc : kD2Stages - 1) && c < nc; ++c) load(c);

  auto linger = [&]() {  // a wait gave up: leave the copies in flight time to land before the CTA ends
    const uint64_t t = globaltimer_ns();
    while (*aborted && globaltimer_ns() - t < 1000000) {
    }
  };
  if (C::kLoader && warp == W) {
    linger();
    return;
  }

  const int g = lane >> 2, t2 = (lane & 3) * 2;
  const int64_t si = delta_slot(a.slot_in, b, a.n_in, a.status), so = delta_slot(a.slot_out, b, a.n_out, a.status);
  const int64_t head_size = (int64_t)a.Hv * kDeltaD * kDeltaD;
  const int col = slice * W * 16 + warp * 16;  // the warp's first column of v
  // S^T: rows g, g + 8 (columns of v), columns 8 j + t2, + 1 (of k)
  float S[16][4];
  {
    const bool have = a.state_in && si >= 0;
    const float* src = a.state_in + si * head_size + ((int64_t)h * kDeltaD + t2) * kDeltaD + col + g;
#pragma unroll
    for (int j = 0; j < 16; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        S[j][e] = have ? __ldg(src + (j * 8 + (e & 1)) * kDeltaD + (e >> 1) * 8) : 0.f;
  }
  uint32_t sbig[4] = {0, 0, 0, 0};  // the largest |S|, four chains of it
#pragma unroll
  for (int j = 0; j < 16; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) sbig[e] = max(sbig[e], magnitude(S[j][e]));
  // addresses of the ldmatrix lanes inside a 64 x 64 image: rows by the lane, a 16-byte piece per k
  const uint32_t sw = (uint32_t)lane & 7u;
  const uint32_t row_n = (((uint32_t)lane & 7u) + ((uint32_t)lane >> 4) * 8u) * 128u;  // rows are n
  const uint32_t row_k = ((uint32_t)lane & 15u) * 128u;                                // rows are k
  const uint32_t pc_n = ((uint32_t)lane >> 3) & 1u, pc_k = (uint32_t)lane >> 4;
  const uint32_t v_row = ((((uint32_t)lane >> 4) & 1u) * 8u + sw) * 128u;
  const uint32_t v_pc = (((uint32_t)(warp & 3) * 2u + pc_n) ^ sw) << 4;

  for (int c = 0; c < nc; ++c) {
    const int s = c % kD2Stages;
    const uint32_t K = base + s * C::kStage, Q = K + kD2Q, X = K + kD2Item, V = K + kD2V + (warp >> 2) * kDcBlock;
    const float* f = reinterpret_cast<const float*>(smem + s * C::kStage + kD2Item + kDcFactors);
    const int n = (int)(len - (int64_t)c * kDcTok < kDcTok ? len - (int64_t)c * kDcTok : kDcTok);
    float down_s;
    const float up_s = operand_scale(__reduce_max_sync(0xffffffffu, max(max(sbig[0], sbig[1]), max(sbig[2], sbig[3]))), down_s);
    wait(full + s, (c / kD2Stages) & 1);
    if (n < kDcTok) {  // the last chunk: rows of K that are another request's, out of the sum over the tokens
      for (int i = tid; i < (kDcTok - n) * 16; i += W * 32) {
        const int r = n + (i >> 4), x = i & 15;
        asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(K + (x >> 3) * kDcBlock + r * 128 + (x & 7) * 16), "r"(0)
                     : "memory");
      }
      asm volatile("bar.sync 1, %0;" ::"n"(W * 32) : "memory");
    }
    // A warp has its SM sub-partition to itself, so nothing but its own other work fills the latency of a
    // load or the time of an MMA: loads run a step ahead, and what is not on the way from S to the next
    // S (the products for o, its output) is spread over the steps that are.
    float R[8][4], O[8][4];
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) R[j][e] = O[j][e] = 0.f;
    auto at_n = [&](int ks) { return (ks >> 2) * kDcBlock + row_n + (((uint32_t)(ks & 3) * 2u + pc_n) ^ sw) * 16u; };
    uint32_t bk[4][4], sh[8][4];
    // S^T k
#pragma unroll
    for (int j = 0; j < 4; ++j) ldsm4(K + at_n(0) + j * 2048, bk[j]);
    uint32_t lo[2][4];
    auto split_s = [&](int ks, int q) {
      const float* x = S[2 * ks + (q >> 1)] + (q & 1) * 2;
      split2(x[0] * up_s, x[1] * up_s, sh[ks][q], lo[ks & 1][q]);
    };
#pragma unroll
    for (int q = 0; q < 4; ++q) split_s(0, q);
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        mma_16816(R[2 * j], sh[ks], bk[j][0], bk[j][1]);
        if (ks < 7) split_s(ks + 1, j);
        mma_16816(R[2 * j + 1], sh[ks], bk[j][2], bk[j][3]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        mma_16816(R[2 * j], lo[ks & 1], bk[j][0], bk[j][1]);
        mma_16816(R[2 * j + 1], lo[ks & 1], bk[j][2], bk[j][3]);
        ldsm4((ks < 7 ? K + at_n(ks + 1) : Q + at_n(0)) + j * 2048, bk[j]);
      }
    }
    if (!C::kLoader && warp == 0 && c + kD2Stages - 1 < nc) load(c + kD2Stages - 1);  // the other warps left that stage a chunk ago
    // S^T q, and beside it R = v - exp(gamma) S^T k
    uint32_t big[4] = {0, 0, 0, 0}, vv[4];
    ldsm4_trans(V + v_row + v_pc, vv);
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      const int tok = ks * 8 + t2;
      const float2 cc = *reinterpret_cast<const float2*>(f + tok);
      auto residual = [&](int q) {  // columns of v g + 8 q
        const float2 w = __half22float2(*reinterpret_cast<const __half2*>(&vv[(ks & 1) * 2 + q]));
        float &x = R[ks][q * 2], &y = R[ks][q * 2 + 1];
        x = tok < n ? fmaf(-cc.x * down_s, x, w.x) : 0.f;
        y = tok + 1 < n ? fmaf(-cc.y * down_s, y, w.y) : 0.f;
        big[q * 2] = max(big[q * 2], magnitude(x));
        big[q * 2 + 1] = max(big[q * 2 + 1], magnitude(y));
      };
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        mma_16816(O[2 * j], sh[ks], bk[j][0], bk[j][1]);
        if (j == 1) residual(0);
        if (j == 2) residual(1);
        mma_16816(O[2 * j + 1], sh[ks], bk[j][2], bk[j][3]);
        if (ks < 7) ldsm4(Q + at_n(ks + 1) + j * 2048, bk[j]);
      }
      if ((ks & 1) && ks < 7) ldsm4_trans(V + (ks / 2 + 1) * 2048 + v_row + v_pc, vv);
    }
    float down_r;
    const float up_r = operand_scale(__reduce_max_sync(0xffffffffu, max(max(big[0], big[1]), max(big[2], big[3]))), down_r);
    uint32_t rh[4][4], rl[4][4];
    auto split_r = [&](int ks, int q) {
      const float* x = R[2 * ks + (q >> 1)] + (q & 1) * 2;
      split2(x[0] * up_r, x[1] * up_r, rh[ks][q], rl[ks][q]);
    };
#pragma unroll
    for (int q = 0; q < 4; ++q) split_r(0, q);
    // U = T R (rows past a token do not reach it: their tiles are left out); o's first part to R's scale
    float U[8][4];
#pragma unroll
    for (int nt = 0; nt < 8; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) U[nt][e] = 0.f;
    auto at_x = [&](int ks, int j) { return X + row_n + (((uint32_t)ks * 2u + pc_n) ^ sw) * 16u + j * 2048; };
    constexpr int kAt[11][2] = {{0, 0}, {0, 1}, {0, 2}, {0, 3}, {1, 1}, {1, 2}, {1, 3}, {2, 2}, {2, 3}, {3, 3}, {3, 3}};
    uint32_t th[2][4], tl[2][4];
    ldsm4(at_x(0, 0), th[0]);
    ldsm4(at_x(0, 0) + 2 * kDcBlock, tl[0]);
#pragma unroll
    for (int i = 0; i < 10; ++i) {
      const int ks = kAt[i][0], j = kAt[i][1], x = i & 1;
      const uint32_t at = at_x(kAt[i + 1][0], kAt[i + 1][1]);
      if (i < 9) {
        ldsm4(at, th[x ^ 1]);
        ldsm4(at + 2 * kDcBlock, tl[x ^ 1]);
      } else {
        ldsm4(at_x(0, 0) + kDcBlock, th[x ^ 1]);  // P T's first
      }
      mma_16816(U[2 * j], rh[ks], th[x][0], th[x][1]);
      mma_16816(U[2 * j + 1], rh[ks], th[x][2], th[x][3]);
      // R's later terms, a step or more ahead of their first use
      if (i < 4) split_r(1, i);
      if (i >= 4 && i < 6) {
        split_r(2, (i - 4) * 2);
        split_r(2, (i - 4) * 2 + 1);
      }
      if (i >= 6 && i < 8) {
        split_r(3, (i - 6) * 2);
        split_r(3, (i - 6) * 2 + 1);
      }
      if (i < 8) {
        const float2 qq = *reinterpret_cast<const float2*>(f + 128 + i * 8 + t2);
        const float qx = qq.x * down_s * up_r, qy = qq.y * down_s * up_r;
        O[i][0] *= qx;
        O[i][1] *= qy;
        O[i][2] *= qx;
        O[i][3] *= qy;
      }
      mma_16816(U[2 * j], rl[ks], th[x][0], th[x][1]);
      mma_16816(U[2 * j + 1], rl[ks], th[x][2], th[x][3]);
      mma_16816(U[2 * j], rh[ks], tl[x][0], tl[x][1]);
      mma_16816(U[2 * j + 1], rh[ks], tl[x][2], tl[x][3]);
    }
    // w U, and beside it o += P T R
    big[0] = big[1] = big[2] = big[3] = 0;
#pragma unroll
    for (int i = 0; i < 10; ++i) {
      const int ks = kAt[i][0], j = kAt[i][1], x = i & 1;
      if (i < 9) ldsm4(at_x(kAt[i + 1][0], kAt[i + 1][1]) + kDcBlock, th[x ^ 1]);
      mma_16816(O[2 * j], rh[ks], th[x][0], th[x][1]);
      mma_16816(O[2 * j + 1], rh[ks], th[x][2], th[x][3]);
      if (i < 8) {
        const float2 ww = *reinterpret_cast<const float2*>(f + 64 + i * 8 + t2);
        const float wx = ww.x * down_r, wy = ww.y * down_r;
        U[i][0] *= wx;
        U[i][1] *= wy;
        U[i][2] *= wx;
        U[i][3] *= wy;
#pragma unroll
        for (int e = 0; e < 4; ++e) big[e] = max(big[e], magnitude(U[i][e]));
      }
    }
    float down_u;
    const float up_u = operand_scale(__reduce_max_sync(0xffffffffu, max(max(big[0], big[1]), max(big[2], big[3]))), down_u);
    auto split_u = [&](int ks, int q) {
      const float* x = U[2 * ks + (q >> 1)] + (q & 1) * 2;
      split2(x[0] * up_u, x[1] * up_u, rh[ks][q], rl[ks][q]);
    };
#pragma unroll
    for (int q = 0; q < 4; ++q) split_u(0, q);
    // S <- exp(gamma_C) S + K^T (w U); the increment is summed by itself, so that the state's own
    // rounding is one fp32 fma a chunk.  Beside it o goes out, back in rows of tokens.
    const float dec = f[192];
    sbig[0] = sbig[1] = sbig[2] = sbig[3] = 0;
    auto at_k = [&](int i) {  // step i: 16 columns i / 4 of k, 16 tokens i % 4
      const int j = i >> 2;
      return K + (j >> 2) * kDcBlock + row_k + (((uint32_t)(j & 3) * 2u + pc_k) ^ sw) * 16u + (i & 3) * 2048;
    };
    __half* dst = a.o + ((t0 + (int64_t)c * kDcTok + g) * a.Hv + h) * kDeltaD + col + t2;
    const int64_t step = (int64_t)8 * a.Hv * kDeltaD;
    uint32_t kt[2][4];
    ldsm4_trans(at_k(0), kt[0]);
    float dh[2][2][4], dl[2][2][4];  // of two steps: one is summed up while the next one's MMAs run
    auto add_up = [&](int j, int x) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        S[2 * j + x][e] = fmaf(dec, S[2 * j + x][e], (dh[j & 1][x][e] + dl[j & 1][x][e]) * down_u);
        sbig[e] = max(sbig[e], magnitude(S[2 * j + x][e]));
      }
    };
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int z = j & 1;
#pragma unroll
      for (int e = 0; e < 4; ++e) dh[z][0][e] = dh[z][1][e] = dl[z][0][e] = dl[z][1][e] = 0.f;
      uint32_t ox = 0, oy = 0;
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        const int i = j * 4 + ks, x = i & 1;
        if (i < 31) ldsm4_trans(at_k(i + 1), kt[x ^ 1]);
        mma_16816(dh[z][0], rh[ks], kt[x][0], kt[x][1]);
        if (j == 0 && ks < 3) {
          split_u(ks + 1, 0);
          split_u(ks + 1, 1);
        }
        if (j > 0 && ks == 1) add_up(j - 1, 0);
        mma_16816(dh[z][1], rh[ks], kt[x][2], kt[x][3]);
        if (j == 0 && ks < 3) {
          split_u(ks + 1, 2);
          split_u(ks + 1, 3);
        }
        if (j > 0 && ks == 2) add_up(j - 1, 1);
        mma_16816(dl[z][0], rl[ks], kt[x][0], kt[x][1]);
        if (ks == 0) ox = transpose8x8(pack_half2(O[j][0] * down_r, O[j][1] * down_r));
        if (ks == 1) oy = transpose8x8(pack_half2(O[j][2] * down_r, O[j][3] * down_r));
        mma_16816(dl[z][1], rl[ks], kt[x][2], kt[x][3]);
      }
      if (j * 8 + g < n) {
        *reinterpret_cast<uint32_t*>(dst) = ox;
        *reinterpret_cast<uint32_t*>(dst + 8) = oy;
      }
      dst += step;
    }
    add_up(7, 0);
    add_up(7, 1);
    __syncwarp();
    if (lane == 0) mbar_arrive_reads(empty + s);
  }
  if (a.state_out && so >= 0) {
    float* dst = a.state_out + so * head_size + ((int64_t)h * kDeltaD + t2) * kDeltaD + col + g;
#pragma unroll
    for (int j = 0; j < 16; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) dst[(j * 8 + (e & 1)) * kDeltaD + (e >> 1) * 8] = S[j][e];
  }
  if (!C::kLoader && warp == 0) linger();
}

template <int W>
static int launch_scan(const ChunkArgs& p, const DeviceFacts& f, cudaStream_t s) {
  using C = ScanCfg<W>;
  const DeltaArgs& a = p.a;
  CUtensorMap tk, tq, tv;
  int rc = token_map(&tk, a.k, a.T, a.Hk, kDeltaD, a.ldk, 1, kDcTok);
  if (rc == TB_OK) rc = token_map(&tq, a.q, a.T, a.Hk, kDeltaD, a.ldq, 1, kDcTok);
  if (rc == TB_OK) rc = token_map(&tv, a.v, a.T, a.Hv, kDeltaD, a.ldv, 1, kDcTok);
  if (rc == TB_OK) rc = ensure_dynamic_smem(reinterpret_cast<const void*>(delta_scan_kernel<W>), f.device, C::kSmem);
  if (rc != TB_OK) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.B * a.Hv * (8 / W)));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, delta_scan_kernel<W>, tk, tq, tv, p);
  if (e != cudaSuccess) {
    record_cuda_error(e);
    return TB_ERR_CUDA;
  }
  return check_launch();
}

size_t delta_chunk_workspace(int64_t T, int64_t B, int64_t Hv) {
  return (size_t)((T / kDcTok + B) * Hv) * kDcItem;  // at most: ceil(x) <= floor(x) + 1 per request
}

int launch_delta_chunks(const DeltaArgs& a, void* workspace, cudaStream_t s) {
  DeviceFacts f;
  int rc = device_facts(&f);
  if (rc != TB_OK) return rc;
  ChunkArgs p;
  p.a = a;
  p.ws = static_cast<uint8_t*>(workspace);
  rc = ensure_dynamic_smem(reinterpret_cast<const void*>(delta_prep_kernel), f.device, kD1Smem);
  if (rc != TB_OK) return rc;
  const int64_t prep = (a.T / kDcTok + a.B) * a.Hk, heads = (int64_t)a.B * a.Hv;
  if (prep > INT32_MAX || heads > INT32_MAX / 2) return TB_ERR_TOO_LARGE;
  delta_prep_kernel<<<(unsigned)prep, kD1Threads, kD1Smem, s>>>(p);
  rc = check_launch();
  if (rc != TB_OK) return rc;
  // half heads per CTA while they do not fill the SMs: one warp per SM sub-partition each, where two
  // would share its tensor core
  return heads * 2 <= f.sms ? launch_scan<4>(p, f, s) : launch_scan<8>(p, f, s);
}

}  // namespace tb
