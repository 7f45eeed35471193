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
// Kernel 2, a CTA per (request, value head, 32 columns of v), walks the chunks.  The state is fp32 in
// registers (thread = row of S); every product is a tcgen05 MMA of 128 rows, its fp32 result in tensor
// memory:
//   [K; Q] S      rows: 64 tokens of K and of Q       -> S^T k, S^T q
//   [T; P T] R    rows: 64 tokens twice               -> U, the chunk's part of o
//   K^T (w U)     rows: the 128 rows of the state     -> the state's increment
// An fp32 factor (S, R, w U) goes in as two fp16 terms, x 2^e = hi + lo 2^-11, side by side in the 64
// columns of one operand, so that one MMA gives both partial sums: 22 bits of x, with a power of two
// per chunk that keeps it inside fp16's range (operand_scale).  K and Q are fp16 already.  T also has
// two terms.  What goes into o alone (P T) has one.
// The products of a chunk depend on one another through S, so a CTA's chunk costs three round trips
// between tensor memory and registers, about 1.3 us; two CTAs share an SM and fill each other's waits.
//
// [K; Q] has to be 128 consecutive rows, K is needed until the chunk's last product, and Q's room can
// be used again after the first: K has two places, with Q between them, and every other chunk reads
// [Q; K] and [P T; T] instead.
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
constexpr int kDcCols = 32;   // columns of v per CTA of kernel 2
constexpr int kDcBlock = kDcTok * 128;  // bytes of a 64 x 64 fp16 image
// a (chunk, value head) in the workspace: [T; P T] (or [P T; T]), T's low part, factors
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

TB_DEVI void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
TB_DEVI void ldsm4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
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
    const int t_at = (c & 1) ? kDcBlock : 0, pt_at = kDcBlock - t_at;  // odd chunks: [P T; T]
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int o = (e * 64 + l64) * 16;
      *reinterpret_cast<uint4*>(item + t_at + o) = *reinterpret_cast<const uint4*>(img + o);
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
          *reinterpret_cast<uint32_t*>(item + pt_at + i * 128 + ((j ^ (i & 7)) << 4) + (lane & 3) * 4) =
              pack_half2(acc[j][2 * e], acc[j][2 * e + 1]);
        }
    }
    sync_pair();  // the image has been read before the next head's A^T takes its place
  }
}

// ---------------------------------------------------------------- kernel 2
constexpr int kD2Threads = 192;  // warps 0-3: registers <-> tensor memory; 4: loads; 5: MMAs
constexpr int kD2KQ = 24576;     // 64 elements of [K even | Q | K odd], 64 rows each
constexpr int kD2X = 2 * kD2KQ;              // [T; P T]
constexpr int kD2TLow = kD2X + 2 * kDcBlock; // T's low part (what lies behind it is read as idle rows)
constexpr int kD2S = kD2TLow + kDcBlock;     // the state's operand: 128 rows of 128 bytes
constexpr int kD2R = kD2S + 16384;           // R, then w U: 64 rows of 128 bytes
constexpr int kD2Bars = kD2R + kDcBlock;
constexpr int kD2Smem = kD2Bars + 256 + 1024;
constexpr float kDcLow = 1.f / 2048.f;

// 16 fp32 values (columns 16 half ..) of a row of the operand [hi (32 halves) | lo (32 halves)], in the
// 128-byte swizzle; x = hi + lo / 2048
TB_DEVI void store_split(uint32_t base, int row, int half, const float (&x)[16]) {
  const uint32_t at = base + (uint32_t)row * 128u, sw = (uint32_t)row & 7u;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float u = x[c * 8 + e * 2], v = x[c * 8 + e * 2 + 1];
      const __half2 h = __floats2half2_rn(u, v);
      const float2 f = __half22float2(h);
      hi[e] = *reinterpret_cast<const uint32_t*>(&h);
      lo[e] = pack_half2((u - f.x) * 2048.f, (v - f.y) * 2048.f);
    }
    const uint32_t k = (uint32_t)(half * 2 + c);
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at + 16u * (k ^ sw)), "r"(hi[0]), "r"(hi[1]), "r"(hi[2]),
                 "r"(hi[3])
                 : "memory");
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at + 16u * ((k + 4) ^ sw)), "r"(lo[0]), "r"(lo[1]),
                 "r"(lo[2]), "r"(lo[3])
                 : "memory");
  }
}

// 16 columns of the high and of the low partial sums of the thread's lane; complete after tmem_wait_ld()
TB_DEVI void tmem_ld16(uint32_t taddr, float (&d)[16]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(d);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// The operands' scale for magnitudes up to `bits` (an fp32's): a power of two that takes them to 2^7.
// S, R and w U of the next chunk are at most some 2^8 times the largest of S now and of the next v
// (a column of S grows by at most 64 steps of |v|, and 128 of its elements meet a k of norm 1), so
// fp16's 2^15 holds them, and 22 bits remain down to 2^-26 of that.  Inputs for which this does not
// hold (steps above 1 on long keys) overflow to infinity, as the recurrence itself then does.
TB_DEVI float operand_scale(uint32_t bits, float& inverse) {
  int e = 261 - (int)(bits >> 23);
  e = e < 127 - 60 ? 127 - 60 : (e > 127 + 60 ? 127 + 60 : e);
  inverse = __int_as_float((254 - e) << 23);
  return __int_as_float(e << 23);
}

__global__ void __launch_bounds__(kD2Threads, 2)
    delta_scan_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmQ, const ChunkArgs p) {
  const DeltaArgs& a = p.a;
  extern __shared__ uint8_t d2_raw[];
  const uint32_t raw = smem_u32(d2_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = d2_raw + (base - raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kD2Bars);
  uint64_t *k_full = bars, *k_empty = bars + 2;  // [2] each
  uint64_t *q_full = bars + 4, *q_empty = bars + 5, *x_full = bars + 6, *x_empty = bars + 7;
  uint64_t *s_ready = bars + 8, *r_ready = bars + 9, *u_ready = bars + 10;
  uint64_t *d1_full = bars + 11, *d2_full = bars + 12, *d3_full = bars + 13;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 14);
  volatile int* aborted = reinterpret_cast<volatile int*>(bars + 15);
  // largest |S|, |v| that a chunk's operands come from, as fp32 bits: one word for this chunk, one that
  // is being collected for the next, one to spare
  uint32_t* largest = reinterpret_cast<uint32_t*>(bars + 16);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kSlices = kDeltaD / kDcCols;
  const int slice = (int)(blockIdx.x % kSlices);
  const int64_t bh = blockIdx.x / kSlices;
  const int h = (int)(bh % a.Hv), b = (int)(bh / a.Hv), hk = h / (a.Hv / a.Hk);

  if (tid == 0) {
    *aborted = 0;
    largest[0] = largest[1] = largest[2] = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(k_full + i, 1);
      mbar_init(k_empty + i, 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(x_full, 1);
    mbar_init(x_empty, 1);
    mbar_init(s_ready, 4);
    mbar_init(r_ready, 2);
    mbar_init(u_ready, 4);
    mbar_init(d1_full, 1);
    mbar_init(d2_full, 1);
    mbar_init(d3_full, 1);
    fence_barrier_init();
  }
  if (warp == 5) tmem_alloc(tmem_slot, 256);

  int64_t t0, len;
  if (!delta_rows(a, b, t0, len)) {
    if (tid == 0 && h == 0 && slice == 0) set_status(a.status, TB_DEV_BAD_LEN);
    len = 0;
  }
  const int nc = (int)((len + kDcTok - 1) / kDcTok);
  // the request's first chunk
  int64_t first = 0;
  {
    const ChunkScan sc = chunk_scan(a, lane);
    int64_t before = sc.upto - sc.own;
    const int src = b / sc.per;
    if (lane == src)
      for (int i = lane * sc.per; i < b; ++i) before += chunks_of(a, i);
    first = __shfl_sync(0xffffffffu, before, src);
  }
  auto item = [&](int c) { return p.ws + ((first + c) * a.Hv + h) * (int64_t)kDcItem; };

  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = *tmem_slot;
  // tensor memory: [K;Q] S | [T;PT] R | T low R | K^T wU, 64 columns each
  constexpr uint32_t kT1 = 0, kT2 = 64, kT2b = 128, kT3 = 192;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity) || *aborted) return;
    if (!mbar_wait(bar, parity)) {
      *aborted = 1;
      set_status(a.status, TB_DEV_TIMEOUT);
    }
  };

  if (warp == 4) {
    if (lane == 0) {
      bool waited = false;
      for (int c = 0; c < nc; ++c) {
        const int odd = c & 1, row = (int)(t0 + (int64_t)c * kDcTok);
        if (c >= 2) wait(k_empty + odd, ((c >> 1) - 1) & 1);
        mbar_arrive_expect_tx(k_full + odd, 2 * kDcBlock);
        for (int d = 0; d < 2; ++d)
          tma_load_3d<1>(base + d * kD2KQ + odd * 2 * kDcBlock, &tmK, d * 64, hk, row, smem_u32(k_full + odd));
        if (c >= 1) wait(q_empty, (c - 1) & 1);
        mbar_arrive_expect_tx(q_full, 2 * kDcBlock);
        for (int d = 0; d < 2; ++d) tma_load_3d<1>(base + d * kD2KQ + kDcBlock, &tmQ, d * 64, hk, row, smem_u32(q_full));
        if (c >= 1) wait(x_empty, (c - 1) & 1);
        if (!waited) {  // kernel 1's results
          asm volatile("griddepcontrol.wait;" ::: "memory");
          waited = true;
        }
        mbar_arrive_expect_tx(x_full, 3 * kDcBlock);
        bulk_g2s(smem + kD2X, item(c), 3 * kDcBlock, x_full);
      }
      if (*aborted) {  // a wait gave up: leave the copies in flight time to land before the CTA ends
        const uint64_t t = globaltimer_ns();
        while (globaltimer_ns() - t < 1000000) {
        }
      }
    }
    __syncwarp();
  } else if (warp == 5) {
    if (lane == 0) {
      constexpr uint32_t kN64 = (64u >> 3) << 17, kM128 = (128u >> 4) << 24, kF32 = 1u << 4, kTransA = 1u << 15,
                         kTransB = 1u << 16;
      constexpr uint32_t kId = kF32 | kTransB | kN64 | kM128, kIdT = kId | kTransA;
      const uint64_t sdesc = smem_desc_mn128(base + kD2S, 0, 1024), rdesc = smem_desc_mn128(base + kD2R, 0, 1024);
      for (int c = 0; c < nc; ++c) {
        const int odd = c & 1;
        wait(k_full + odd, (c >> 1) & 1);
        wait(q_full, c & 1);
        wait(s_ready, c & 1);
        tmem_fence_after();
#pragma unroll
        for (int d = 0; d < 2; ++d)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_f16_ss<1>(tmem + kT1, smem_desc_sw128(base + d * kD2KQ + odd * kDcBlock + kk * 32, 1024),
                          sdesc + (d * 4 + kk) * (2048 >> 4), kId, (d | kk) != 0);
        mma_commit(d1_full);
        mma_commit(q_empty);
        wait(x_full, c & 1);
        wait(r_ready, c & 1);
        tmem_fence_after();
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_f16_ss<1>(tmem + kT2, smem_desc_sw128(base + kD2X + kk * 32, 1024), rdesc + kk * (2048 >> 4), kId, kk != 0);
        // T's low part in the rows that T has: the other 64 rows read whatever lies there, into lanes
        // that nobody reads
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_f16_ss<1>(tmem + kT2b, smem_desc_sw128(base + kD2TLow - odd * kDcBlock + kk * 32, 1024),
                        rdesc + kk * (2048 >> 4), kId, kk != 0);
        mma_commit(d2_full);
        mma_commit(x_empty);
        wait(u_ready, c & 1);
        tmem_fence_after();
        const uint64_t kt = smem_desc_mn128(base + odd * 2 * kDcBlock, kD2KQ, 1024);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_f16_ss<1>(tmem + kT3, kt + kk * (2048 >> 4), rdesc + kk * (2048 >> 4), kIdT, kk != 0);
        mma_commit(d3_full);
        mma_commit(k_empty + odd);
      }
    }
    __syncwarp();
  } else {
    const int row = tid;  // of the state, and lane of tensor memory
    const uint32_t mine = tmem + ((uint32_t)warp << 21);
    const int64_t si = delta_slot(a.slot_in, b, a.n_in, a.status), so = delta_slot(a.slot_out, b, a.n_out, a.status);
    const int64_t in_head = ((int64_t)h * kDeltaD + row) * kDeltaD + slice * kDcCols;
    const int64_t head_size = (int64_t)a.Hv * kDeltaD * kDeltaD;
    float S[32];
    if (a.state_in && si >= 0) {
      const float4* src = reinterpret_cast<const float4*>(a.state_in + si * head_size + in_head);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 v = __ldg(src + i);
        S[4 * i] = v.x;
        S[4 * i + 1] = v.y;
        S[4 * i + 2] = v.z;
        S[4 * i + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) S[i] = 0.f;
    }
    const int tok = row & 63;
    // what a chunk needs besides the MMAs: the token's factors, and v where the thread has its K row
    // (it has K rows in one chunk and Q rows in the next); fetched a chunk ahead
    float f0 = 0.f, f1 = 0.f, decay = 0.f;
    uint4 v[4];
    auto fetch = [&](int c) {
      const float* f = reinterpret_cast<const float*>(item(c) + kDcFactors);
      const bool keys = (row >> 6) == (c & 1);
      decay = __ldcg(f + 192);
      f0 = __ldcg(f + (keys ? 0 : 128) + tok);
      if (keys) {
        f1 = __ldcg(f + 64 + tok);
        const int64_t t = t0 + (int64_t)c * kDcTok + tok;
        const uint4* vp = reinterpret_cast<const uint4*>(a.v + t * a.ldv + h * kDeltaD + slice * kDcCols);
        const bool live = t < t0 + len;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = live ? __ldg(vp + i) : make_uint4(0, 0, 0, 0);
      }
    };
    auto collect = [&](uint32_t bits, int c) {  // into the word of chunk c
      bits = __reduce_max_sync(0xffffffffu, bits);
      if (lane == 0) atomicMax(largest + c % 3, bits);
    };
    auto largest_s = [&]() {
      float m = 0.f;
      bool nan = false;
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        m = fmaxf(m, fabsf(S[i]));
        nan |= S[i] != S[i];
      }
      return nan ? 0x7f800000u : __float_as_uint(m);
    };
    auto largest_v = [&]() {  // fp16 magnitudes order as integers
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) m = max(m, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
      }
      return m >= 0x7c00u ? 0x7f800000u : __float_as_uint(half_bits_to_float((uint16_t)m));
    };
    float up = 1.f, down = 1.f;  // the chunk's scale and its inverse
    auto store_state = [&]() {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float y[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = S[half * 16 + i] * up;
        store_split(base + kD2S, row, half, y);
      }
      fence_proxy_async_smem();
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(s_ready);
    };
    if (nc > 0) {
      asm volatile("griddepcontrol.wait;" ::: "memory");
      fetch(0);
      collect(largest_s(), 0);
      if ((row >> 6) == 0) collect(largest_v(), 0);
      asm volatile("bar.sync 1, 128;" ::: "memory");
      up = operand_scale(*reinterpret_cast<volatile uint32_t*>(largest), down);
      store_state();
    }
    for (int c = 0; c < nc; ++c) {
      const int odd = c & 1;
      const bool keys = (row >> 6) == odd;  // this thread's token: its K row (R, U), or its Q row (o)
      const bool live = (int64_t)c * kDcTok + tok < len;
      const float c0 = f0, c1 = f1, dec = decay;
      uint4 cv[4];
      if (keys) {
#pragma unroll
        for (int i = 0; i < 4; ++i) cv[i] = v[i];
      }
      if (c + 1 < nc) fetch(c + 1);
      if (row == 0) largest[(c + 2) % 3] = 0;
      collect(largest_s(), c + 1);
      wait(d1_full, c & 1);
      tmem_fence_after();
      if (keys) {
        // R = v - exp(gamma) S^T k, all times the scale
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float x[16], y[16];
          tmem_ld16(mine + kT1 + half * 16, x);
          tmem_ld16(mine + kT1 + 32 + half * 16, y);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const __half2* hv = reinterpret_cast<const __half2*>(&cv[half * 2 + i]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int k = i * 8 + e * 2;
              const float2 w = __half22float2(hv[e]);
              x[k] = live ? fmaf(-c0, fmaf(y[k], kDcLow, x[k]), w.x * up) : 0.f;
              x[k + 1] = live ? fmaf(-c0, fmaf(y[k + 1], kDcLow, x[k + 1]), w.y * up) : 0.f;
            }
          }
          store_split(base + kD2R, tok, half, x);
        }
        fence_proxy_async_smem();
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(r_ready);
        wait(d2_full, c & 1);
        tmem_fence_after();
        // w U
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float x[16], y[16], z[16];
          tmem_ld16(mine + kT2 + half * 16, x);
          tmem_ld16(mine + kT2 + 32 + half * 16, y);
          tmem_ld16(mine + kT2b + half * 16, z);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = live ? c1 * (fmaf(y[i], kDcLow, x[i]) + z[i]) : 0.f;
          store_split(base + kD2R, tok, half, x);
        }
        if (!live) {  // rows of K that are another request's: out of the sum over the tokens
#pragma unroll
          for (int d = 0; d < 2; ++d)
#pragma unroll
            for (int e = 0; e < 8; ++e)
              asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(base + d * kD2KQ + odd * 2 * kDcBlock +
                                                                         (uint32_t)tok * 128u + e * 16),
                           "r"(0)
                           : "memory");
        }
        fence_proxy_async_smem();
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(u_ready);
      } else {
        // o = exp(gamma) scale S^T q + the chunk's own part
        float y[32];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float x[16], z[16];
          tmem_ld16(mine + kT1 + half * 16, x);
          tmem_ld16(mine + kT1 + 32 + half * 16, z);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) y[half * 16 + i] = c0 * fmaf(z[i], kDcLow, x[i]);
        }
        if (c + 1 < nc) collect(largest_v(), c + 1);  // the next chunk's v, which this thread has
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(u_ready);  // the word for the next chunk's scale is complete
        wait(d2_full, c & 1);
        tmem_fence_after();
        uint4* dst = reinterpret_cast<uint4*>(a.o + ((t0 + (int64_t)c * kDcTok + tok) * a.Hv + h) * kDeltaD + slice * kDcCols);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float x[16], z[16];
          tmem_ld16(mine + kT2 + half * 16, x);
          tmem_ld16(mine + kT2 + 32 + half * 16, z);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = down * (y[half * 16 + i] + fmaf(z[i], kDcLow, x[i]));
          if (live) {
            dst[half * 2] = make_uint4(pack_half2(x[0], x[1]), pack_half2(x[2], x[3]), pack_half2(x[4], x[5]),
                                       pack_half2(x[6], x[7]));
            dst[half * 2 + 1] = make_uint4(pack_half2(x[8], x[9]), pack_half2(x[10], x[11]), pack_half2(x[12], x[13]),
                                           pack_half2(x[14], x[15]));
          }
        }
      }
      wait(d3_full, c & 1);
      tmem_fence_after();
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float x[16], y[16];
        tmem_ld16(mine + kT3 + half * 16, x);
        tmem_ld16(mine + kT3 + 32 + half * 16, y);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i)
          S[half * 16 + i] = fmaf(dec, S[half * 16 + i], fmaf(y[i], kDcLow, x[i]) * down);
      }
      if (c + 1 < nc) {
        up = operand_scale(*reinterpret_cast<volatile uint32_t*>(largest + (c + 1) % 3), down);
        store_state();
      }
    }
    if (a.state_out && so >= 0) {
      float4* dst = reinterpret_cast<float4*>(a.state_out + so * head_size + in_head);
#pragma unroll
      for (int i = 0; i < 8; ++i) dst[i] = make_float4(S[4 * i], S[4 * i + 1], S[4 * i + 2], S[4 * i + 3]);
    }
  }
  tmem_fence_before();
  __syncthreads();
  if (warp == 5) tmem_dealloc(tmem, 256);
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
  CUtensorMap tk, tq;
  rc = token_map(&tk, a.k, a.T, a.Hk, kDeltaD, a.ldk, 1, kDcTok);
  if (rc == TB_OK) rc = token_map(&tq, a.q, a.T, a.Hk, kDeltaD, a.ldq, 1, kDcTok);
  if (rc == TB_OK) rc = ensure_dynamic_smem(reinterpret_cast<const void*>(delta_prep_kernel), f.device, kD1Smem);
  if (rc == TB_OK) rc = ensure_dynamic_smem(reinterpret_cast<const void*>(delta_scan_kernel), f.device, kD2Smem);
  if (rc != TB_OK) return rc;
  const int64_t prep = (a.T / kDcTok + a.B) * a.Hk, scan = (int64_t)a.B * a.Hv * (kDeltaD / kDcCols);
  if (prep > INT32_MAX || scan > INT32_MAX) return TB_ERR_TOO_LARGE;
  delta_prep_kernel<<<(unsigned)prep, kD1Threads, kD1Smem, s>>>(p);
  rc = check_launch();
  if (rc != TB_OK) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)scan);
  cfg.blockDim = dim3(kD2Threads);
  cfg.dynamicSmemBytes = kD2Smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, delta_scan_kernel, tk, tq, p);
  if (e != cudaSuccess) {
    record_cuda_error(e);
    return TB_ERR_CUDA;
  }
  return check_launch();
}

}  // namespace tb
