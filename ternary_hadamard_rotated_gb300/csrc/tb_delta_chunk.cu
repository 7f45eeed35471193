// The gated delta rule over prompts, in chunks of 64 tokens (csrc/tb_delta.cu has the recurrent form
// and the entry point).
//
// Inside a chunk, with gamma_i the decays' running sum, D_ij = exp(gamma_i - gamma_j) for j <= i, S the
// state before the chunk, and q, k already divided by their norms:
//   A_ij = (k_i . k_j) D_ij beta_j  (j < i),     T = (I + A)^-1
//   R_i  = v_i - exp(gamma_i) S^T k_i,           U = diag(beta) T R
//   o_i  = scale (exp(gamma_i) S^T q_i + sum_{j <= i} (q_i . k_j) D_ij u_j)
//   S   <- exp(gamma_C) S + sum_j exp(gamma_C - gamma_j) k_j u_j^T
// T does not depend on the state, so one kernel computes it for all chunks at once, and with it
// P T, P_ij = scale (q_i . k_j) D_ij beta_j: the second kernel then gets U and the chunk's own part of o from
// one product [T; P T] R.  The steps beta stand where no fp16 operand depends on their size: T has ones on its
// diagonal and, where a step contracts (beta |k|^2 <= 2), nothing above beta_j |k_i| |k_j| beside it; P T goes under
// a power of two a chunk and head, from its largest value; and U's rows take beta in fp32.  (With diag(beta) inside
// T, steps below 2^-14 were left with the bits of fp16's subnormal numbers.)  Steps that do not contract make T grow:
// up to 65504 times within a chunk it is held.
//
// Kernel 1, a CTA per (chunk, key head), which its value heads share: K K^T and Q K^T by mma.sync (fp16
// inputs, exact products), per value head the triangular system by blocks of 16 and P T.  It writes T
// (fp16, high and low part) and P T (fp16) as the fragments that kernel 2's MMAs take, and each token's
// factors.  8192 tokens, 16/48 heads: 109 us, bound by the latency of each head's chain of steps.
//
// Kernel 2 walks the chunks, a warp per 16 columns of v, which no other warp's columns depend on: S^T
// stays in the warp's registers as fp32 accumulators of mma.sync, and every product's left factor (S^T,
// R^T, (w U)^T, 16 rows) comes out of the product before it in the layout that the next one wants, so
// a chunk has no exchange between warps at all.  K, Q, V and kernel 1's results come by TMA, three
// chunks deep, and the next item's state (read by the warps themselves, 64 requests of one chunk took 351
// us instead of 308 at that time; 317 now).  An fp32 factor goes in as two fp16 terms, x 2^e = hi + lo with the warp's largest |x|
// at 2^14: 22 bits, and K and Q are fp16 already.  T has two terms too.  What goes into o alone is rounded
// once: P T, and the state in S^T q, to fp16.
// 8192 tokens: 348 us, 2.7 us a chunk.  Its 420 MMAs a warp, at one per 7.8 clocks and SM sub-partition,
// are 1.7 of them; the rest is the issue and the latencies of one warp's own chain.  (With a second warp on
// the sub-partition that makes o from S and R, passed through shared memory, the call took 476 us instead
// of 445; it is 454 now, with the power of two of P T.  The same walk on tcgen05, 32
// columns a CTA, took 2.7 us a chunk alone on its SM and 3.4 with a second CTA, with fewer terms: 20
// MMAs of 44 to 60 clocks, and three trips through registers, shared memory and a barrier of 800 to
// 1000 each.)  CTAs stay and take the (request, head, half) items with the most chunks first; the loading
// warp goes on to the next item's chunks.
#include <cuda.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>

#include "tb_attention.cuh"
#include "tb_attn_tc.cuh"
#include "tb_common.cuh"
#include "tb_delta.cuh"
#include "tb_host.h"

namespace tb {

constexpr int kDcTok = 64;              // tokens per chunk
constexpr int kDcBlock = kDcTok * 128;  // bytes of a 64 x 64 fp16 image
// A (chunk, value head) in the workspace: T, P T and T's low part, then the tokens' factors.  Of each matrix
// the ten 16 x 16 blocks up to the diagonal, block (i, j) at i (i + 1) / 2 + j, as the right operand's
// fragments of mma.sync: 16 bytes a lane.
constexpr int kDcFrag = 512, kDcMatrix = 10 * kDcFrag;
constexpr int kDcItem = 16384;
// floats: c [64], w [64], q [64], exp(gamma_C), the tokens before the first whose k, decay or step is not
// finite, and what takes P T's power of two off again
constexpr int kDcFactors = 3 * kDcMatrix;
// The powers of two of P T, and of R against S, stay below 2^36, so that their product with a sum of 2^37 (S^T q)
// stays inside fp32.  P T below 2^-36 2^-25 adds nothing to an fp16 output, nor does R below 2^-36 of S to a state
// in fp32.
constexpr int kDcPScale = 36;

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

// Chunks that the workspace has room for and kernel 1 makes.  Requests in order, one after another, have no more
// (ceil(x) <= floor(x) + 1); where row starts go back, requests that lie in [0, T] one by one can have more
// together, and those whose chunks come later than this are not computed.
TB_DEVI int64_t chunk_room(const DeltaArgs& a) { return a.T / kDcTok + a.B; }
// the request's first chunk among all requests' (whole warps call this)
TB_DEVI int64_t first_chunk(const DeltaArgs& a, const ChunkScan& s, int b, int lane) {
  int64_t first = s.upto - s.own;
  const int src = b / s.per;
  if (lane == src)
    for (int r = lane * s.per; r < b; ++r) first += chunks_of(a, r);
  return __shfl_sync(0xffffffffu, first, src);
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

// x, y -> fp16 pair and the fp16 pair of what it leaves
TB_DEVI void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x, y);
  const float2 f = __half22float2(h);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = pack_half2(x - f.x, y - f.y);
}
// the same of x * scale, y * scale
TB_DEVI void split2(const float* x, float scale, uint32_t& hi, uint32_t& lo) {
  const float2 u = mul_f32x2(make_float2(x[0], x[1]), make_float2(scale, scale));
  const __half2 h = __floats2half2_rn(u.x, u.y);
  const float2 r = fma_f32x2(__half22float2(h), make_float2(-1.f, -1.f), u);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = pack_half2(r.x, r.y);
}
TB_DEVI float2 lds2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr));
  return v;
}
TB_DEVI void lds4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
// the largest magnitude
TB_DEVI float max3_abs(float a, float b, float c) {
  float d;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// two values of a tile's row by their own factors
TB_DEVI void mul_pair(float* x, float2 f) {
  const float2 y = mul_f32x2(make_float2(x[0], x[1]), f);
  x[0] = y.x;
  x[1] = y.y;
}
TB_DEVI uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// (hi, lo) += (x, y): a sum of fp32 pairs, hi the rounded sum and lo what it leaves (Knuth's two-sum)
TB_DEVI void add_pair(float& hi, float& lo, float x, float y) {
  const float s = __fadd_rn(hi, x), b = __fsub_rn(s, hi);
  const float e = __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(x, b));
  const float t = __fadd_rn(__fadd_rn(lo, y), e);
  hi = __fadd_rn(s, t);
  lo = __fsub_rn(t, __fsub_rn(hi, s));
}

// ---------------------------------------------------------------- kernel 1
constexpr int kD1Threads = 128;
constexpr int kD1Pitch = 136;               // halves per row of K and Q in shared memory
constexpr int kD1KQ = 64 * kD1Pitch * 2;    // bytes of one of them
static_assert(2 * kD1KQ >= 4 * kDcBlock, "two heads' images take the place of K and Q");

// Warp w has rows 16 w .. of the chunk's matrices, as accumulator tiles of 8 columns.  (I + A)^-1 block by
// block of 16: the diagonal blocks D_w by substitution (a lane per column), then with E = D A (left of
// the diagonal) T_w = D_w - sum_{s < w} E_ws T_s, one block row a step, fp32 factors in two
// fp16 terms (three products).  P T goes along, P from Q K^T's accumulators as they are.
__global__ void __launch_bounds__(kD1Threads, 4) delta_prep_kernel(const ChunkArgs p) {
  const DeltaArgs& a = p.a;
  __shared__ __align__(1024) uint8_t kq[2 * kD1KQ];
  __shared__ float rk[64], rq[64];
  __shared__ float nk[64], nq[64];  // the norms of k as it enters and of scale q
  __shared__ int pscale[4];         // the exponent of P's power of two
  __shared__ float most_pt[2][4];   // the largest of P T, by warps, of two heads in turn
  __shared__ __align__(16) float2 gam[4][64];  // running sums of the decays in log2 units, high and low part
  __shared__ __align__(8) float bet[4][64];
  __shared__ int sound[4];       // tokens before the first whose k, decay or step is not finite
  __shared__ __align__(16) float diag_t[4][16][20];  // a warp's diagonal block of A, transposed
  __shared__ float diag[4][16][17];                  // its inverse
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

  // the decays and steps of the head that this warp sums up next, two tokens a lane
  const int group = a.Hv / a.Hk;
  float next_g[2] = {0.f, 0.f}, next_b[2] = {0.f, 0.f};
  auto fetch_decays = [&](int h4) {
    if (h4 + warp >= group) return;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int64_t at = (t0 + lane * 2 + e) * a.Hv + hk * group + h4 + warp;
      const bool in = lane * 2 + e < n;
      next_g[e] = in ? __ldg(a.g + at) : 0.f;
      next_b[e] = in ? __ldg(a.beta + at) : 0.f;
    }
  };
  fetch_decays(0);

  // K and Q; rows past the request's end are zeros
  __half* Ks = reinterpret_cast<__half*>(kq);
  __half* Qs = reinterpret_cast<__half*>(kq + kD1KQ);
  {
    const int part = (tid & 15) * 8;
    uint4 w[16];  // eight rows of K, then of Q, sixteen threads a row
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int row = (r & 7) * 8 + (tid >> 4);
      const __half* src = r < 8 ? a.k + (t0 + row) * a.ldk : a.q + (t0 + row) * a.ldq;
      w[r] = row < n ? __ldg(reinterpret_cast<const uint4*>(src + hk * kDeltaD + part)) : make_uint4(0, 0, 0, 0);
    }
    float v[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      *reinterpret_cast<uint4*>((r < 8 ? Ks : Qs) + ((r & 7) * 8 + (tid >> 4)) * kD1Pitch + part) = w[r];
      const __half2* h2 = reinterpret_cast<const __half2*>(&w[r]);
      v[r] = 0.f;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float2 f = __half22float2(h2[x]);
        v[r] = fmaf(f.x, f.x, fmaf(f.y, f.y, v[r]));
      }
    }
    // the sixteen sums over sixteen lanes: each step halves the sums a lane carries; lane l ends with sum l
#pragma unroll
    for (int d = 8; d; d >>= 1) {
      const bool up = lane & d;
#pragma unroll
      for (int r = 0; r < d; ++r) {
        const float keep = up ? v[r + d] : v[r], give = up ? v[r] : v[r + d];
        v[r] = keep + __shfl_xor_sync(0xffffffffu, give, d);
      }
    }
    const int r = lane & 15, row = (r & 7) * 8 + (tid >> 4);
    float inv = a.normalise ? 1.f / sqrtf(v[0] + kDeltaEps) : 1.f;
    if (!(v[0] < INFINITY)) inv = NAN;
    const float norm = a.normalise ? 1.f : sqrtf(v[0]);  // (or a little less than 1)
    if (r < 8) {
      rk[row] = inv;
      nk[row] = norm;
    } else {
      rq[row] = inv * a.scale;
      nq[row] = norm < INFINITY ? norm * fabsf(a.scale) : 0.f;
    }
  }
  __syncthreads();

  // K K^T and Q K^T, tiles up to the diagonal
  float G[8][4], QK[8][4];
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) G[j][e] = QK[j][e] = 0.f;
#pragma unroll 2
  for (int k = 0; k < kDeltaD; k += 16) {
    uint32_t ak[4], aq[4];
    const int at = (warp * 16 + (lane & 15)) * kD1Pitch + k + (lane >> 4) * 8;
    ldsm4(smem_u32(Ks + at), ak);
    ldsm4(smem_u32(Qs + at), aq);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j > warp) break;
      uint32_t bf[4];  // keys j*16 + 0..7 (k, k+8), then 8..15
      ldsm4(smem_u32(Ks + (j * 16 + (lane & 7) + (lane >> 4) * 8) * kD1Pitch + k + ((lane >> 3) & 1) * 8), bf);
      mma_16816(G[2 * j], ak, bf[0], bf[1]);
      mma_16816(G[2 * j + 1], ak, bf[2], bf[3]);
      mma_16816(QK[2 * j], aq, bf[0], bf[1]);
      mma_16816(QK[2 * j + 1], aq, bf[2], bf[3]);
    }
  }
  const int g = lane >> 2, t2 = (lane & 3) * 2, i0 = warp * 16 + g;
  // every value head weighs them by the keys' and queries' norms
  {
    const float k0 = rk[i0], k1 = rk[i0 + 8], f0 = rq[i0], f1 = rq[i0 + 8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = rk[j * 8 + t2], y = rk[j * 8 + t2 + 1];
      G[j][0] *= k0 * x;
      G[j][1] *= k0 * y;
      G[j][2] *= k1 * x;
      G[j][3] *= k1 * y;
      QK[j][0] *= f0 * x;
      QK[j][1] *= f0 * y;
      QK[j][2] *= f1 * x;
      QK[j][3] *= f1 * y;
    }
  }

  for (int h4 = 0; h4 < group; ++h4) {
    const int slot = h4 & 3, h = hk * group + h4;
    if (slot == 0) {
      __syncthreads();  // K and Q, and the last four heads' sums, have been read
      if (h4 + warp < group) {  // a warp per head: the decays' sums, of two tokens a lane, as two floats
        float hi[2], lo[2];
        // From such a token on nothing is computed here (a zero times it would reach the tokens before it);
        // kernel 2 makes o and the state NaN from there.  A decay of minus infinity forgets, and is sound.
        unsigned bad[2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
          bad[e] = __ballot_sync(0xffffffffu, !(next_g[e] < INFINITY) || !(fabsf(next_b[e]) < INFINITY) ||
                                                  !(rk[lane * 2 + e] < INFINITY));
        const int f0 = bad[0] ? (__ffs(bad[0]) - 1) * 2 : 64, f1 = bad[1] ? (__ffs(bad[1]) - 1) * 2 + 1 : 64;
        const int ok = f0 < f1 ? f0 : f1;
        if (lane == 0) sound[warp] = ok;
        float most_b = 0.f;  // the largest beta |k|
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float gv = next_g[e] < -200.f ? -200.f : next_g[e];  // e^-200 is 0 in fp32 already
          hi[e] = gv * 1.44269502f;  // times log2 e, in two parts as well
          lo[e] = fmaf(gv, 1.44269502f, -hi[e]) + gv * 1.92596303e-8f;
          const bool in = lane * 2 + e < ok;
          bet[warp][lane * 2 + e] = in ? next_b[e] : 0.f;
          if (in) most_b = fmaxf(most_b, fabsf(next_b[e]) * nk[lane * 2 + e]);
        }
        most_b = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most_b)));
        const float most_q = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(nq[lane * 2], nq[lane * 2 + 1]))));
        if (lane == 0) {  // takes P's bound, scale max|q| max(beta |k|), to 2^12 .. 2^13
          const int e = 266 - (int)(__float_as_uint(most_b * most_q) >> 23);
          pscale[warp] = e < 127 - 60 ? 127 - 60 : (e > 127 + 60 ? 127 + 60 : e);
        }
        add_pair(hi[1], lo[1], hi[0], lo[0]);
        float sh = hi[1], sl = lo[1];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const float yh = __shfl_up_sync(0xffffffffu, sh, d), yl = __shfl_up_sync(0xffffffffu, sl, d);
          if (lane >= d) add_pair(sh, sl, yh, yl);
        }
        float ph = __shfl_up_sync(0xffffffffu, sh, 1), pl = __shfl_up_sync(0xffffffffu, sl, 1);
        if (lane == 0) ph = pl = 0.f;
        add_pair(hi[0], lo[0], ph, pl);
        gam[warp][lane * 2] = make_float2(hi[0], lo[0]);
        gam[warp][lane * 2 + 1] = make_float2(sh, sl);
      }
      fetch_decays(h4 + 4);
      __syncthreads();
    }
    uint8_t* item = p.ws + (chunk * a.Hv + h) * (int64_t)kDcItem;
    uint4* out = reinterpret_cast<uint4*>(item) + warp * (warp + 1) / 2 * 32 + lane;  // the warp's blocks
    uint8_t* img = kq + (h4 & 1) * 2 * kDcBlock;  // T's high part, then its low part
    const float2* gm = gam[slot];
    const float* be = bet[slot];
    if (tid < 64) {
      float* f = reinterpret_cast<float*>(item + kDcFactors);
      const float2 mine = gm[tid], last = gm[63];
      const float eg = ex2(mine.x) * (1.f + 0.6931472f * mine.y);
      f[tid] = tid < sound[slot] ? eg * rk[tid] : 0.f;  // (0 where kernel 2 has a row of zeros)
      f[64 + tid] = tid < sound[slot] ? ex2((last.x - mine.x) + (last.y - mine.y)) * rk[tid] * be[tid] : 0.f;
      if (tid == 0) {
        f[192] = ex2(last.x) * (1.f + 0.6931472f * last.y);
        f[193] = (float)sound[slot];
      }
    }
    // A (fp32, as accumulator tiles), P (two fp16 terms, as the left factor's tiles)
    float A[8][4];
    uint32_t P[4][4], Pl[4][4];
    {
      const float2 g0 = gm[i0], g1 = gm[i0 + 8];
      const int ok = sound[slot];
      const float ps = __int_as_float(pscale[slot] << 23);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j > 2 * warp + 1) {
          continue;
        }
        float pv[4];
        const float4 gk2 = *reinterpret_cast<const float4*>(&gm[j * 8 + t2]);  // of two tokens
        const float2 be2 = *reinterpret_cast<const float2*>(&be[j * 8 + t2]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int k = j * 8 + t2 + (e & 1), i = i0 + (e >> 1) * 8;
          const float2 gk = (e & 1) ? make_float2(gk2.z, gk2.w) : make_float2(gk2.x, gk2.y), gi = (e >> 1) ? g1 : g0;
          const bool in = i < ok;
          const float d = in && k <= i ? ex2((gi.x - gk.x) + (gi.y - gk.y)) : 0.f;
          const float db = d * ((e & 1) ? be2.y : be2.x);
          A[j][e] = in && k < i ? G[j][e] * db : 0.f;
          pv[e] = in && k <= i ? QK[j][e] * db * ps : 0.f;
        }
        split2(pv[0], pv[1], P[j >> 1][(j & 1) * 2], Pl[j >> 1][(j & 1) * 2]);
        split2(pv[2], pv[3], P[j >> 1][(j & 1) * 2 + 1], Pl[j >> 1][(j & 1) * 2 + 1]);
      }
    }
    // the diagonal block's inverse
#pragma unroll
    for (int w = 0; w < 4; ++w) {  // (the block's registers by a constant index)
      if (w != warp) continue;
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) diag_t[warp][x * 8 + t2 + (e & 1)][g + (e >> 1) * 8] = A[2 * w + x][e];
    }
    __syncwarp();
    if (lane < 16) {
      float x[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = i == lane ? 1.f : 0.f;
#pragma unroll
      for (int k = 0; k < 15; ++k) {
#pragma unroll
        for (int q = (k + 1) / 4; q < 4; ++q) {
          const float4 w = *reinterpret_cast<const float4*>(&diag_t[warp][k][q * 4]);
          if (q * 4 > k) x[q * 4] = fmaf(-w.x, x[k], x[q * 4]);
          if (q * 4 + 1 > k) x[q * 4 + 1] = fmaf(-w.y, x[k], x[q * 4 + 1]);
          if (q * 4 + 2 > k) x[q * 4 + 2] = fmaf(-w.z, x[k], x[q * 4 + 2]);
          x[q * 4 + 3] = fmaf(-w.w, x[k], x[q * 4 + 3]);
        }
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) diag[warp][i][lane] = x[i];
    }
    __syncwarp();
    // E = D A, negated, left of the diagonal block
    uint32_t eh[3][4], el[3][4];
    float T[8][4];
    {
      uint32_t dh[4], dl[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float* d = &diag[warp][g + (q & 1) * 8][t2 + (q >> 1) * 8];
        split2(-d[0], -d[1], dh[q], dl[q]);
      }
#pragma unroll
      for (int j = 0; j < 6; ++j) {
#pragma unroll
        for (int e = 0; e < 4; ++e) T[j][e] = 0.f;
        if (j >= 2 * warp) continue;
        uint32_t h0, h1, l0, l1;
        split2(A[j][0], A[j][1], h0, l0);
        split2(A[j][2], A[j][3], h1, l1);
        h0 = transpose8x8(h0);
        h1 = transpose8x8(h1);
        l0 = transpose8x8(l0);
        l1 = transpose8x8(l1);
        mma_16816(T[j], dh, h0, h1);
        mma_16816(T[j], dh, l0, l1);
        mma_16816(T[j], dl, h0, h1);
      }
#pragma unroll
      for (int s = 0; s < 3; ++s)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float* x = T[2 * s + (q >> 1)] + (q & 1) * 2;
          split2(x[0], x[1], eh[s][q], el[s][q]);
        }
    }
    // T's rows start from D
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        T[j][e] = 0.f;
        if (j >> 1 == warp) T[j][e] = diag[warp][g + (e >> 1) * 8][(j & 1) * 8 + t2 + (e & 1)];
      }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      if (warp == s) {  // this block row is complete
#pragma unroll
        for (int b = 0; b <= s; ++b) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int j = 2 * b + (q & 1), e = q >> 1;
            split2(T[j][2 * e], T[j][2 * e + 1], hi[q], lo[q]);
            const int i = i0 + e * 8, at = i * 128 + ((j ^ (i & 7)) << 4) + t2 * 2;
            *reinterpret_cast<uint32_t*>(img + at) = hi[q];
            *reinterpret_cast<uint32_t*>(img + kDcBlock + at) = lo[q];
          }
          out[b * 32] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          out[kDcMatrix / 8 + b * 32] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
      }
      __syncthreads();
      if (warp <= s) continue;
      uint32_t th[3][4], tl[3][4];
      const int x = s < 3 ? s : 0;  // (no warp is past the last step)
      const uint32_t row = smem_u32(img) + (s * 16 + (lane & 15)) * 128;
#pragma unroll
      for (int j = 0; j <= x; ++j) {
        const uint32_t at = row + (((j * 2 + (lane >> 4)) ^ (lane & 7)) << 4);
        ldsm4_trans(at, th[j]);
        ldsm4_trans(at + kDcBlock, tl[j]);
      }
      // (term by term over the tiles, so that no product waits for the one before it)
#pragma unroll
      for (int j = 0; j <= x; ++j) {
        mma_16816(T[2 * j], eh[x], th[j][0], th[j][1]);
        mma_16816(T[2 * j + 1], eh[x], th[j][2], th[j][3]);
      }
#pragma unroll
      for (int j = 0; j <= x; ++j) {
        mma_16816(T[2 * j], eh[x], tl[j][0], tl[j][1]);
        mma_16816(T[2 * j + 1], eh[x], tl[j][2], tl[j][3]);
      }
#pragma unroll
      for (int j = 0; j <= x; ++j) {
        mma_16816(T[2 * j], el[x], th[j][0], th[j][1]);
        mma_16816(T[2 * j + 1], el[x], th[j][2], th[j][3]);
      }
    }
    // P T, in T's registers
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) T[j][e] = 0.f;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      if (s > warp) break;
#pragma unroll
      for (int j = 0; j <= s; ++j) {
        uint32_t th[4], tl[4];
        const uint32_t at = smem_u32(img) + (s * 16 + (lane & 15)) * 128 + (((j * 2 + (lane >> 4)) ^ (lane & 7)) << 4);
        ldsm4_trans(at, th);
        ldsm4_trans(at + kDcBlock, tl);
        mma_16816(T[2 * j], P[s], th[0], th[1]);
        mma_16816(T[2 * j + 1], P[s], th[2], th[3]);
        mma_16816(T[2 * j], P[s], tl[0], tl[1]);
        mma_16816(T[2 * j + 1], P[s], tl[2], tl[3]);
        mma_16816(T[2 * j], Pl[s], th[0], th[1]);
        mma_16816(T[2 * j + 1], Pl[s], th[2], th[3]);
      }
    }
    // its largest value to 2^14 .. 2^15
    float most = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) most = max3_abs(max3_abs(most, T[j][0], T[j][1]), T[j][2], T[j][3]);
    most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most)));
    if (lane == 0) most_pt[h4 & 1][warp] = most;
    __syncthreads();
    const float* mp = most_pt[h4 & 1];
    most = fmaxf(fmaxf(mp[0], mp[1]), fmaxf(mp[2], mp[3]));
    // both exponents together, biased, within kDcPScale above; what is left for here
    int e = pscale[slot] + 14 + 127 - (int)(__float_as_uint(most) >> 23);
    e = e < 127 - 100 ? 127 - 100 : (e > 127 + kDcPScale ? 127 + kDcPScale : e);
    const float rest = __int_as_float((e - pscale[slot] + 127) << 23);
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      if (b > warp) break;
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int q = 0; q < 4; ++q) T[2 * b + x][q] *= rest;
      out[kDcMatrix / 16 + b * 32] = make_uint4(pack_half2(T[2 * b][0], T[2 * b][1]), pack_half2(T[2 * b + 1][0], T[2 * b + 1][1]),
                                                pack_half2(T[2 * b][2], T[2 * b][3]), pack_half2(T[2 * b + 1][2], T[2 * b + 1][3]));
    }
    if (tid < 64) {
      float* f = reinterpret_cast<float*>(item + kDcFactors);
      const float2 mine = gm[tid];
      f[128 + tid] = ex2(mine.x) * (1.f + 0.6931472f * mine.y) * rq[tid] * __int_as_float(e << 23);
      if (tid == 0) f[194] = __int_as_float((254 - e) << 23);
    }
  }
}

// ---------------------------------------------------------------- kernel 2
constexpr int kD2Stages = 3;
constexpr int kD2Q = 2 * kDcBlock, kD2Item = 4 * kDcBlock, kD2V = kD2Item + kDcItem;  // places in a stage

constexpr int kD2Warps = 4;                     // that walk, 16 columns of v each; one more loads
constexpr int kD2Threads = (kD2Warps + 1) * 32;
constexpr int kD2Slices = kDeltaD / (kD2Warps * 16);  // CTAs a head
constexpr int kD2Stage = kD2V + kDcBlock;
constexpr int kD2Bytes = 5 * kDcBlock + kDcItem;  // loaded per chunk
// the next item's state: 128 rows of k, 64 columns of v, at a pitch that spreads the lanes' reads over the banks
constexpr int kD2StatePitch = 64 * 4 + 16, kD2State = kDeltaD * kD2StatePitch;
constexpr int kD2Smem = 1024 + kD2Stages * kD2Stage + kD2State + 128 + 1024;

// a power of two that takes the warp's largest magnitude to 2^14, 2^(top - 127) at most, and its inverse
TB_DEVI float operand_scale(const float (&most)[2], float& inverse, int top = 127 + 100) {
  const float m = fmaxf(most[0], most[1]);
  const uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(m));  // orders as the values do
  int e = 268 - (int)(bits >> 23);
  e = e < 127 - 100 ? 127 - 100 : (e > top ? top : e);
  inverse = __int_as_float((254 - e) << 23);
  return __int_as_float(e << 23);
}
// Arrival that hands a place back after reads whose values have been used: nothing to release (a release
// waits for the warp's global stores too, 400 clocks a chunk).
TB_DEVI void mbar_arrive_reads(uint64_t* bar) {
  asm volatile("mbarrier.arrive.relaxed.cta.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__global__ void __launch_bounds__(kD2Threads, 1)
    delta_scan_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmQ,
                      const __grid_constant__ CUtensorMap tmV, const ChunkArgs p) {
  const DeltaArgs& a = p.a;
  extern __shared__ uint8_t d2_raw[];
  const uint32_t raw = smem_u32(d2_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = d2_raw + (base - raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kD2Stages * kD2Stage + kD2State);
  uint64_t* ready = full + kD2Stages;  // the loading warp has looked the stage over
  uint64_t* empty = full + 2 * kD2Stages;
  uint64_t* state_full = full + 3 * kD2Stages;
  uint64_t* state_empty = state_full + 1;
  volatile int* aborted = reinterpret_cast<volatile int*>(state_full + 2);
  // per column of v of the item, for four items in turn: the request's first token from which o and the
  // state are NaN (three chunks are under way at most, so four items with chunks)
  int* spoilt = reinterpret_cast<int*>(state_full + 3);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // the requests with the most chunks first, so that what comes last is short; each lane ranks two
  int rank[2] = {0, 0};
  if (a.B <= 64) {
    int mine[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) mine[e] = lane + 32 * e < a.B ? (int)chunks_of(a, lane + 32 * e) : -1;
    for (int i = 0; i < a.B; ++i) {
      const int other = __shfl_sync(0xffffffffu, i < 32 ? mine[0] : mine[1], i & 31);
#pragma unroll
      for (int e = 0; e < 2; ++e) rank[e] += other > mine[e] || (other == mine[e] && i < lane + 32 * e);
    }
  }
  const ChunkScan sc = chunk_scan(a, lane);
  const bool crowded = __shfl_sync(0xffffffffu, sc.upto, 31) > chunk_room(a);
  // the i-th item of this CTA: a request, a value head and half of its columns; CTAs take turns back and
  // forth.  False: no more.
  struct Item {
    int b, h, slice, nc;
    int64_t t0, len;
  };
  auto item_at = [&](int i, Item& it) {
    const int64_t k = (int64_t)i * gridDim.x + ((i & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
    const int64_t r = k / (a.Hv * kD2Slices);
    const int rest = (int)(k - r * (a.Hv * kD2Slices));
    it.h = rest / kD2Slices;
    it.slice = rest - it.h * kD2Slices;
    it.b = (int)r;
    if (r >= a.B) return false;
    if (a.B <= 64) {
      const unsigned w0 = __ballot_sync(0xffffffffu, lane < a.B && rank[0] == it.b);
      const unsigned w1 = __ballot_sync(0xffffffffu, lane + 32 < a.B && rank[1] == it.b);
      it.b = w0 ? __ffs(w0) - 1 : __ffs(w1) + 31;
    }
    if (!delta_rows(a, it.b, it.t0, it.len)) {
      if (tid == 0 && rest == 0) set_status(a.status, TB_DEV_BAD_LEN);
      it.len = 0;
    }
    it.nc = (int)((it.len + kDcTok - 1) / kDcTok);
    if (crowded && first_chunk(a, sc, it.b, lane) + it.nc > chunk_room(a)) {
      if (tid == 0 && rest == 0) set_status(a.status, TB_DEV_BAD_LEN);
      it.len = it.nc = 0;
    }
    return true;
  };
  for (int i = tid; i < 256; i += kD2Threads) spoilt[i] = INT_MAX;
  if (tid == 0) {
    *aborted = 0;
    for (int i = 0; i < kD2Stages; ++i) {
      mbar_init(full + i, 1);
      mbar_init(ready + i, 1);
      mbar_init(empty + i, kD2Warps);
    }
    mbar_init(state_full, 1);
    mbar_init(state_empty, kD2Warps);
    fence_barrier_init();
  }
  __syncthreads();
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity) || *aborted) return;
    if (!mbar_wait(bar, parity)) {
      *aborted = 1;
      set_status(a.status, TB_DEV_TIMEOUT);
    }
  };

  if (warp == kD2Warps) {
    int loaded = 0, looked = 0, states = 0;  // chunks of all items; states
    auto load = [&](const Item& it, int64_t first, int c) {  // a lane per copy
      const int s = loaded % kD2Stages, row = (int)it.t0 + c * kDcTok;
      const int h = it.h, hk = h / (a.Hv / a.Hk), slice = it.slice;
      const uint32_t sa = base + s * kD2Stage, bar = smem_u32(full + s);
      if (loaded >= kD2Stages) wait(empty + s, (loaded / kD2Stages - 1) & 1);
      if (lane == 0) {
        mbar_arrive_expect_tx(full + s, kD2Bytes);
        if (loaded == 0) asm volatile("griddepcontrol.wait;" ::: "memory");  // kernel 1's results
        bulk_g2s(smem + s * kD2Stage + kD2Item, p.ws + ((first + c) * a.Hv + h) * (int64_t)kDcItem, kDcItem, full + s);
      } else if (lane < 6) {
        const int d = (lane - 1) & 1;
        const CUtensorMap* tm = lane == 5 ? &tmV : (lane >= 3 ? &tmQ : &tmK);
        const uint32_t dst = sa + (lane == 5 ? kD2V : (lane >= 3 ? kD2Q : 0) + d * kDcBlock);
        tma_load_3d<1>(dst, tm, (lane == 5 ? slice : d) * 64, lane == 5 ? h : hk, row, bar);
      }
      __syncwarp();
      ++loaded;
    };
    auto load_state = [&](const Item& it, int64_t slot) {  // once the walking warps have taken up the last one
      if (states > 0) wait(state_empty, (states - 1) & 1);
      ++states;
      if (lane == 0) mbar_arrive_expect_tx(state_full, kDeltaD * 256);
      __syncwarp();
      const float* src = a.state_in + (slot * a.Hv + it.h) * (int64_t)(kDeltaD * kDeltaD) + it.slice * 64;
#pragma unroll
      for (int r = lane; r < kDeltaD; r += 32)
        bulk_g2s(smem + kD2Stages * kD2Stage + r * kD2StatePitch, src + r * kDeltaD, 256, state_full);
    };
    // What must not meet the zeros of T or of the sums over the tokens is taken out of the stage before the
    // others see it, and noted: tokens of another request behind the last one, tokens from one on whose k,
    // decay or step is not finite, and a v that is not.
    auto look_over = [&](int64_t len, int* spoilt, int c) {
      const int s = looked % kD2Stages;
      const uint32_t st = base + s * kD2Stage;
      wait(full + s, (looked / kD2Stages) & 1);
      ++looked;
      const int left = (int)(len - (int64_t)c * kDcTok < kDcTok ? len - (int64_t)c * kDcTok : kDcTok);
      const int sound = (int)reinterpret_cast<const float*>(smem + s * kD2Stage + kD2Item + kDcFactors)[193];
      const int ok = min(left, sound);
      if (ok < left)
        for (int i = lane; i < 64; i += 32) atomicMin(spoilt + i, c * kDcTok + ok);
      if (ok < kDcTok) {
        for (int i = lane; i < (kDcTok - ok) * 24; i += 32) {  // 16-byte pieces: 16 of K, 8 of V a row
          const int r = ok + i / 24, x = i % 24;
          asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(st + (x < 16 ? (x >> 3) * kDcBlock : kD2V) + r * 128 +
                                                                     (x & 7) * 16),
                       "r"(0)
                       : "memory");
        }
        __syncwarp();
      }
      __half2 odd[2] = {__half2half2(__ushort_as_half(0)), __half2half2(__ushort_as_half(0))};  // 0 times what is not finite is NaN
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        uint4 w = ld_shared_v4(st + kD2V + (i * 32 + lane) * 16);
        const __half2* hv = reinterpret_cast<const __half2*>(&w);
#pragma unroll
        for (int e = 0; e < 4; ++e) odd[e & 1] = __hfma2(hv[e], __half2half2(__ushort_as_half(0)), odd[e & 1]);
      }
      odd[0] = __hadd2(odd[0], odd[1]);
      if (__any_sync(0xffffffffu, __hisnan(__low2half(odd[0])) || __hisnan(__high2half(odd[0])))) {
        for (int i = lane; i < kDcTok * 64; i += 32) {
          const int r = i >> 6, col = i & 63;
          __half* v = reinterpret_cast<__half*>(smem + s * kD2Stage + kD2V + r * 128 + (((col >> 3) ^ (r & 7)) << 4)) + (col & 7);
          if ((__half_as_ushort(*v) & 0x7c00u) == 0x7c00u) {
            atomicMin(spoilt + col, c * kDcTok + r);
            *v = __ushort_as_half(0);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(ready + s);
    };
    // a chunk's copies go out before the last one's are looked over, also from one item to the next
    Item it;
    int64_t last_len = 0;
    int last_c = -1, seg = 0;
    int* last_spoilt = spoilt;
    for (int i = 0; item_at(i, it); ++i) {
      if (it.nc == 0) continue;
      const int64_t first = first_chunk(a, sc, it.b, lane);
      for (int c = 0; c < it.nc; ++c) {
        const int64_t si = c == 0 && a.state_in ? delta_slot(a.slot_in, it.b, a.n_in, a.status) : -1;
        const bool first_state = si >= 0 && states == 0;
        if (first_state) load_state(it, si);  // (does not wait for kernel 1)
        load(it, first, c);
        if (last_c >= 0) look_over(last_len, last_spoilt, last_c);
        if (si >= 0 && !first_state) load_state(it, si);
        last_c = c;
        last_len = it.len;
        last_spoilt = spoilt + (seg & 3) * 64;
      }
      ++seg;
    }
    if (last_c >= 0) look_over(last_len, last_spoilt, last_c);
    if (*aborted) {  // a wait gave up: leave the copies in flight time to land before the CTA ends
      const uint64_t t = globaltimer_ns();
      while (globaltimer_ns() - t < 1000000) {
      }
    }
    return;
  }

  const int g = lane >> 2, t2 = (lane & 3) * 2;
  // addresses of the ldmatrix lanes inside a 64 x 64 image: rows by the lane, a 16-byte piece per k
  const uint32_t sw = (uint32_t)lane & 7u;
  const uint32_t row_n = (((uint32_t)lane & 7u) + ((uint32_t)lane >> 4) * 8u) * 128u;  // rows are n
  const uint32_t row_k = ((uint32_t)lane & 15u) * 128u;                                // rows are k
  const uint32_t pc_n = ((uint32_t)lane >> 3) & 1u, pc_k = (uint32_t)lane >> 4;
  const uint32_t v_row = ((((uint32_t)lane >> 4) & 1u) * 8u + sw) * 128u;
  const uint32_t v_pc = (((uint32_t)warp * 2u + pc_n) ^ sw) << 4;

  int done = 0, seg = 0, states = 0;  // chunks of all items, items with chunks, states of those
  Item it;
  for (int i = 0; item_at(i, it); ++i) {
    const int h = it.h, nc = it.nc;
    const int64_t t0 = it.t0, len = it.len, head_size = (int64_t)a.Hv * kDeltaD * kDeltaD;
    const int col = (it.slice * kD2Warps + warp) * 16;  // the warp's first column of v
    int* mine = spoilt + (seg & 3) * 64 + warp * 16;
    const int64_t si = delta_slot(a.slot_in, it.b, a.n_in, a.status);
    const bool have = a.state_in && si >= 0;
    if (nc == 0) {  // no tokens: the state goes through
      const int64_t so = delta_slot(a.slot_out, it.b, a.n_out, a.status);
      if (a.state_out && so >= 0) {
        const int64_t at = (int64_t)h * kDeltaD * kDeltaD + col + (lane & 3) * 4;
        for (int k = lane >> 2; k < kDeltaD; k += 8) {
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
          if (have) x = *reinterpret_cast<const float4*>(a.state_in + si * head_size + at + k * kDeltaD);
          *reinterpret_cast<float4*>(a.state_out + so * head_size + at + k * kDeltaD) = x;
        }
      }
      continue;
    }
    // S^T: rows g, g + 8 (columns of v), columns 8 j + t2, + 1 (of k)
    float S[16][4];
    if (have) wait(state_full, states++ & 1);
    {
      const uint8_t* src = smem + kD2Stages * kD2Stage + t2 * kD2StatePitch + (warp * 16 + g) * 4;
#pragma unroll
      for (int j = 0; j < 16; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          S[j][e] = have ? *reinterpret_cast<const float*>(src + (j * 8 + (e & 1)) * kD2StatePitch + (e >> 1) * 32) : 0.f;
    }
    float sbig[2] = {0.f, 0.f};  // the largest |S|, two chains of it
#pragma unroll
    for (int j = 0; j < 16; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (!(fabsf(S[j][e]) < INFINITY)) {  // a column that is NaN from the start
          atomicMin(&mine[g + (e >> 1) * 8], 0);
          S[j][e] = 0.f;
        }
        sbig[e / 2] = fmaxf(sbig[e / 2], fabsf(S[j][e]));
      }
    if (have) {
      fence_proxy_async_smem();  // the reads above before the next state's copy
      __syncwarp();
      if (lane == 0) mbar_arrive_reads(state_empty);
    }
    __half* dst = a.o + ((t0 + g) * a.Hv + h) * kDeltaD + col + t2;
    for (int left = (int)len; left > 0; left -= kDcTok) {  // tokens
      const int s = done % kD2Stages;
      const uint32_t K = base + s * kD2Stage, Q = K + kD2Q, X = K + kD2Item, V = K + kD2V;
      auto factors = [&](int at) { return lds2(X + kDcFactors + (at + t2) * 4); };  // of two tokens
      float down_s;
      const float up_s = operand_scale(sbig, down_s);
      wait(ready + s, (done / kD2Stages) & 1);
      ++done;
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
        split2(S[2 * ks + (q >> 1)] + (q & 1) * 2, up_s, sh[ks][q], lo[ks & 1][q]);
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
      // S^T q, and beside it R = v - exp(gamma) S^T k
      float big[2] = {0.f, 0.f};
      uint32_t vv[4];
      ldsm4_trans(V + v_row + v_pc, vv);
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        const float2 cc = factors(ks * 8);
        const float2 cn = mul_f32x2(cc, make_float2(-down_s, -down_s));
        auto residual = [&](int q) {  // columns of v g + 8 q
          const float2 w = __half22float2(*reinterpret_cast<const __half2*>(&vv[(ks & 1) * 2 + q]));
          float* x = R[ks] + q * 2;
          const float2 r = fma_f32x2(cn, make_float2(x[0], x[1]), w);
          x[0] = r.x;
          x[1] = r.y;
          big[q] = max3_abs(big[q], r.x, r.y);
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
      const float up_p = lds2(X + kDcFactors + 194 * 4).x;
      float down_r;
      const float up_r = operand_scale(big, down_r, min((int)(__float_as_uint(up_s) >> 23) + kDcPScale, 127 + 100));
      uint32_t rh[4][4], rl[4][4];
      auto split_r = [&](int ks, int q) {
        split2(R[2 * ks + (q >> 1)] + (q & 1) * 2, up_r, rh[ks][q], rl[ks][q]);
      };
#pragma unroll
      for (int q = 0; q < 4; ++q) split_r(0, q);
      // U = T R and o += P T R (rows past a token do not reach it: their blocks are left out), a block of
      // T and one of P T at a time, so that no MMA waits for one of the last three; w U as its rows are done
      float U[8][4];
#pragma unroll
      for (int nt = 0; nt < 8; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) U[nt][e] = 0.f;
      auto frag = [&](int matrix, int ks, int j, uint32_t (&r)[4]) {
        lds4(X + matrix * kDcMatrix + (j * (j + 1) / 2 + ks) * kDcFrag + lane * 16, r);
      };
      auto scale_o = [&](int j) {  // o's first part to R's scale
        const float2 qq = factors(128 + j * 8);
        const float2 qs = mul_f32x2(qq, make_float2(down_s * up_r, down_s * up_r));
        mul_pair(O[j], qs);
        mul_pair(O[j] + 2, qs);
      };
      big[0] = big[1] = 0.f;
      auto weigh = [&](int j) {
        const float2 ww = factors(64 + j * 8);
        const float2 ws = mul_f32x2(ww, make_float2(down_r, down_r));
        mul_pair(U[j], ws);
        mul_pair(U[j] + 2, ws);
        big[0] = max3_abs(big[0], U[j][0], U[j][1]);
        big[1] = max3_abs(big[1], U[j][2], U[j][3]);
      };
      constexpr int kAt[10][2] = {{0, 0}, {0, 1}, {0, 2}, {0, 3}, {1, 1}, {1, 2}, {1, 3}, {2, 2}, {2, 3}, {3, 3}};
      uint32_t th[2][4], tl[2][4], pt[2][4];
      frag(0, 0, 0, th[0]);
      frag(1, 0, 0, pt[0]);
      frag(2, 0, 0, tl[0]);
      scale_o(0);
      scale_o(1);
#pragma unroll
      for (int i = 0; i < 10; ++i) {
        const int ks = kAt[i][0], j = kAt[i][1], x = i & 1;
        if (i < 9) {
          frag(0, kAt[i + 1][0], kAt[i + 1][1], th[x ^ 1]);
          frag(1, kAt[i + 1][0], kAt[i + 1][1], pt[x ^ 1]);
          frag(2, kAt[i + 1][0], kAt[i + 1][1], tl[x ^ 1]);
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
        mma_16816(O[2 * j], rh[ks], pt[x][0], pt[x][1]);
        mma_16816(O[2 * j + 1], rh[ks], pt[x][2], pt[x][3]);
        if (i < 3) scale_o(2 * i + 2);
        mma_16816(U[2 * j], rl[ks], th[x][0], th[x][1]);
        mma_16816(U[2 * j + 1], rl[ks], th[x][2], th[x][3]);
        if (i < 3) scale_o(2 * i + 3);
        if (i == 1 || i == 5 || i == 8) weigh(i == 1 ? 0 : (i == 5 ? 2 : 4));
        mma_16816(O[2 * j], rl[ks], pt[x][0], pt[x][1]);
        mma_16816(O[2 * j + 1], rl[ks], pt[x][2], pt[x][3]);
        if (i == 1 || i == 5 || i == 8) weigh(i == 1 ? 1 : (i == 5 ? 3 : 5));
        mma_16816(U[2 * j], rh[ks], tl[x][0], tl[x][1]);
        mma_16816(U[2 * j + 1], rh[ks], tl[x][2], tl[x][3]);
      }
      weigh(6);
      weigh(7);
      const float down_o = up_p * down_r;
      float down_u;
      const float up_u = operand_scale(big, down_u);
      auto split_u = [&](int ks, int q) {
        split2(U[2 * ks + (q >> 1)] + (q & 1) * 2, up_u, rh[ks][q], rl[ks][q]);
      };
#pragma unroll
      for (int q = 0; q < 4; ++q) split_u(0, q);
      // S <- exp(gamma_C) S + K^T (w U); the increment is summed by itself, so that the state's own
      // rounding is one fp32 fma a chunk.  Beside it o goes out, back in rows of tokens.
      const float dec = lds2(X + kDcFactors + 192 * 4).x;
      sbig[0] = sbig[1] = 0.f;
      auto at_k = [&](int i) {  // step i: 16 columns i / 4 of k, 16 tokens i % 4
        const int j = i >> 2;
        return K + (j >> 2) * kDcBlock + row_k + (((uint32_t)(j & 3) * 2u + pc_k) ^ sw) * 16u + (i & 3) * 2048;
      };
      uint32_t kt[2][4];
      ldsm4_trans(at_k(0), kt[0]);
      float dh[2][2][4], dl[2][2][4];  // of two steps: one is summed up while the next one's MMAs run
      auto add_up = [&](int j, int x) {
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          float* y = S[2 * j + x] + e;
          const float *h = dh[j & 1][x] + e, *l = dl[j & 1][x] + e;
          const float2 d = add_f32x2(make_float2(h[0], h[1]), make_float2(l[0], l[1]));
          const float2 r = fma_f32x2(make_float2(dec, dec), make_float2(y[0], y[1]), mul_f32x2(d, make_float2(down_u, down_u)));
          y[0] = r.x;
          y[1] = r.y;
          sbig[e / 2] = max3_abs(sbig[e / 2], r.x, r.y);
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
          if (ks == 0) {
            mul_pair(O[j], make_float2(down_o, down_o));
            ox = transpose8x8(pack_half2(O[j][0], O[j][1]));
          }
          if (ks == 1) {
            mul_pair(O[j] + 2, make_float2(down_o, down_o));
            oy = transpose8x8(pack_half2(O[j][2], O[j][3]));
          }
          mma_16816(dl[z][1], rl[ks], kt[x][2], kt[x][3]);
        }
        if (j * 8 + g < left) {
          *reinterpret_cast<uint32_t*>(dst) = ox;
          *reinterpret_cast<uint32_t*>(dst + 8) = oy;
        }
        dst += (int64_t)8 * a.Hv * kDeltaD;
      }
      add_up(7, 0);
      add_up(7, 1);
      fence_proxy_async_smem();  // this warp's reads before the copy that refills the stage
      __syncwarp();
      if (lane == 0) mbar_arrive_reads(empty + s);
    }
    const int64_t so = delta_slot(a.slot_out, it.b, a.n_out, a.status);
    if (a.state_out && so >= 0) {
      float* dst = a.state_out + so * head_size + ((int64_t)h * kDeltaD + t2) * kDeltaD + col + g;
#pragma unroll
      for (int j = 0; j < 16; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) dst[(j * 8 + (e & 1)) * kDeltaD + (e >> 1) * 8] = S[j][e];
    }
    ++seg;
    // what is NaN (rarely anything), over what this warp wrote there
    __syncwarp();
    const int from = lane < 16 ? mine[lane] : INT_MAX;
    for (unsigned who = __ballot_sync(0xffffffffu, from != INT_MAX); who; who &= who - 1) {
      const int x = __ffs(who) - 1, at = __shfl_sync(0xffffffffu, from, x);
      for (int64_t t = at + lane; t < len; t += 32) a.o[((t0 + t) * a.Hv + h) * kDeltaD + col + x] = __float2half_rn(NAN);
      if (a.state_out && so >= 0)
        for (int k = lane; k < kDeltaD; k += 32) a.state_out[so * head_size + ((int64_t)h * kDeltaD + k) * kDeltaD + col + x] = NAN;
    }
    if (from != INT_MAX) mine[lane] = INT_MAX;  // (for the item after the next three)
    __syncwarp();
  }
}

static int launch_scan(const ChunkArgs& p, const DeviceFacts& f, cudaStream_t s) {
  const DeltaArgs& a = p.a;
  CUtensorMap tk, tq, tv;
  int rc = token_map(&tk, a.k, a.T, a.Hk, kDeltaD, a.ldk, 1, kDcTok);
  if (rc == TB_OK) rc = token_map(&tq, a.q, a.T, a.Hk, kDeltaD, a.ldq, 1, kDcTok);
  if (rc == TB_OK) rc = token_map(&tv, a.v, a.T, a.Hv, kDeltaD, a.ldv, 1, kDcTok);
  if (rc == TB_OK) rc = ensure_dynamic_smem(reinterpret_cast<const void*>(delta_scan_kernel), f.device, kD2Smem);
  if (rc != TB_OK) return rc;
  cudaLaunchConfig_t cfg = {};
  const int64_t items = (int64_t)a.B * a.Hv * kD2Slices;
  cfg.gridDim = dim3((unsigned)(items < f.sms ? items : f.sms));
  cfg.blockDim = dim3(kD2Threads);
  cfg.dynamicSmemBytes = kD2Smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, delta_scan_kernel, tk, tq, tv, p);
  if (e != cudaSuccess) {
    record_cuda_error(e);
    return TB_ERR_CUDA;
  }
  return check_launch();
}

size_t delta_chunk_workspace(int64_t T, int64_t B, int64_t Hv) {
  return (size_t)((T / kDcTok + B) * Hv) * kDcItem;  // chunk_room() of them
}

int launch_delta_chunks(const DeltaArgs& a, void* workspace, cudaStream_t s) {
  DeviceFacts f;
  int rc = device_facts(&f);
  if (rc != TB_OK) return rc;
  ChunkArgs p;
  p.a = a;
  p.ws = static_cast<uint8_t*>(workspace);
  const int64_t prep = (a.T / kDcTok + a.B) * a.Hk, heads = (int64_t)a.B * a.Hv;
  if (prep > INT32_MAX || heads > INT32_MAX / kD2Slices) return TB_ERR_TOO_LARGE;
  delta_prep_kernel<<<(unsigned)prep, kD1Threads, 0, s>>>(p);
  rc = check_launch();
  if (rc != TB_OK) return rc;
  return launch_scan(p, f, s);
}

}  // namespace tb
