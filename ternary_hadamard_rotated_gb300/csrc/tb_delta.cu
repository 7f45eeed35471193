// The gated delta rule: the mixer of the hybrid model's linear-attention layers ([ARCH]: 16 key
// heads and 48 value heads of 128, an fp32 state).  Per value head, with S a 128 x 128 state,
//   S <- exp(g_t) S;   u = beta_t (v_t - S^T k_t);   S <- S + k_t u^T;   o_t = scale S^T q_t.
//
// Recurrent form (few tokens per request).  A CTA keeps a slice of the state in registers for all
// tokens of its request.  One pass over the slice per token gives both S^T k and S^T q, since
//   o = scale (e^g S^T q + (k . q) u)       with S before the token,
// so a token costs one reduction over the state's rows and one CTA barrier.
// One token for each of 64 requests, 48 heads (405 MB, the states read and written once): 64.3 us, 6300 GB/s,
// 0.93 of measured HBM, in a replayed graph, 66.9 us a call.  One request: 3.7 us; each further token 1.25 us.
#include <cuda_runtime.h>
#include <math.h>

#include "tb_common.cuh"
#include "tb_delta.cuh"
#include "tb_host.h"

namespace tb {

constexpr int kDlThreads = 256;

// COLS columns of v per CTA: 256 threads as (COLS / 4) column quads x row groups; row group r holds
// rows r, r + RG, ...; the row groups of one warp are summed by shuffles, the 8 warps through
// shared memory.
template <int COLS>
__global__ void __launch_bounds__(kDlThreads) delta_step_kernel(const DeltaArgs a) {
  constexpr int Q = COLS / 4;            // column quads
  constexpr int RG = kDlThreads / Q;     // row groups
  constexpr int R = kDeltaD / RG;        // rows per thread
  __shared__ float4 kq[3][2][kDeltaD / 4];      // k and q of a token, normalised and scaled
  __shared__ float vv[3][COLS];
  __shared__ float scal[3][4];                  // e^g, beta, k . q
  __shared__ float4 part[2][2][kDlThreads / 32][Q];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int quad = tid % Q, rg = tid / Q;
  const int slices = kDeltaD / COLS;
  const int slice = (int)(blockIdx.x % slices);
  const int64_t bh = blockIdx.x / slices;
  const int h = (int)(bh % a.Hv), b = (int)(bh / a.Hv);
  const int hk = h / (a.Hv / a.Hk);
  int64_t t0, n;
  if (!delta_rows(a, b, t0, n)) {
    if (tid == 0 && h == 0 && slice == 0) set_status(a.status, TB_DEV_BAD_LEN);
    n = 0;
  }
  const int64_t si = delta_slot(a.slot_in, b, a.n_in, a.status), so = delta_slot(a.slot_out, b, a.n_out, a.status);
  const int c0 = slice * COLS + quad * 4;

  float4 S[R];
  if (a.state_in && si >= 0) {
    const float* src = a.state_in + (si * a.Hv + h) * (int64_t)(kDeltaD * kDeltaD) + c0;
#pragma unroll
    for (int i = 0; i < R; ++i) S[i] = __ldcs(reinterpret_cast<const float4*>(src + (rg + RG * i) * kDeltaD));
  } else {
#pragma unroll
    for (int i = 0; i < R; ++i) S[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }

  // warp 0 carries k and q of a token (four elements of each per lane), warp 1 v and the scalars
  float4 nk, nq;
  float nv[COLS / 32], ng = 0.f, nb = 0.f;
  auto fetch = [&](int64_t t) {
    if (warp == 0) {
      nk = load_half4(a.k + (t0 + t) * a.ldk + hk * kDeltaD + lane * 4);
      nq = load_half4(a.q + (t0 + t) * a.ldq + hk * kDeltaD + lane * 4);
    } else if (warp == 1) {
#pragma unroll
      for (int i = 0; i < COLS / 32; ++i)
        nv[i] = __half2float(a.v[(t0 + t) * a.ldv + h * kDeltaD + slice * COLS + i * 32 + lane]);
      ng = a.g[(t0 + t) * a.Hv + h];
      nb = a.beta[(t0 + t) * a.Hv + h];
    }
  };
  auto publish = [&](int buf) {
    if (warp == 0) {
      float kk = dot4(nk, nk), qq = dot4(nq, nq), kq_ = dot4(nk, nq);
#pragma unroll
      for (int d = 16; d; d >>= 1) {
        kk += __shfl_xor_sync(0xffffffffu, kk, d);
        qq += __shfl_xor_sync(0xffffffffu, qq, d);
        kq_ += __shfl_xor_sync(0xffffffffu, kq_, d);
      }
      const float rk = a.normalise ? 1.f / sqrtf(kk + kDeltaEps) : 1.f;
      const float rq = a.normalise ? a.scale / sqrtf(qq + kDeltaEps) : a.scale;
      kq[buf][0][lane] = make_float4(nk.x * rk, nk.y * rk, nk.z * rk, nk.w * rk);
      kq[buf][1][lane] = make_float4(nq.x * rq, nq.y * rq, nq.z * rq, nq.w * rq);
      if (lane == 0) scal[buf][2] = kq_ * rk * rq;
    } else if (warp == 1) {
#pragma unroll
      for (int i = 0; i < COLS / 32; ++i) vv[buf][i * 32 + lane] = nv[i];
      if (lane == 0) {
        scal[buf][0] = expf(ng);
        scal[buf][1] = nb;
      }
    }
  };

  if (n > 0) {
    fetch(0);
    publish(0);
    if (n > 1) fetch(1);
  }
  __syncthreads();
  for (int64_t t = 0; t < n; ++t) {
    // token t + 1 goes to the third buffer: its readers of two tokens ago are behind a barrier
    const int buf = (int)(t % 3), pb = (int)(t & 1);
    const float* kr = reinterpret_cast<const float*>(kq[buf][0]);
    const float* qr = reinterpret_cast<const float*>(kq[buf][1]);
    float4 sk = make_float4(0.f, 0.f, 0.f, 0.f), sq = sk;
    float kk[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      kk[i] = kr[rg + RG * i];
      const float qv = qr[rg + RG * i];
      fma4(sk, kk[i], S[i]);
      fma4(sq, qv, S[i]);
    }
    if (Q < 32) {
#pragma unroll
      for (int d = Q; d < 32; d <<= 1) {
        add4_xor(sk, d);
        add4_xor(sq, d);
      }
    }
    if (lane < Q) {
      part[pb][0][warp][lane] = sk;
      part[pb][1][warp][lane] = sq;
    }
    if (t + 1 < n) {
      publish((int)((t + 1) % 3));
      if (t + 2 < n) fetch(t + 2);
    }
    __syncthreads();
    const float eg = scal[buf][0], be = scal[buf][1];
    sk = part[pb][0][0][quad];
#pragma unroll
    for (int w = 1; w < kDlThreads / 32; ++w) add4(sk, part[pb][0][w][quad]);
    const float4 v4 = *reinterpret_cast<const float4*>(&vv[buf][quad * 4]);
    const float4 u = make_float4(be * (v4.x - eg * sk.x), be * (v4.y - eg * sk.y), be * (v4.z - eg * sk.z),
                                 be * (v4.w - eg * sk.w));
    if (rg == 0) {
      sq = part[pb][1][0][quad];
#pragma unroll
      for (int w = 1; w < kDlThreads / 32; ++w) add4(sq, part[pb][1][w][quad]);
      const float d = scal[buf][2];
      uint2 o;
      o.x = pack_half2(eg * sq.x + d * u.x, eg * sq.y + d * u.y);
      o.y = pack_half2(eg * sq.z + d * u.z, eg * sq.w + d * u.w);
      *reinterpret_cast<uint2*>(a.o + ((t0 + t) * a.Hv + h) * kDeltaD + c0) = o;
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      S[i].x = fmaf(eg, S[i].x, kk[i] * u.x);
      S[i].y = fmaf(eg, S[i].y, kk[i] * u.y);
      S[i].z = fmaf(eg, S[i].z, kk[i] * u.z);
      S[i].w = fmaf(eg, S[i].w, kk[i] * u.w);
    }
  }
  if (a.state_out && so >= 0) {
    float* dst = a.state_out + (so * a.Hv + h) * (int64_t)(kDeltaD * kDeltaD) + c0;
#pragma unroll
    for (int i = 0; i < R; ++i) __stcs(reinterpret_cast<float4*>(dst + (rg + RG * i) * kDeltaD), S[i]);
  }
}

}  // namespace tb

extern "C" size_t tb_gated_delta_workspace_size(int64_t T, int64_t B, int64_t max_len, int64_t Hk, int64_t Hv) {
  (void)Hk;
  if (T < 1 || B < 1 || Hv < 1 || max_len <= tb::kDeltaStepTokens) return 0;
  return tb::delta_chunk_workspace(T, B, Hv);
}

extern "C" int tb_gated_delta(const uint16_t* q, int64_t ldq, const uint16_t* k, int64_t ldk, const uint16_t* v,
                              int64_t ldv, const float* g, const float* beta, int64_t T, int64_t Hk, int64_t Hv,
                              int64_t D, const int32_t* row_start, int64_t B, int64_t max_len, int normalise,
                              float scale, const float* state_in, const int32_t* slot_in, int64_t n_in,
                              float* state_out, const int32_t* slot_out, int64_t n_out, uint16_t* o,
                              void* workspace, size_t workspace_bytes, int32_t* dev_status, void* stream) {
  using namespace tb;
  if (T < 0 || T > INT32_MAX || B < 1 || B > INT32_MAX || Hk < 1 || Hv < Hk || Hv > 1024 || Hv % Hk || max_len < 0)
    return TB_ERR_SHAPE;
  if (D != kDeltaD) return TB_ERR_UNSUPPORTED;
  if (ldq < Hk * D || ldk < Hk * D || ldv < Hv * D || ldq % 8 || ldk % 8 || ldv % 8 || ldq > 1ll << 31 ||
      ldk > 1ll << 31 || ldv > 1ll << 31)
    return TB_ERR_SHAPE;
  if ((state_in && (n_in < 1 || (!slot_in && n_in < B))) || (state_out && (n_out < 1 || (!slot_out && n_out < B))))
    return TB_ERR_SHAPE;
  if (!(scale > -INFINITY && scale < INFINITY)) return TB_ERR_VALUE;
  if (!row_start || (T && (!q || !k || !v || !g || !beta || !o))) return TB_ERR_NULL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned_to(g, 4) || !aligned_to(beta, 4) ||
      !aligned16(o) || !aligned_to(row_start, 4) || !aligned16(state_in) || !aligned16(state_out) ||
      !aligned_to(slot_in, 4) || !aligned_to(slot_out, 4) || !aligned16(workspace))
    return TB_ERR_ALIGN;
  if (max_len > kDeltaStepTokens && T && !workspace) return TB_ERR_WORKSPACE;
  if (workspace_bytes < tb_gated_delta_workspace_size(T, B, max_len, Hk, Hv)) return TB_ERR_WORKSPACE;
  DeviceFacts f;
  int rc = device_facts(&f);
  if (rc != TB_OK) return rc;
  DeltaArgs a;
  a.q = reinterpret_cast<const __half*>(q);
  a.k = reinterpret_cast<const __half*>(k);
  a.v = reinterpret_cast<const __half*>(v);
  a.g = g;
  a.beta = beta;
  a.row_start = row_start;
  a.state_in = state_in;
  a.state_out = state_out;
  a.slot_in = slot_in;
  a.slot_out = slot_out;
  a.o = reinterpret_cast<__half*>(o);
  a.status = dev_status;
  a.ldq = ldq;
  a.ldk = ldk;
  a.ldv = ldv;
  a.n_in = n_in;
  a.n_out = n_out;
  a.T = T;
  a.B = (int)B;
  a.Hk = (int)Hk;
  a.Hv = (int)Hv;
  a.normalise = normalise;
  a.scale = scale;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t heads = B * Hv;
  if (heads * 4 > INT32_MAX) return TB_ERR_TOO_LARGE;
  if (max_len > kDeltaStepTokens && T) return launch_delta_chunks(a, workspace, s);
  // whole heads per CTA once they fill the SMs twice over; below that a quarter of a head each, which
  // spreads one request's 48 heads over all SMs
  if (heads >= 2 * f.sms) delta_step_kernel<128><<<(int)heads, kDlThreads, 0, s>>>(a);
  else delta_step_kernel<32><<<(int)(heads * 4), kDlThreads, 0, s>>>(a);
  return check_launch();
}
