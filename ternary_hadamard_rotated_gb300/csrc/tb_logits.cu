// Changes to the logits before a token is chosen: penalties for tokens that a request's history holds, biases,
// and grammar masks.
//
// Per row and token, in this order, in fp32 with every step rounded as written (no product joined to a sum, so
// that the same formulas give the same bits anywhere):
//   l <- l > 0 ? l / repetition : l * repetition   if the token is in the history (or among the row's drafts)
//   l <- l - frequency * count - presence          if it was generated, count times
//   l <- l + bias                                  if it has one
//   l <- -infinity                                 if its bit of the mask is 0
#include <cuda_runtime.h>
#include <limits.h>
#include <stddef.h>

#include "tb_common.cuh"
#include "tb_host.h"

namespace tb {

// Two launches.  The first moves all rows from in to out under their masks, in whole sectors, next rows' logits on their
// way while the present ones are stored (not launched in place and without a mask, where nothing would change).  The
// second (programmatic: it begins beside the first) counts the requests' tokens in hash tables in shared memory and works
// out the few that have a count or a bias, for all rows of their request; it waits for the first before it stores them.
struct LogitsArgs {
  const __half* in;
  void* out;
  const int32_t *row_start, *history, *slot, *hist_len, *prompt_len, *fresh;
  const unsigned long long* tree;
  const float *repetition, *presence, *frequency;
  const int32_t *bias_start, *bias_ids;
  const float* bias_values;
  const uint32_t* mask;
  const int32_t* mask_row;
  int32_t* status;
  int64_t ld, ldo, ldh, n_hist, n_bias, mask_rows;
  int T, V, B;
  int chunks;      // of a row, of kMoveChunk tokens
  int parts_log2, part_tokens;  // a request's tokens are shared out to at most so many CTAs, of about so many each
};

// ---------------------------------------------------------------- moving
// `have` of E logits of a row, one at a time
template <int E>
TB_DEVI void load_some(uint32_t (&v)[E / 2], const __half* p, int have) {
  const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
  for (int j = 0; j < E / 2; ++j) v[j] = (2 * j < have ? h[2 * j] : 0u) | (2 * j + 1 < have ? (uint32_t)h[2 * j + 1] << 16 : 0u);
}
// minus infinity where the mask's bit is 0
template <int E>
TB_DEVI void mask_logits(uint32_t (&v)[E / 2], uint32_t allowed) {
#pragma unroll
  for (int j = 0; j < E / 2; ++j) {
    const uint32_t keep = (allowed >> 2 * j & 1 ? 0xffffu : 0u) | (allowed >> 2 * j & 2 ? 0xffff0000u : 0u);
    v[j] = lop3_and_or(v[j], keep, 0xfc00fc00u & ~keep);
  }
}
template <int E>
TB_DEVI void store_logits(__half* p, const uint32_t (&v)[E / 2]) {
  __stcs(reinterpret_cast<uint4*>(p), make_uint4(v[0], v[1], v[2], v[3]));
}
template <int E>
TB_DEVI void store_logits(float* p, const uint32_t (&v)[E / 2]) {
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&v[0])), b = __half22float2(*reinterpret_cast<const __half2*>(&v[1]));
  __stcs(reinterpret_cast<float4*>(p), make_float4(a.x, a.y, b.x, b.y));
}
TB_DEVI void store_logit(__half* p, float v) { *p = __float2half_rn(v); }
TB_DEVI void store_logit(float* p, float v) { *p = v; }
template <int E, typename Out>
TB_DEVI void store_some(Out* p, const uint32_t (&v)[E / 2], int have) {
#pragma unroll
  for (int j = 0; j < E; ++j)
    if (j < have) store_logit(p + j, half_bits_to_float((uint16_t)(v[j / 2] >> (j & 1) * 16)));
}

// Whether a row is one of a request's.  A request counts where no row start before it is above its own and it ends at
// or before T: such requests do not overlap, whatever the row starts hold, and of those that a row lies in only the
// first can be one (a later one that counts would begin behind the row).
TB_DEVI bool row_counts(const LogitsArgs& a, int t, int* found) {
  if (!a.row_start) return true;
  __syncthreads();
  if (threadIdx.x == 0) *found = a.B;
  __syncthreads();
  for (int b = threadIdx.x; b < a.B; b += blockDim.x)
    if (a.row_start[b] <= t && t < a.row_start[b + 1]) atomicMin(found, b);
  __syncthreads();
  const int b = *found;
  if (b == a.B) return false;
  const int first = a.row_start[b];
  bool wrong = first < 0 || a.row_start[b + 1] > a.T;
  for (int i = threadIdx.x; i < b; i += blockDim.x) wrong |= a.row_start[i] > first;
  return !__syncthreads_or(wrong);
}

constexpr int kMoveThreads = 256, kMoveChunk = 4096, kMoveStages = 4;

TB_DEVI void cp_async(uint32_t dst, const void* src, int have, int bytes) {  // what there is not of `bytes` is zeroed
  if (bytes == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(have) : "memory");
  if (bytes == 8) asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(have) : "memory");
  if (bytes == 4) asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(have) : "memory");
}

// logits of a thread at a time: 16 bytes of out, so that a warp's accesses are whole sectors
template <typename Out>
constexpr int move_each() { return sizeof(Out) == 2 ? 8 : 4; }
// bytes of a stage: logits, and a mask word for each thread's few
template <typename Out>
constexpr int move_stage() { return kMoveChunk * 2 + kMoveChunk / move_each<Out>() * 4; }

// Every CTA takes an equal run of all rows' chunks; logits and mask words come by cp.async into a ring of the thread's own,
// kMoveStages - 1 chunks ahead (rows whose distance is no multiple of 8: one element at a time, 64 rows of 248319 behind
// 8000 tokens 53.6 us in a graph against 32.3 where the rows are 248320 apart; of 50257 behind 700 14.8 against 8.9; one row
// of 50257 6.1, as of 50256).  64 rows of 248320 to fp32, 96 MB in 16.0 us by itself; 38 MB of them pass DRAM, 2.4 TB/s, as what
// is written stays in L2, so that loads' latency bounds it, not HBM.  Three CTAs an SM of four stages
// leave shared memory for the second launch beside them (with six stages it began when these were through).
template <typename Out, bool ALIGNED>
__global__ void __launch_bounds__(kMoveThreads, 4) logits_move_kernel(const LogitsArgs a) {
  constexpr int E = move_each<Out>(), K = kMoveChunk / (kMoveThreads * E), S = kMoveStages;
  constexpr int kPiece = kMoveThreads * E * 2, kStage = move_stage<Out>();  // bytes
  static_assert(kStage == K * (kPiece + kMoveThreads * 4), "pieces, then words");
  extern __shared__ __align__(16) unsigned char logits_smem[];
  __shared__ int found;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // what came before is over (see launch_early), for the second launch too
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x;
  const uint32_t ring = smem_u32(logits_smem);
  auto piece = [&](int stage, int k) { return ring + stage * kStage + k * kPiece + tid * (E * 2); };
  auto word = [&](int stage, int k) { return ring + stage * kStage + K * kPiece + (k * kMoveThreads + tid) * 4; };
  const int64_t units = (int64_t)a.T * a.chunks, stop = units * (blockIdx.x + 1) / gridDim.x;
  const int64_t mask_words = (a.V + 31) / 32;
  struct Cursor {
    int64_t u;
    int t, chunk;
  };
  auto mask_of = [&](int t) -> const uint32_t* {
    const int64_t m = !a.mask ? -1 : a.mask_row ? a.mask_row[t] : t;
    return m >= 0 && m < a.mask_rows ? a.mask + m * mask_words : nullptr;
  };
  Cursor f;  // what is fetched next, and what is stored next
  f.u = units * blockIdx.x / gridDim.x;
  f.t = (int)(f.u / a.chunks);
  f.chunk = (int)(f.u - (int64_t)f.t * a.chunks);
  Cursor c = f;
  auto advance = [&](Cursor& n) {
    ++n.u;
    if (++n.chunk == a.chunks) n.chunk = 0, ++n.t;
  };
  int fetch_row = -1;
  const uint32_t* fetch_mask = nullptr;
  auto fetch = [&](int stage) {
    if (f.u < stop) {
      if (f.t != fetch_row) fetch_mask = mask_of(f.t);
      fetch_row = f.t;
      const int v = f.chunk * kMoveChunk + tid * E;
      const __half* in = a.in + f.t * a.ld + v;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int w = v + k * kMoveThreads * E, have = min(E, a.V - w);
        if (ALIGNED && have > 0) cp_async(piece(stage, k), in + k * kMoveThreads * E, have * 2, E * 2);
        if (fetch_mask && have > 0) cp_async(word(stage, k), fetch_mask + (w >> 5), 4, 4);
      }
      advance(f);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i) fetch(i);
  int row = -1, stage = 0;
  bool counts = false, masked = false;
  for (; c.u < stop; advance(c)) {
    fetch(stage == 0 ? S - 1 : stage - 1);
    if (c.t != row) {
      counts = row_counts(a, c.t, &found);
      masked = mask_of(c.t) != nullptr;
      row = c.t;
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
    const int v = c.chunk * kMoveChunk + tid * E;
    const __half* in = a.in + c.t * a.ld + v;
    Out* out = static_cast<Out*>(a.out) + c.t * a.ldo + v;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int at = k * kMoveThreads * E, have = a.V - v - at;
      if (!counts || have <= 0) continue;
      uint32_t x[E / 2];
      if constexpr (!ALIGNED) {
        load_some<E>(x, in + at, have);
      } else if constexpr (E == 8) {
        const uint4 q = ld_shared_v4(piece(stage, k));
        x[0] = q.x, x[1] = q.y, x[2] = q.z, x[3] = q.w;
      } else {
        const uint2 q = ld_shared_v2(piece(stage, k));
        x[0] = q.x, x[1] = q.y;
      }
      if (masked) mask_logits<E>(x, __float_as_uint(ld_shared_f(word(stage, k))) >> ((v + at) & 31));
      if (ALIGNED && have >= E) store_logits<E>(out + at, x);
      else store_some<E>(out + at, x, have);
    }
    stage = stage == S - 1 ? 0 : stage + 1;
  }
}
// ---------------------------------------------------------------- counted and biased tokens
// A CTA takes a request's tokens whose mixed numbers end in its part's; a part has about `part_tokens` of the history, so
// that its table is nearly never too full.  Where it is, its tokens are done in two halves by the next bit, and so on.
// Bound by latency: every part reads the whole history (from L2) for its own tokens, counts them, and then a thread's tokens
// have a chain of a scattered load and a scattered store a row.  64 requests with histories up to 8000, by itself 19.6 us,
// both launches 25.4 in a graph; nine trees of 5 to 16 drafts behind 2000 to 30000, 31.4 and 42.2: about 13 to count, 10
// to gather the rows' logits, 6 to store them, 3 for the masks.  (With counts of the whole vocabulary in one launch
// that moves the rows too: 31 to 46, and 46 to 89.)  Alone, in place without a mask: 64 requests of 8000 31.9 us (to another
// place 32.4, in place under masks 38.6).  Three CTAs an SM, 40 registers a thread, 16 bytes spilled.
constexpr int kFixThreads = 512, kTable = 4096, kMostTokens = kTable / 4 * 3;
constexpr int kRows = 64;    // of a request at a time
constexpr int kResults = 4096;
constexpr uint32_t kNoResult = 0xffffdeadu;  // (a NaN that no operation gives)
constexpr int kDrafts = 64;  // of a request that are counted
// of a token's count: in the prompt, has a bias, is a drafted one's
constexpr uint32_t kPromptBit = 0x80000000u, kBiasBit = 0x40000000u, kDraftBit = 0x20000000u, kCountBits = kDraftBit - 1;

struct FixShared {
  uint32_t key[kTable];    // token + 1, 0: none
  uint32_t count[kTable];  // times generated, and the bits above
  uint16_t list[kTable];   // places taken
  uint32_t listed, pad[3];
  unsigned long long path[kRows];  // of the rows: the drafts they count
  int32_t mask_row[kRows];         // of the rows, -1: none
  int32_t draft[kDrafts];          // the drafted tokens
  float result[kResults];          // of rows and listed tokens, or kNoResult
  uint32_t bias[kTable];           // where there are biases: the last place of the token's in the lists
};
static_assert(kMostTokens + kFixThreads < kTable && kMostTokens + kFixThreads <= kResults, "the threads that do not yet know of a full table find places");

TB_DEVI uint32_t token_place(uint32_t id) { return (id * 2654435761u) >> 20; }
static_assert(kTable == 1 << 12, "token_place gives 12 bits");
TB_DEVI uint32_t token_mix(uint32_t id) { return (id ^ id >> 11) * 2246822519u >> 8; }  // 24 bits

// the place of a token in the table, new or not
TB_DEVI int table_insert(FixShared& s, uint32_t id) {
  for (uint32_t p = token_place(id);; p = (p + 1) & (kTable - 1)) {
    const uint32_t k = atomicCAS(&s.key[p], 0u, id + 1);
    if (k == id + 1) return (int)p;
    if (k == 0) {
      s.list[atomicAdd(&s.listed, 1u)] = (uint16_t)p;
      return (int)p;
    }
  }
}

template <typename Out>
__global__ void __launch_bounds__(kFixThreads, 3) logits_fix_kernel(const LogitsArgs a) {
  extern __shared__ __align__(16) unsigned char fix_smem[];
  FixShared& s = *reinterpret_cast<FixShared*>(fix_smem);
  const int tid = threadIdx.x, b = blockIdx.y, part = blockIdx.x;
  int bad = 0;
  // the request's lengths, whose errors its first CTA reports
  const int64_t row = a.slot ? __ldg(a.slot + b) : b;
  int len = __ldg(a.hist_len + b);
  const int prompt = a.prompt_len ? __ldg(a.prompt_len + b) : 0;
  int bias_from = a.bias_ids ? __ldg(a.bias_start + b) : 0, bias_to = a.bias_ids ? __ldg(a.bias_start + b + 1) : 0;
  int first = b, end = b + 1;
  if (a.row_start) first = __ldg(a.row_start + b), end = __ldg(a.row_start + b + 1);
  if (row >= a.n_hist) bad |= TB_DEV_BAD_ID;
  if (len < 0 || len > a.ldh || prompt < 0 || prompt > len) bad |= TB_DEV_BAD_LEN;
  if (row < 0 || row >= a.n_hist || len < 0) len = 0;
  if (len > a.ldh) len = (int)a.ldh;
  if (bias_from < 0 || bias_to < bias_from || bias_to > a.n_bias) {
    bad |= TB_DEV_BAD_LEN;
    bias_from = bias_to = 0;
  }
  int parts_log2 = 0;
  while (parts_log2 < a.parts_log2 && (int64_t)a.part_tokens << parts_log2 < (int64_t)len + (bias_to - bias_from)) ++parts_log2;
  if (part >> parts_log2) return;
  if (a.row_start) {  // (a request that counts: see row_counts)
    bool wrong = first < 0 || end < first || end > a.T;
    for (int i = tid; i < b; i += kFixThreads) wrong |= __ldg(a.row_start + i) > first;
    if (__syncthreads_or(wrong)) {
      if (tid == 0) set_status(a.status, TB_DEV_BAD_LEN);
      end = first;
    }
  }
  if (first >= end) {
    if (bad && tid == 0) set_status(a.status, bad);
    asm volatile("griddepcontrol.wait;" ::: "memory");  // this launch is not over before the first
    return;
  }
  const int drafts = a.fresh ? min(end - first, kDrafts) : 0;
  if (a.fresh && end - first > kDrafts) bad |= TB_DEV_BAD_LEN;
  if (tid < drafts) s.draft[tid] = __ldg(a.fresh + first + tid);
  const float rho = a.repetition ? __ldg(a.repetition + b) : 1.f;
  const float presence = a.presence ? __ldg(a.presence + b) : 0.f, frequency = a.frequency ? __ldg(a.frequency + b) : 0.f;
  const int64_t mask_words = (a.V + 31) / 32;
  bool waited = false;
  int highest = -1;
  // the part's tokens whose next `bits` bits are `value`
  uint32_t bits = 0, value = 0;
  while (true) {
    for (int i = tid; i < kTable / 4; i += kFixThreads) reinterpret_cast<uint4*>(s.key)[i] = reinterpret_cast<uint4*>(s.count)[i] = make_uint4(0, 0, 0, 0);
    if (bias_to > bias_from)
      for (int i = tid; i < kTable / 4; i += kFixThreads) reinterpret_cast<uint4*>(s.bias)[i] = make_uint4(0, 0, 0, 0);
    if (tid == 0) s.listed = 0;
    __syncthreads();
    const uint32_t want = (uint32_t)part | value << parts_log2, care = (1u << (parts_log2 + bits)) - 1;
    auto mine = [&](int id) { return (token_mix((uint32_t)id) & care) == want; };
    auto full = [&] { return *reinterpret_cast<volatile uint32_t*>(&s.listed) > kMostTokens; };
    const int32_t* history = a.history + row * a.ldh + tid;
    constexpr int kAhead = 8;
    for (int i0 = 0; i0 < len; i0 += kFixThreads * kAhead) {
      int id[kAhead];
      const int left = len - i0 - tid;
#pragma unroll
      for (int j = 0; j < kAhead; ++j) id[j] = j * kFixThreads < left ? __ldg(history + i0 + j * kFixThreads) : -1;
      uint32_t hits = 0;
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        highest = max(highest, id[j]);
        hits |= mine(id[j]) ? 1u << j : 0u;
      }
      // equal tokens of a warp are counted together: the most frequent ones are a large share of any text (verifying
      // drafts behind up to 30000 tokens: 44 us; each by itself: 49)
#pragma unroll 1
      for (; __any_sync(0xffffffffu, hits != 0); hits &= hits - 1) {
        const int at = (__ffs(hits) - 1) * kFixThreads;
        const int id = hits && at < left ? __ldg(history + i0 + at) : -1;
        const bool is = (unsigned)id < (unsigned)a.V;  // (not padding, and a token)
        const uint32_t key = is ? (uint32_t)id | (i0 + tid + at < prompt ? kPromptBit : 0u) : ~0u;
        const unsigned equal = __match_any_sync(0xffffffffu, key);
        if (is && (tid & 31) == __ffs(equal) - 1 && !full()) {
          uint32_t* c = &s.count[table_insert(s, (uint32_t)id)];
          if (key & kPromptBit) atomicOr(c, kPromptBit);
          else atomicAdd(c, (uint32_t)__popc(equal));
        }
        __syncwarp();
      }
    }
    for (int i = bias_from + tid; i < bias_to; i += kFixThreads) {
      const int id = __ldg(a.bias_ids + i);
      highest = max(highest, id);
      if ((unsigned)id >= (unsigned)a.V || !mine(id) || full()) continue;
      const int p = table_insert(s, id);
      atomicOr(&s.count[p], kBiasBit);
      atomicMax(&s.bias[p], (uint32_t)i);
    }
    if (tid < drafts) {
      const int id = s.draft[tid];
      highest = max(highest, id);
      if ((unsigned)id < (unsigned)a.V && mine(id) && !full()) atomicOr(&s.count[table_insert(s, (uint32_t)id)], kDraftBit);
    }
    __syncthreads();
    const int listed = s.listed;
    if (listed > kMostTokens && bits + parts_log2 < 24) {
      ++bits;
      __syncthreads();
      continue;
    }
    // as many rows at a time as there is room for their results
    const int together = listed ? min(kRows, max(1, kResults / listed)) : kRows;
    for (int t = first; t < end; t += together) {
      const int rows = min(together, end - t);
      if (tid < rows) {
        const int r = t + tid, i = r - first;
        s.path[tid] = !a.fresh ? 0 : a.tree ? a.tree[r] : i < 63 ? (2ull << i) - 1 : ~0ull;
        const int64_t m = !a.mask ? -1 : a.mask_row ? __ldg(a.mask_row + r) : r;
        if (a.mask && m >= a.mask_rows) bad |= TB_DEV_BAD_ID;
        s.mask_row[tid] = a.mask && m < a.mask_rows ? (int)m : -1;
      }
      __syncthreads();
      // results of a thread's tokens, in all rows.  In place, what the first launch does to the logits read here is to
      // write them again, or minus infinity where the mask leaves them out, which is looked at here too
      for (int i = tid; i < listed; i += kFixThreads) {
        const int p = s.list[i], v = (int)s.key[p] - 1;
        const uint32_t base = s.count[p];
        const float bias = base & kBiasBit ? __ldg(a.bias_values + s.bias[p]) : 0.f;
        unsigned long long same = 0;
        if (base & kDraftBit)
          for (int j = 0; j < drafts; ++j)
            if (s.draft[j] == v) same |= 1ull << j;
        // first the logits alone, several on their way at once
        float* const result = s.result + i;
        const __half* in = a.in + t * a.ld + v;
        for (int r0 = 0; r0 < rows; r0 += 8) {
          unsigned short x[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = r0 + j < rows ? __ldcg(reinterpret_cast<const unsigned short*>(in + (r0 + j) * a.ld)) : 0;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (r0 + j < rows) result[(r0 + j) * listed] = half_bits_to_float(x[j]);
        }
#pragma unroll 1
        for (int r = 0; r < rows; ++r) {
          const int m = s.mask_row[r];
          const uint32_t c = (base & ~kDraftBit) + __popcll(s.path[r] & same);
          float l = result[r * listed];
          if (c & ~kBiasBit) {
            l = l > 0.f ? __fdiv_rn(l, rho) : __fmul_rn(l, rho);
            if (c & kCountBits) l = __fsub_rn(__fsub_rn(l, __fmul_rn(frequency, (float)(c & kCountBits))), presence);
          }
          if (c & kBiasBit) l = __fadd_rn(l, bias);
          if (__float_as_uint(l) == kNoResult) l = -l;  // (a NaN as any other)
          const bool allowed = m < 0 || (__ldg(a.mask + m * mask_words + (v >> 5)) >> (v & 31) & 1);
          result[r * listed] = c && allowed ? l : __uint_as_float(kNoResult);
        }
      }
      if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");  // the rows are where they go
      waited = true;
      for (int i = tid; i < listed; i += kFixThreads) {
        Out* out = static_cast<Out*>(a.out) + t * a.ldo + (s.key[s.list[i]] - 1);
#pragma unroll 1
        for (int r = 0; r < rows; ++r, out += a.ldo) {
          const float l = s.result[r * listed + i];
          if (__float_as_uint(l) != kNoResult) store_logit(out, l);
        }
      }
      __syncthreads();  // the rows' words, and the table, have been used
    }
    // the next value of so many bits, or of fewer
    while (bits && (value >> (bits - 1) & 1)) value &= ~(1u << --bits);
    if (!bits) break;
    value |= 1u << (bits - 1);
  }
  if (highest >= a.V) bad |= TB_DEV_BAD_ID;
  if (bad) set_status(a.status, bad);
}

}  // namespace tb

extern "C" int tb_logits_adjust(const uint16_t* logits, int64_t ld, int64_t T, int64_t V, const int32_t* row_start, int64_t B,
                                const int32_t* history, int64_t n_hist, int64_t ldh, const int32_t* slot, const int32_t* hist_len,
                                const int32_t* prompt_len, const int32_t* fresh, const uint64_t* tree, const float* repetition,
                                const float* presence, const float* frequency, const int32_t* bias_start, const int32_t* bias_ids,
                                const float* bias_values, int64_t n_bias, const uint32_t* mask, int64_t mask_rows,
                                const int32_t* mask_row, void* out, int64_t ldo, int out_type, int32_t* dev_status, void* stream) {
  using namespace tb;
  if (T < 0 || T > INT_MAX || V < 1 || V > (1 << 24) || ld < V || ldo < V || B < 1 || n_hist < 1 || ldh < 0 || ldh > (1 << 28) || n_bias < 0 ||
      n_bias >= INT_MAX || mask_rows < 0)
    return TB_ERR_SHAPE;
  if (!row_start && B != T) return TB_ERR_SHAPE;  // row t is request t's
  if (!slot && n_hist < B) return TB_ERR_SHAPE;
  if (mask && !mask_row && mask_rows < T) return TB_ERR_SHAPE;
  if (out_type != TB_OUT_F16 && out_type != TB_OUT_F32) return TB_ERR_UNSUPPORTED;
  if (T > 65535 || B > 65535) return TB_ERR_TOO_LARGE;
  if (T == 0) return TB_OK;
  if (!logits || !out || !hist_len || (ldh && !history) || (n_bias && (!bias_start || !bias_ids || !bias_values)) || (tree && !fresh))
    return TB_ERR_NULL;
  if (!aligned16(logits) || !aligned16(out) || !aligned_to(row_start, 4) || !aligned_to(history, 4) || !aligned_to(slot, 4) ||
      !aligned_to(hist_len, 4) || !aligned_to(prompt_len, 4) || !aligned_to(fresh, 4) || !aligned_to(tree, 8) ||
      !aligned_to(repetition, 4) || !aligned_to(presence, 4) || !aligned_to(frequency, 4) || !aligned_to(bias_start, 4) ||
      !aligned_to(bias_ids, 4) || !aligned_to(bias_values, 4) || !aligned_to(mask, 4) || !aligned_to(mask_row, 4))
    return TB_ERR_ALIGN;
  if (out == logits && (out_type != TB_OUT_F16 || (ldo != ld && T > 1))) return TB_ERR_SHAPE;  // in place only element for element
  DeviceFacts f;
  int rc = device_facts(&f);
  if (rc != TB_OK) return rc;
  LogitsArgs a = {};
  a.in = reinterpret_cast<const __half*>(logits);
  a.out = out;
  a.row_start = row_start;
  a.history = history;
  a.slot = slot;
  a.hist_len = hist_len;
  a.prompt_len = prompt_len;
  a.fresh = fresh;
  a.tree = reinterpret_cast<const unsigned long long*>(tree);
  a.repetition = repetition;
  a.presence = presence;
  a.frequency = frequency;
  a.bias_start = bias_start;
  a.bias_ids = n_bias ? bias_ids : nullptr;
  a.bias_values = bias_values;
  a.mask = mask;
  a.mask_row = mask_row;
  a.status = dev_status;
  a.ld = ld;
  a.ldo = ldo;
  a.ldh = ldh;
  a.n_hist = n_hist;
  a.n_bias = n_bias;
  a.mask_rows = mask_rows;
  a.T = (int)T;
  a.V = (int)V;
  a.B = (int)B;
  a.chunks = (int)((V + kMoveChunk - 1) / kMoveChunk);
  // 1024 tokens of the history a CTA (half as many, or twice, cost 64 decoding requests and verification 5 to 15 us more),
  // 256 where requests are few: one of 700, 4000 and 30000 tokens takes 6.2, 6.3 and 17.3 us in a graph, with 1024 a CTA 7.9, 9.7
  // and 17.3; three 6.8, 7.0 and 18.7, with 1024 8.1, 10.1 and 18.6.  (Four, and eight, would gain the same by 256: 6.8, 6.8 and
  // 18.6 against 8.2, 10.4 and 18.4; 7.2, 7.8 and 24.7 against 8.3, 11.0 and 24.7.)  There are CTAs for what the buffer can hold,
  // whose surplus leaves at once: 64 requests of 8000 tokens in a buffer of 262144 take 36.1 us, in one of 8000 32.4; of 700 21.0
  // and 16.2
  a.part_tokens = B >= 4 ? 1024 : 256;
  a.parts_log2 = 0;
  while (a.parts_log2 < 5 && (int64_t)a.part_tokens << a.parts_log2 < ldh + n_bias / B) ++a.parts_log2;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool aligned = ld % 8 == 0 && ldo % 8 == 0, half = out_type == TB_OUT_F16;
  if (out != logits || mask) {
    void (*move)(const LogitsArgs) = half ? (aligned ? logits_move_kernel<__half, true> : logits_move_kernel<__half, false>)
                                          : (aligned ? logits_move_kernel<float, true> : logits_move_kernel<float, false>);
    const int64_t units = T * a.chunks, most = 3ll * f.sms;
    const int ring = kMoveStages * (half ? move_stage<__half>() : move_stage<float>());
    rc = ensure_dynamic_smem(reinterpret_cast<const void*>(move), f.device, ring);
    if (rc != TB_OK) return rc;
    rc = launch_early(move, dim3((unsigned)(units < most ? units : most)), kMoveThreads, (size_t)ring, s, a);
    if (rc != TB_OK) return rc;
  }
  void (*fix)(const LogitsArgs) = half ? logits_fix_kernel<__half> : logits_fix_kernel<float>;
  const int smem = n_bias ? (int)sizeof(FixShared) : (int)offsetof(FixShared, bias);
  rc = ensure_dynamic_smem(reinterpret_cast<const void*>(fix), f.device, smem);
  if (rc != TB_OK) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1u << a.parts_log2, (unsigned)B);
  cfg.blockDim = dim3(kFixThreads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = out != logits || mask ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, fix, (const LogitsArgs)a);
  if (e != cudaSuccess) {
    record_cuda_error(e);
    return TB_ERR_CUDA;
  }
  return check_launch();
}
