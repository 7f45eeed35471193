/*
 * tb.h — C ABI of the folded-Hadamard ternary "Packed" layer on one GB300 (sm_103a).
 *
 * The layer (restated from two pages about the Ternary-Bonsai-2-27B-mlx-2bit pack):
 *   [ARCH] "3.9GB 里藏了什么Bonsai 的混合注意力 推测解码 262K 上下文端侧架构逐层拆"
 *          (kwkr.cn/news/564617), sections "Hadamard 旋转把量化误差抹平的免费午餐" and
 *          "打包格式的工程MLX 2.25 bits 与 GGUF 的两种装箱";
 *   [PACK] PACK-RUNTIME.md walkthrough (lpnh.cn/news/2438023), sections
 *          "文本模型加载artifact.load_model 与 Packed 模块" and
 *          "仿射 2-bit 格式与 Prism contract v1".
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - All array arguments are DEVICE pointers owned by the caller; the library
 *    allocates no device memory and keeps no state between calls.
 *  - fp16 arrays are passed as uint16_t* holding IEEE binary16 bit patterns.
 *  - Every array is row-major and contiguous.  Device pointers must be 16-byte
 *    aligned (TB_ERR_ALIGN otherwise).
 *  - `stream` is a cudaStream_t (NULL = legacy default stream).  Every call is
 *    asynchronous on that stream; the return value reports argument validation
 *    and launch errors only.  Errors that depend on data (a bad code, an id out
 *    of range, a bounded wait that ran out) are OR-ed into the optional device
 *    word `dev_status` (TB_DEV_* bits), which the caller reads after a sync.
 *    Kernels never trap.
 *  - The layer refuses rather than guesses: a shape, block or group size it
 *    does not implement is an error, never a silent fallback.
 *  - Codes: ternary t in {-1,0,1} is stored as q = t + 1 in {0,1,2}; a uint32
 *    word holds 16 codes, code i of the word at bits 2i..2i+1 (least
 *    significant first); word j of a row holds the row's codes 16j..16j+15.
 *  - Group size 128 and 2 bits per code are fixed.  Per group: one fp16 scale s
 *    and one fp16 bias b (= -s in the pack); a code decodes to s*q + b.
 *  - Scale-only form: every call that takes `biases` also accepts NULL there.
 *    Each bias is then taken as the pack's -s (the fp16 sign bit of s flipped)
 *    and never read, so a code decodes to s*(q - 1) = s*t and the call reads
 *    1/64 byte less per weight.  For a pack written by tb_pack_w2 the result is
 *    bit-identical to passing its stored biases.  ([ARCH] "打包格式的工程": the
 *    stored bias is always -scale, so it adds bytes but no information.)
 *  - Hadamard block: 1024 (the pack's block_size) or 0 (= module not folded,
 *    no transform).  The transform is the normalised Sylvester-Walsh-Hadamard
 *    matrix in natural order, H[i][j] = (-1)^popcount(i&j), scaled by
 *    1/sqrt(1024) = 1/32, applied to consecutive 1024-element blocks of the
 *    last axis; the sign vector is indexed by the absolute position on that axis.
 */
#ifndef TB_H
#define TB_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* return codes */
enum {
  TB_OK = 0,
  TB_ERR_NULL = -1,        /* a required pointer is NULL */
  TB_ERR_SHAPE = -2,       /* M, N, K, T, V or D out of range or not a multiple it must be */
  TB_ERR_UNSUPPORTED = -3, /* block not 0, 512, 1024, 2048 or 4096 (the chain and the
                              no-allocation GEMV: not 0 or 1024), or an algorithm not built */
  TB_ERR_VALUE = -4,       /* a host-checked value is invalid */
  TB_ERR_CUDA = -5,        /* a CUDA launch or query failed (see tb_last_cuda_error) */
  TB_ERR_ALIGN = -6,       /* a device pointer is not 16-byte aligned */
  TB_ERR_WORKSPACE = -7,   /* workspace NULL or smaller than the size query returned */
  TB_ERR_TOO_LARGE = -8    /* beyond a fixed limit: the no-allocation scratch, or the chain's M <= 8 and SM ring */
};

/* bits OR-ed into *dev_status by kernels */
#define TB_DEV_BAD_CODE 1  /* tb_pack_w2: a code outside {-1,0,1}; tb_transcode_gguf: a block
                              slot or digit that is not a trit */
#define TB_DEV_BAD_ID 2    /* tb_embed_lookup: an id outside [0, V) (its row is written as zeros); a slot, an
                              adapter, a token or a mask's row past its table (taken as none) */
#define TB_DEV_TIMEOUT 4   /* a bounded wait inside a kernel gave up; outputs are not valid */
#define TB_DEV_BAD_PLAN 8  /* tb_chain_run, tb_rotary*, tb_adapter_linear: the plan does not match the launch
                              (nothing computed); tb_rotary_plan: a frequency that is not finite (taken as 0) */
#define TB_DEV_BAD_SLOT 16 /* a slot or page number outside the cache (its token is left out) */
#define TB_DEV_NO_PAGE 32  /* tb_cache_plan: no page left on the free list, or a table row too short */
#define TB_DEV_BAD_LEN 64  /* lengths or row starts that do not fit together or the arguments */

/* algorithm choice for tb_packed_linear_algo */
#define TB_ALGO_AUTO 0       /* the GEMV for M <= 2, the batched GEMV on mma.sync for 3..32
                                tokens, the batched-decode GEMV on tensor memory for 33..64, the
                                tensor-core GEMM above */
#define TB_ALGO_GEMV 1       /* fused sign*FWHT prologue + streaming W2 GEMV (the warp-level one);
                                any M (passes of 8 tokens) */
#define TB_ALGO_TC 2         /* FWHT kernel into the workspace + tcgen05/TMEM GEMM; any M */
#define TB_ALGO_GEMV_SYNC 3  /* the warp-level GEMV only (mma.sync on fp16 operands); any M */
#define TB_ALGO_GEMV_TMEM 4  /* the tensor-memory GEMV (tcgen05.mma on e4m3 operands, decoded
                                codes in tensor memory): M <= 2, K a multiple of 1024, block 0
                                or 1024, at most 6 1024-blocks of x per SM's share of the work;
                                TB_ERR_UNSUPPORTED where it does not apply.  Slower than the
                                warp-level GEMV at these token counts; never chosen by AUTO */
#define TB_ALGO_GEMV_WIDE 5  /* the batched-decode GEMV on tensor memory: the weights the MMA's
                                128-row side (decoded to fp16 s*q + b in tensor memory), the
                                tokens its N side; x' rotated into the workspace first, as for
                                TB_ALGO_TC (same workspace); M <= 64 (else passes of 64 tokens),
                                K a multiple of 1024 (TB_ERR_UNSUPPORTED otherwise) */
#define TB_ALGO_GEMV_BATCH 6 /* the batched-decode GEMV on mma.sync: x' rotated once into the
                                workspace as the mma's operand image (per 512-k chunk and pass of
                                8, 16, 32 or 64 tokens), then every unit of packed codes decoded
                                once and run against all tokens of the pass; any M (passes of 64
                                tokens above 32), K a multiple of 1024 (TB_ERR_UNSUPPORTED
                                otherwise); tb_packed_linear_algo_workspace_size gives its
                                workspace */

/* Human-readable text of a return code; never NULL. */
const char* tb_status_string(int status);

/* Text of the last CUDA error seen by this thread's calls (or ""). */
const char* tb_last_cuda_error(void);

/* Library version, major*10000 + minor*100 + patch. */
int tb_version(void);

/*
 * tb_pack_w2 — weight packer of the W2-g128 affine container.
 * [ARCH] "打包格式的工程": codes {0,1,2} rearranged into uint32 words; bias = -scale.
 *   codes   int8 [N, K], values in {-1,0,1}
 *   scales  fp16 [N, K/128]
 *   w       uint32 [N, K/16]   (out) packed codes, layout as above
 *   biases  fp16 [N, K/128]    (out) -scales (sign bit flipped; exact)
 *   dev_status optional int32: TB_DEV_BAD_CODE if a code is not -1, 0 or 1
 *              (that field is still written, as (t+1) & 3).
 * K must be a positive multiple of 128, N >= 1.
 */
int tb_pack_w2(const int8_t* codes, const uint16_t* scales, int64_t N, int64_t K,
               uint32_t* w, uint16_t* biases, int32_t* dev_status, void* stream);

/*
 * tb_unpack_w2 — inverse of the packer (verification support).
 * [ARCH] "打包格式的工程": the codec ships an independent unpack() to check the packing.
 *   w      uint32 [N, K/16];  codes int8 [N, K] (out) = q - 1 (a field q = 3 gives 2).
 * K must be a positive multiple of 16, N >= 1.
 */
int tb_unpack_w2(const uint32_t* w, int64_t N, int64_t K, int8_t* codes, void* stream);

/* GGUF block formats of the same trits (tb_transcode_gguf) */
#define TB_FMT_PQ2_0 1  /* 34 bytes per 128 weights: fp16 scale, 128 2-bit slots */
#define TB_FMT_PTQ1_0 2 /* 28 bytes per 128 weights: fp16 scale, 128 trits five per byte */

/*
 * tb_transcode_gguf — lossless transcoding of GGUF blocks into the W2-g128 container.
 * [ARCH] "打包格式的工程": PQ2_0 (34 bytes per 128 weights, each trit in a 2-bit slot) and
 * PTQ1_0 (28 bytes, dense trits) carry the same trits and group scales; the transcoder takes
 * the scale from the block header, sets the bias to its negation and rearranges the codes
 * into uint32 words.  The page gives the block sizes, not the byte layout inside a block;
 * the layout read here: bytes 0-1 the fp16 scale; PQ2_0: slot i at bits 2(i%4) of byte
 * 2 + i/4, slot value t + 1; PTQ1_0: byte 2 + j = sum_i (t[5j+i] + 1) * 3^i over the trits
 * 5j .. 5j+4 below 128 (first trit least significant; byte 27 holds trits 125..127).
 *   blocks  uint8, N * (K/128) blocks back to back, row by row (row n, group g at block
 *           n*K/128 + g); 2-byte aligned for PQ2_0, 4-byte aligned for PTQ1_0;
 *   format  TB_FMT_PQ2_0 or TB_FMT_PTQ1_0 (else TB_ERR_UNSUPPORTED);
 *   w       uint32 [N, K/16] (out), as tb_pack_w2 writes it; 16-byte aligned;
 *   scales  fp16 [N, K/128] (out); biases fp16 [N, K/128] (out, = -scales) or NULL.
 * K a positive multiple of 128, N >= 1.  dev_status optional: TB_DEV_BAD_CODE when a PQ2_0
 * slot holds 3, a PTQ1_0 byte is 243 or more, or a digit past trit 127 is not zero (the
 * outputs of such a block are then not valid).
 */
int tb_transcode_gguf(const uint8_t* blocks, int format, int64_t N, int64_t K, uint32_t* w,
                      uint16_t* scales, uint16_t* biases, int32_t* dev_status, void* stream);

/*
 * tb_gguf_linear — the packed layer read straight from GGUF blocks, no transcoding:
 *   y[M,N] = fwht(x)[M,K] . W[N,K]^T,  W[n, 128g + i] = d[n,g] * t[n, 128g + i],
 * the trits t and block scales d as the blocks hold them (the layout tb_transcode_gguf reads;
 * the scale-only form: a code q = t + 1 decodes to d * (q - 1)).  [ARCH] "打包格式的工程":
 * PQ2_0 and PTQ1_0 carry the same trits and scales as the 2.25-bit container; PTQ1_0 is the
 * densest of the three (1.75 bits per weight) and costs extra arithmetic to decode.
 *   x       fp16 [M, K];  signs, block: as tb_packed_linear (block 0: x used as it is);
 *   blocks  uint8, N * (K/128) blocks of `format` back to back, row by row; 16-byte aligned;
 *   format  TB_FMT_PQ2_0 or TB_FMT_PTQ1_0 (else TB_ERR_UNSUPPORTED);
 *   y       fp16 [M, N] (out);
 *   workspace  device scratch of at least tb_gguf_linear_workspace_size(M, K, block) bytes
 *           (x' [M, K] fp16; none needed for block 0), 16-byte aligned.
 * K a multiple of 1024 (TB_ERR_SHAPE otherwise), M, N >= 1.  dev_status optional:
 * TB_DEV_BAD_CODE when a PQ2_0 slot holds 3 (read as d * 2), a PTQ1_0 byte is 243 or more (read
 * as five trits of -1) or a PTQ1_0 digit past trit 127 is not zero (not read).  Tokens are taken
 * in passes of up to 4 (fewer when x' of 4 tokens does not fit in shared memory).
 */
/*
 * tb_encode_gguf — the other direction: the W2-g128 container (words and scales, the scale-only
 * reading: each bias taken as -scale, not read) written as GGUF blocks of `format`, in the layout
 * tb_transcode_gguf reads.  Lossless for codes 0..2; a code of 3 is not a trit: TB_DEV_BAD_CODE,
 * kept in its slot by PQ2_0, written as 2 by PTQ1_0.
 *   w       uint32 [N, K/16], 16-byte aligned;  scales fp16 [N, K/128];
 *   blocks  uint8 (out), N * (K/128) blocks; 2-byte aligned for PQ2_0, 4-byte for PTQ1_0.
 * K a positive multiple of 128, N >= 1.
 */
int tb_encode_gguf(const uint32_t* w, const uint16_t* scales, int64_t N, int64_t K, int format,
                   uint8_t* blocks, int32_t* dev_status, void* stream);

size_t tb_gguf_linear_workspace_size(int64_t M, int64_t K, int block);
int tb_gguf_linear(const uint16_t* x, const int8_t* signs, int block, const uint8_t* blocks, int format,
                   int64_t M, int64_t K, int64_t N, uint16_t* y, void* workspace, size_t workspace_bytes,
                   int32_t* dev_status, void* stream);

/*
 * tb_fwht — sign * normalised Walsh-Hadamard transform over blocks of `block` elements.
 * [ARCH] "Hadamard 旋转": fwht uses hadamard_transform with scale 1/sqrt(block);
 * forward multiplies by the signs first, the inverse multiplies by them again at the end.
 * [PACK] "仿射 2-bit 格式与 Prism contract v1": the pack uses block 1024; its loader also
 * accepts 512, 2048 and 4096.
 *   x  fp16 [M, K];  y fp16 [M, K] (out; y may equal x);
 *   signs int8 [K] of +-1, or NULL for all +1 (not checked on the device);
 *   forward (inverse = 0): y = (H/sqrt(block)) (signs * x) per block;
 *   inverse (inverse = 1): y = signs * ((H/sqrt(block)) x) per block.
 * Computed in fp32 (the scale 1/sqrt(block) rounded to fp32 for 512 and 2048, exact for
 * 1024 and 4096), rounded to fp16 (round to nearest even).  block: 512, 1024, 2048 or 4096
 * (else TB_ERR_UNSUPPORTED); K a positive multiple of block, M >= 1.
 */
int tb_fwht(const uint16_t* x, uint16_t* y, const int8_t* signs, int64_t M, int64_t K,
            int block, int inverse, void* stream);

/*
 * Bytes of workspace tb_packed_linear uses for these sizes.  Layout: a fixup region
 * (about 2 MB) for the decode GEMV's split schedule: counters of output tiles shared by
 * several SMs in its first 1024 bytes, then the SMs' fp32 parts of those tiles; then, for
 * the tensor-core path, the rotated activations x' (fp16 [M, K]) and the split schedule's
 * counters and parts; then, for a block other than 0 and 1024, x' in natural order (fp16
 * [M, K]).  The first 1024 bytes
 * must be zero before the first call that uses the workspace (zero-filling the whole
 * workspace will do); every completed call leaves them zero (a call that reported
 * TB_DEV_TIMEOUT may not: zero them again).  Calls sharing one workspace must be
 * ordered on one stream.
 */
size_t tb_packed_linear_workspace_size(int64_t M, int64_t K, int64_t N, int block);
size_t tb_packed_linear_algo_workspace_size(int64_t M, int64_t K, int64_t N, int block, int algo);

/*
 * tb_packed_linear — Packed.__call__ on the non-embedding path.
 * [ARCH] "Hadamard 旋转" (a folded module rotates its input, then multiplies it by the
 * transposed 2-bit, group-128 affine matrix)
 * and [PACK] "文本模型加载" (packed weights consumed directly, never expanded).
 *   y[m, n] = sum_k x'[m, k] * (s[n, k/128] * q[n, k] + b[n, k/128]),
 *   x' = fwht(x, block, signs) rounded to fp16 (x' = x when block = 0);
 *   x fp16 [M, K]; signs int8 [K] (+-1) or NULL (all +1; ignored when block = 0);
 *   w uint32 [N, K/16]; scales fp16 [N, K/128]; biases fp16 [N, K/128] or NULL
 *   (scale-only, b = -s); y fp16 [M, N] (out).
 * fp32 accumulation, fp16 output (round to nearest even).
 * block: 1024 (the pack's; the transform is fused into the matmul kernels), 0 (no transform),
 * or 512, 2048, 4096 (accepted by the pack's loader: x' = tb_fwht(x) into the workspace
 * first, then the matmul on it; the same x' rounded to fp16, one more launch).
 * K: positive multiple of 128 and of block.  M, N >= 1.
 * workspace: device memory of at least tb_packed_linear_workspace_size(...) bytes,
 * zero-filled before its first use (see above).  The GEMV path (M <= 8) with block 0 or 1024
 * also runs with workspace = NULL, then with output tiles never split between SMs (slower on
 * shapes whose row-tile count is not a multiple of the SM count).
 * dev_status optional (TB_DEV_TIMEOUT).
 */
int tb_packed_linear(const uint16_t* x, int64_t M, int64_t K, const int8_t* signs, int block,
                     const uint32_t* w, const uint16_t* scales, const uint16_t* biases, int64_t N,
                     uint16_t* y, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                     void* stream);

/* Same as tb_packed_linear with an explicit algorithm (TB_ALGO_*). */
int tb_packed_linear_algo(const uint16_t* x, int64_t M, int64_t K, const int8_t* signs, int block,
                          const uint32_t* w, const uint16_t* scales, const uint16_t* biases,
                          int64_t N, uint16_t* y, void* workspace, size_t workspace_bytes,
                          int32_t* dev_status, int algo, void* stream);

/*
 * tb_packed_linear_multi — tb_packed_linear for n (1..4) packed matrices that read the same
 * input x, as the q/k/v, gate/up and in_proj_qkv/in_proj_z modules of one layer do
 * ([ARCH] "Hadamard 旋转": the folded transform depends only on the input width, so the
 * modules that share x also share x' = fwht(x)).  x' is computed once per launch; matrix i
 * writes y[i] (fp16 [M, N[i]]).  w, scales, biases, N, y are HOST arrays of n entries holding
 * device pointers / row counts; biases (the array, or any entry) may be NULL (scale-only for
 * those matrices); K must be a positive multiple of 1024 (and of block); block as for
 * tb_packed_linear (512, 2048, 4096: x' computed once into the workspace).  Workspace as for
 * tb_packed_linear, sized with tb_packed_linear_workspace_size(M, K, max N, block).
 * The kernels are those AUTO picks for M: M <= 2, one decode GEMV launch for all matrices;
 * 3..32, one rotation into the operand image, then one batched GEMV launch per matrix; above,
 * one rotation, then one batched-decode GEMV (33..64) or tensor-core GEMM launch per matrix.
 */
int tb_packed_linear_multi(const uint16_t* x, int64_t M, int64_t K, const int8_t* signs, int block,
                           int n, const uint32_t* const* w, const uint16_t* const* scales,
                           const uint16_t* const* biases, const int64_t* N, uint16_t* const* y,
                           void* workspace, size_t workspace_bytes, int32_t* dev_status,
                           void* stream);

/*
 * Chained decode: a sequence of Packed linears (M <= 8 tokens) in one persistent launch.
 * [ARCH] "Hadamard 旋转": each linear is Packed.__call__ (fwht of its input, then the W2-g128
 * matmul); a decode step runs the model's linears one after another, every one reading what
 * an earlier one wrote.  [PACK] "文本模型加载": the modules and their packed tensors.
 *
 * Link i computes, for its input x and its n matrices (1..4, the modules that read the same
 * input), exactly what tb_packed_linear_multi computes.  The result of the whole chain equals
 * calling tb_packed_linear_multi once per link, in order, on one stream: link i reads x only
 * after every output of links 0..i-1 is complete, so x of a link may be (a slice of) any
 * earlier link's y.  The launch keeps one CTA per SM resident (a cooperative launch); while
 * the SMs wait for link i to complete, they already stream the packed weights of link i+1.
 */
typedef struct tb_chain_link {
  const uint16_t* x;          /* fp16 [M, K]; may be an output of an earlier link */
  const int8_t* signs;        /* int8 [K] (+-1) or NULL (all +1); ignored when block = 0 */
  int64_t K;                  /* positive multiple of 1024 (at most 2^20) */
  int32_t block;              /* 1024, or 0 = module not folded */
  int32_t n;                  /* matrices reading x: 1..4 */
  const uint32_t* w[4];       /* uint32 [N[i], K/16] packed codes */
  const uint16_t* scales[4];  /* fp16 [N[i], K/128] */
  const uint16_t* biases[4];  /* fp16 [N[i], K/128], or NULL (scale-only, b = -s) */
  int64_t N[4];               /* rows of matrix i, >= 1 */
  uint16_t* y[4];             /* fp16 [M, N[i]] (out) */
} tb_chain_link;

/* Bytes of device memory a plan of n_links links needs (an upper bound: 4 matrices per link). */
size_t tb_chain_plan_size(int n_links);

/*
 * tb_chain_plan — validate the links (same rules as tb_packed_linear_multi; M in 1..8) and
 * write the plan (link table + one TMA descriptor per matrix) to `plan`, device memory of at
 * least tb_chain_plan_size(n_links) bytes, 128-byte aligned, owned by the caller.  Copies the
 * plan on `stream` and waits for that copy (call it before any stream capture).  The plan
 * stays valid while every pointer in the links stays valid; it holds no other state.
 * Errors: TB_ERR_NULL, TB_ERR_SHAPE, TB_ERR_UNSUPPORTED, TB_ERR_ALIGN, TB_ERR_TOO_LARGE (M > 8),
 * TB_ERR_WORKSPACE (plan_bytes too small), TB_ERR_CUDA.
 */
int tb_chain_plan(const tb_chain_link* links, int n_links, int64_t M, void* plan,
                  size_t plan_bytes, void* stream);

/*
 * Bytes of workspace tb_chain_run uses (about 2 MB): counters in its first 1280 bytes, which
 * must be zero before the first run (zero-filling the whole workspace will do) and which every
 * completed run leaves zero (a run that reported TB_DEV_TIMEOUT may not: zero them again),
 * then per-SM fp32 parts of output tiles shared by several SMs (scratch).
 */
size_t tb_chain_workspace_size(void);

/*
 * tb_chain_set_wait — the bound of a plan's waits on the previous link.
 * Before its prologue, every CTA waits until all CTAs have counted the previous link complete;
 * that wait gives up after wait_ns nanoseconds (0 = the library default, 2 s), sets
 * TB_DEV_TIMEOUT and lets the run wind down (its outputs are then not valid; zero the
 * workspace's counters before the next run).  extra_count raises the count each link waits for
 * by that many, so that the wait cannot complete: it exists to test the timeout path without a
 * fault or a hang, and must be 0 for a run whose results are used.  Writes the two fields of the
 * plan on `stream` and waits for that copy.  Errors: TB_ERR_NULL, TB_ERR_ALIGN, TB_ERR_VALUE
 * (a negative value), TB_ERR_CUDA.  A new plan starts with wait_ns = 0 and extra_count = 0.
 */
int tb_chain_set_wait(void* plan, int64_t wait_ns, int32_t extra_count, void* stream);

/*
 * tb_chain_run — run a plan: one launch on `stream`, asynchronous.  n_links, M and max_K
 * (the largest K of the links) must be the values the plan was made with; a mismatch that
 * the device can see sets TB_DEV_BAD_PLAN and computes nothing.  Runs that share one
 * workspace must be ordered on one stream.  Errors: TB_ERR_NULL, TB_ERR_SHAPE, TB_ERR_ALIGN,
 * TB_ERR_WORKSPACE, TB_ERR_TOO_LARGE (more than 256 SMs, or M and max_K leave no room for
 * the weight ring in shared memory), TB_ERR_CUDA.  dev_status optional (TB_DEV_TIMEOUT,
 * TB_DEV_BAD_PLAN).
 */
int tb_chain_run(const void* plan, int n_links, int64_t M, int64_t max_K, void* workspace,
                 size_t workspace_bytes, int32_t* dev_status, void* stream);

/*
 * tb_embed_lookup — Packed.__call__ on the embedding path.
 * [ARCH] "Hadamard 旋转" (the looked-up rows are dequantised, then inverse-transformed) and
 * [PACK] "文本模型加载" (mx.dequantize of the looked-up rows, then the inverse transform).
 *   out[t, :] = signs * ((H/32) e) per block,  e = s*q + b of row ids[t] of the table.
 *   ids int32 [T]; w uint32 [V, D/16]; scales fp16 [V, D/128]; biases the same or NULL
 *   (scale-only, b = -s);
 *   signs int8 [D] (+-1) or NULL (all +1); out fp16 [T, D] (out).
 * An id outside [0, V) writes a row of zeros and sets TB_DEV_BAD_ID in dev_status.
 * block 1024 (fused), 512, 2048 or 4096 (the rows decoded into out, then the inverse
 * tb_fwht in place: the same result, since the pack's rows {-s, 0, s} are exact in fp16;
 * rows of a general affine bias are rounded to fp16 before that transform), or 0; D a
 * multiple of 128 and of block; T >= 0 (T = 0 is a no-op).
 */
int tb_embed_lookup(const int32_t* ids, int64_t T, const uint32_t* w, const uint16_t* scales,
                    const uint16_t* biases, int64_t V, int64_t D, const int8_t* signs, int block,
                    uint16_t* out, int32_t* dev_status, void* stream);

/*
 * tb_packed_linear_gemv_noalloc — the decode GEMV of tb_packed_linear for callers that
 * cannot provide device memory.  (No counterpart on the pages: it exists for callers
 * that are not allowed to allocate, e.g. code running under CUDA graph capture, plugins
 * inside a host runtime that owns all device memory, or services with a fixed memory
 * budget after start-up.)
 * Same arguments and result as tb_packed_linear for M <= 8 tokens, without workspace.
 * The state of the GEMV's split schedule lives in a fixed array inside the library
 * (about 2 MiB on every GPU that loads it, held until the process exits).
 *   - It allocates nothing: no cudaMalloc, no cudaFree, no allocating library call.
 *   - Limits: M <= 8 and a GPU with at most 256 SMs, else TB_ERR_TOO_LARGE;
 *     K a positive multiple of 1024 (block 1024, or block 0 with such a K), else TB_ERR_SHAPE.
 *   - The first call on each device looks up the array's device address for that device
 *     (cudaGetSymbolAddress); make that first call before any stream capture.
 *   - Each call clears the array's counters on `stream` before using it (cudaMemsetAsync).  All calls
 *     share the one array: calls that can overlap on the GPU (different streams, or
 *     different host threads) race and give wrong results; order them on one stream.
 */
int tb_packed_linear_gemv_noalloc(const uint16_t* x, int64_t M, int64_t K, const int8_t* signs,
                                  int block, const uint32_t* w, const uint16_t* scales,
                                  const uint16_t* biases, int64_t N, uint16_t* y,
                                  int32_t* dev_status, void* stream);

/*
 * The mixers between the packed linears ([ARCH] "混合注意力": 64 layers, full attention every
 * fourth with 24 query heads, 4 KV heads of 256; linear attention in the others with 16 key heads,
 * 48 value heads of 128 and an fp32 state).  Tokens of several requests lie packed one after
 * another: request b's rows are row_start[b] .. row_start[b+1] - 1 (int32 [B + 1]).  q, k and v may
 * be slices of a wider matrix (a fused projection): ld* is the distance of two tokens in elements,
 * a multiple of 8 and at least heads * D; within a token, heads are contiguous.  Query head h
 * reads KV (or key) head h / (heads / KV heads).  Rows of no request are neither read nor written.
 * Inference only: these calls have no gradient.  16-byte alignment is asked of the fp16 arrays, the
 * states and the workspaces; arrays of indices, lengths, decays and steps need that of their type.
 *
 * The paged K/V cache: two fp16 arrays [pages, Hkv, page, D]; page is 16, 32, 64, 128 or 256 tokens.
 * table int32 [B, max_pages]: the page that holds tokens p*page .. of request b.  A slot (int64)
 * is page number * page + place in the page; -1 is a padded token.
 */

/*
 * tb_cache_plan — the cache's bookkeeping for one step, from the requests' lengths.
 *   cached, fresh  int32 [B]: tokens already in the cache, and tokens this step adds (>= 0);
 *   free_pages     int32 [n_free]: pages to hand out, taken from its front in the order of the
 *                  requests and, within one, of its pages (may be NULL when n_free is 0);
 *   table          int32 [B, max_pages] (in/out): entries of the ceil(cached/page) pages held are
 *                  read, those of new pages written (-1 where none is left), others left alone;
 *   slots          int64 [T] (out): the new tokens' slots, packed by request; -1 past the last
 *                  token and for a token without a page (T: room, e.g. a graph's fixed size);
 *   row_start      int32 [B + 1] (out): running sums of fresh;  total int32 [B] (out): cached + fresh;
 *   used           int32 [1] (out) or NULL: pages taken from free_pages.
 * One launch; the result depends on the inputs alone (a second call with them gives it again).
 * Outputs must not overlap inputs.  B in 1..16384 (else TB_ERR_TOO_LARGE).  dev_status optional:
 * TB_DEV_NO_PAGE, TB_DEV_BAD_LEN (a negative length is taken as 0, a sum above T is cut),
 * TB_DEV_BAD_SLOT (a held page's entry is negative).
 */
int tb_cache_plan(const int32_t* cached, const int32_t* fresh, int64_t B, int64_t page,
                  const int32_t* free_pages, int64_t n_free, int32_t* table, int64_t max_pages,
                  int64_t* slots, int64_t T, int32_t* row_start, int32_t* total, int32_t* used,
                  int32_t* dev_status, void* stream);

/*
 * tb_cache_write — write the new tokens' K and V rows to their slots.
 *   k, v     fp16 [T, Hkv, D], tokens ldk / ldv elements apart;  slots int64 [T], no slot twice;
 *   k_cache, v_cache  fp16 [pages, Hkv, page, D] (out).
 * A negative slot is skipped; one past the cache is skipped and sets TB_DEV_BAD_SLOT.  D a multiple
 * of 8 up to 1024; T >= 0 (T = 0 is a no-op).
 */
int tb_cache_write(const uint16_t* k, int64_t ldk, const uint16_t* v, int64_t ldv,
                   const int64_t* slots, int64_t T, int64_t Hkv, int64_t D, uint16_t* k_cache,
                   uint16_t* v_cache, int64_t pages, int64_t page, int32_t* dev_status, void* stream);

/*
 * tb_tree_attention — attention of each request's newest tokens over its cache: one token per
 * request (ordinary decode), a run of them, or a tree of drafted tokens to verify.
 *   q        fp16 [T, Hq, D], tokens ldq apart; request b's n_b rows (n_b <= max_q <= 64) are the
 *            last n_b of its total[b] cached tokens (their K and V already written);
 *   tree     uint64 [T] or NULL: a row sees every token before its request's n_b newest, and of
 *            those the i-th (i < n_b) when bit i of its word is set; NULL: the first up to itself;
 *   scale    positive and finite, e.g. 1/sqrt(D);  o fp16 [T, Hq, D] (out).
 * o_i = sum_j w_ij v_j, w_i the softmax of scale q_i . k_j over what row i sees; a row that sees
 * nothing (or only scores of -infinity) gives zeros.  What a row does not see does not reach it,
 * not even as NaN or infinity.  D 64, 128 or 256 (else TB_ERR_UNSUPPORTED); max_q above 64:
 * TB_ERR_TOO_LARGE.  workspace: at least tb_tree_attention_workspace_size(B, T, max_q, Hq, Hkv, D)
 * bytes of scratch; its contents do not matter; calls that share one are ordered on one stream.  dev_status optional: TB_DEV_BAD_LEN (n_b above max_q,
 * total[b] below n_b or above max_pages * page: zeros), TB_DEV_BAD_SLOT (a page outside the cache:
 * its tokens are left out).
 */
size_t tb_tree_attention_workspace_size(int64_t B, int64_t T, int64_t max_q, int64_t Hq, int64_t Hkv,
                                        int64_t D);
int tb_tree_attention(const uint16_t* q, int64_t ldq, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                      const uint16_t* k_cache, const uint16_t* v_cache, int64_t pages, int64_t page,
                      const int32_t* table, int64_t max_pages, const int32_t* total,
                      const int32_t* row_start, int64_t B, int64_t max_q, const uint64_t* tree,
                      float scale, uint16_t* o, void* workspace, size_t workspace_bytes,
                      int32_t* dev_status, void* stream);

/*
 * tb_prompt_attention — causal attention over whole prompts, packed.
 *   q fp16 [Tq, Hq, D], k and v fp16 [Tk, Hkv, D], tokens ldq / ldk / ldv apart; request b's queries
 *   are rows q_start[b] .. of q and its keys rows k_start[b] .. of k and v (int32 [B + 1] each): lq
 *   and lk of them, the queries being the last lq of the lk positions, so query i sees keys
 *   j <= i + lk - lq (fewer keys than queries: the first rows see nothing and give zeros);
 *   scale, o, D: as for tb_tree_attention, with the same rule about what a row does not see.
 * dev_status optional: TB_DEV_BAD_LEN (row starts out of order or past Tq / Tk: zeros where the
 * rows can be told, else not written; in calls so large that 32 bits might not hold the work of requests
 * that overlap, nothing is written where they make more of it than Tq tokens and B requests in order can).
 */
int tb_prompt_attention(const uint16_t* q, int64_t ldq, const uint16_t* k, int64_t ldk,
                        const uint16_t* v, int64_t ldv, int64_t Tq, int64_t Tk, int64_t Hq,
                        int64_t Hkv, int64_t D, const int32_t* q_start, const int32_t* k_start,
                        int64_t B, float scale, uint16_t* o, int32_t* dev_status, void* stream);

/*
 * tb_gated_delta — the gated delta rule, over prompts or single tokens.  Per value head, S its
 * D x D state (rows: k, columns: v), token by token:
 *   S <- exp(g_t) S;  u = beta_t (v_t - S^T k_t);  S <- S + k_t u^T;  o_t = scale S^T q_t
 *   q, k     fp16 [T, Hk, D], v fp16 [T, Hv, D], tokens ldq / ldk / ldv apart; Hv a multiple of Hk;
 *   g, beta  fp32 [T, Hv]: logarithm of the decay (at most 0), and the step;
 *   normalise  nonzero: q and k are first divided by sqrt(sum of squares + 1e-6) (in fp32);
 *   state_in   fp32 [n_in, Hv, D, D] or NULL (zeros); request b starts from row slot_in[b] (int32 [B];
 *              NULL: row b); a negative slot: zeros;
 *   state_out  fp32 [n_out, Hv, D, D] or NULL; the final state goes to row slot_out[b] (NULL: b);
 *              negative: not kept.  state_out may be state_in; a row one request writes must not be
 *              one another request of the call reads or writes;
 *   max_len    the longest request's tokens: chooses the kernel.  Any value gives right results, but for
 *              steps that grow (beta |k|^2 above 2, k as normalised): above 16, where they grow by more than
 *              about 2^16 within 64 tokens, o and the state are NaN from there on;
 *   o        fp16 [T, Hv, D] (out).
 * A request of no tokens copies its state.  States, sums and decays are fp32.  What is not finite in a
 * token's inputs reaches neither the tokens before it nor other requests, and by v no other column;
 * with max_len above 16, o and the state are NaN from that token on where it does reach.  D must be 128
 * (TB_ERR_UNSUPPORTED).  workspace: at least tb_gated_delta_workspace_size(T, B, max_len, Hk, Hv)
 * bytes of scratch (may be 0); its contents do not matter; calls that share one are ordered on one
 * stream.  dev_status optional: TB_DEV_BAD_ID (a slot past its pool: taken as negative),
 * TB_DEV_BAD_LEN (row starts out of order or past T: that request is taken as empty; so are the last
 * requests where row starts that go back make them more together than T tokens and B requests can be).
 */
size_t tb_gated_delta_workspace_size(int64_t T, int64_t B, int64_t max_len, int64_t Hk, int64_t Hv);
int tb_gated_delta(const uint16_t* q, int64_t ldq, const uint16_t* k, int64_t ldk, const uint16_t* v,
                   int64_t ldv, const float* g, const float* beta, int64_t T, int64_t Hk, int64_t Hv,
                   int64_t D, const int32_t* row_start, int64_t B, int64_t max_len, int normalise,
                   float scale, const float* state_in, const int32_t* slot_in, int64_t n_in,
                   float* state_out, const int32_t* slot_out, int64_t n_out, uint16_t* o,
                   void* workspace, size_t workspace_bytes, int32_t* dev_status, void* stream);

/*
 * What a serving step does around the packed linears: rotary positions between the projection of q, k and v and
 * the cache, the requests' low-rank adapters beside a linear, and changes to the lm_head's logits before a token
 * is chosen.  Packing, row starts, token distances and alignment are those of the mixers above.
 */

/* pairs of a head that turn together: (x_i, x_{i+R/2}), or (x_2i, x_{2i+1}) */
#define TB_ROTARY_HALF 0
#define TB_ROTARY_PAIRS 1
/* frequencies scaled for contexts longer than the model's own, by `factor` */
#define TB_ROTARY_NONE 0    /* f_i = base^(-2i/R) */
#define TB_ROTARY_LINEAR 1  /* f_i / factor */
#define TB_ROTARY_BASE 2    /* base is first multiplied by factor^(R/(R-2)) (R above 2) */
#define TB_ROTARY_PARTS 3   /* pairs that turn more than beta_fast times over `original` tokens as they are, those
                               that turn less than beta_slow times divided by factor, a ramp over i between them */

/*
 * tb_rotary_plan — the table that tb_rotary reads: each pair's turns a token, and the rotation's amplitude.
 *   plan       at least tb_rotary_plan_size(R) bytes of device memory (0: R is not an even number in 2..1024);
 *   base       above 1;  factor positive;  original, beta_fast > beta_slow positive (TB_ROTARY_PARTS only);
 *   amplitude  what cosines and sines are multiplied by; 0 chooses it: 0.1 ln(factor) + 1 for TB_ROTARY_PARTS
 *              with a factor above 1, else 1;
 *   freqs      float64 [R/2] on the device, radians a token of each pair, in place of base and scaling (which must
 *              then be TB_ROTARY_NONE), or NULL.
 * One small launch on `stream`; made once for a model.  dev_status optional: TB_DEV_BAD_PLAN.
 */
size_t tb_rotary_plan_size(int64_t R);
int tb_rotary_plan(void* plan, size_t plan_bytes, int64_t R, double base, int scaling, double factor,
                   double original, double beta_fast, double beta_slow, double amplitude,
                   const double* freqs, int32_t* dev_status, void* stream);

/*
 * tb_rotary — q and k turned by their positions: a pair (a, b) of token t becomes
 *   amplitude * (a cos - b sin, a sin + b cos) of the angle pos[t] f_i; elements from R on are copied.
 *   q, k     fp16 [T, Hq, D] and [T, Hk, D], tokens ldq / ldk apart; Hk may be 0 (k and k_out then unused);
 *   pos      int32 [T], any value (a negative one turns back); whole turns are taken off exactly: angles are right to
 *            2^-22 of a turn for all positions and frequencies up to 1;
 *   plan, R  from tb_rotary_plan with the same R <= D;  layout TB_ROTARY_HALF or TB_ROTARY_PAIRS;
 *   inverse  nonzero: by the opposite angle (the transpose, amplitude included: the rotation's gradient);
 *   q_out, k_out  fp16 (out), tokens ldqo / ldko apart; may be q and k (with their distances), and must not
 *                 overlap them otherwise.
 * D a multiple of 8 up to 1024; T = 0 is a no-op.  dev_status optional: TB_DEV_BAD_PLAN.
 */
int tb_rotary(const uint16_t* q, int64_t ldq, int64_t Hq, const uint16_t* k, int64_t ldk, int64_t Hk,
              int64_t T, int64_t D, const int32_t* pos, const void* plan, int64_t R, int layout,
              int inverse, uint16_t* q_out, int64_t ldqo, uint16_t* k_out, int64_t ldko,
              int32_t* dev_status, void* stream);

/*
 * tb_rotary_cache_write — tb_rotary, with k (turned) and v written to their slots as tb_cache_write does.
 *   k_out    NULL: the turned k is kept in the cache only.  Other arguments as in the two calls.
 */
int tb_rotary_cache_write(const uint16_t* q, int64_t ldq, int64_t Hq, const uint16_t* k, int64_t ldk,
                          const uint16_t* v, int64_t ldv, int64_t Hkv, int64_t T, int64_t D,
                          const int32_t* pos, const int64_t* slots, const void* plan, int64_t R,
                          int layout, int inverse, uint16_t* q_out, int64_t ldqo, uint16_t* k_out,
                          int64_t ldko, uint16_t* k_cache, uint16_t* v_cache, int64_t pages, int64_t page,
                          int32_t* dev_status, void* stream);

/*
 * tb_adapter_plan — a step's tokens grouped by adapter, once for all linears of the step.
 *   row_start  int32 [B + 1];  adapter int32 [B]: each request's adapter, negative: none;  n: adapters there are;
 *   T          rows of the step's matrices (row_start[B] <= T; rows of no request are left alone);
 *   plan       at least tb_adapter_plan_size(T, n) bytes of device memory; holds nothing but the grouping.
 * One launch; the result depends on the inputs alone.  B and n up to 16384 (else TB_ERR_TOO_LARGE).  dev_status
 * optional: TB_DEV_BAD_ID (an adapter past n: taken as none), TB_DEV_BAD_LEN (row starts out of order or past
 * T: that request, and those after a row start that is too high, are taken as empty).
 */
size_t tb_adapter_plan_size(int64_t T, int64_t n);
int tb_adapter_plan(const int32_t* row_start, const int32_t* adapter, int64_t B, int64_t T, int64_t n,
                    void* plan, size_t plan_bytes, int32_t* dev_status, void* stream);

/*
 * tb_adapter_linear — the requests' adapters beside a linear that they share:
 *   out[t] = y[t] + scale[g] B[g] (A[g] x[t])   g the adapter of token t's request; out[t] = y[t] without one.
 *   x        fp16 [T, K], rows ldx apart: the linear's input (as given to tb_packed_linear, not rotated);
 *   a, b     fp16 [n, R, K] and [n, N, R];  scale fp32 [n];
 *   rank     int32 [n] or NULL (all R): adapter g uses the first rank[g] rows of A[g] and columns of B[g];
 *            what lies behind them does not matter;
 *   plan     of tb_adapter_plan with the same T and n;
 *   y, out   fp16 [T, N], rows ldy / ldo apart: the linear's output, and the result; out may be y (with its
 *            distance; rows without an adapter are then not touched) and must not overlap it or x otherwise.
 * A x and the sum are fp32; scale A x enters the second product off by at most 2^-22 of itself or 2^-51 of the largest
 * of the token's 64 ranks around it, the greater of the two; sums are rounded to the place of their largest term, in
 * which an element below 2^-14 counts as 2^-14; one rounding to fp16 at the end.  What is not finite stays in the rows
 * and columns that it reaches (an infinite element of B may give NaN there).  A token's row depends on no other token's x
 * and y; the order of its sums, and with it the last bits, also goes by T and n.  K, N and R multiples of 8, R up to
 * 256 (TB_ERR_UNSUPPORTED above).  workspace: at least
 * tb_adapter_linear_workspace_size(T, n, K, N, R) bytes of scratch; its contents do not matter; calls that share
 * one are ordered on one stream.  dev_status optional: TB_DEV_BAD_PLAN.
 */
size_t tb_adapter_linear_workspace_size(int64_t T, int64_t n, int64_t K, int64_t N, int64_t R);
int tb_adapter_linear(const uint16_t* x, int64_t ldx, int64_t T, int64_t K, const uint16_t* a,
                      const uint16_t* b, int64_t n, int64_t R, int64_t N, const int32_t* rank,
                      const float* scale, const void* plan, const uint16_t* y, int64_t ldy,
                      uint16_t* out, int64_t ldo, void* workspace, size_t workspace_bytes,
                      int32_t* dev_status, void* stream);

/* element type of an output */
#define TB_OUT_F16 0
#define TB_OUT_F32 1

/*
 * tb_logits_adjust — penalties, biases and grammar masks on logits.  Row t belongs to the request b with
 * row_start[b] <= t < row_start[b+1] (row_start NULL: to request t, and B = T).  For each token v, in this order:
 *   known (in the history's first hist_len[b] tokens, or on the row's path):  l <- l > 0 ? l / repetition[b]
 *                                                                                       : l * repetition[b]
 *   generated c times (behind the first prompt_len[b] of them, or on the path):  l <- l - frequency[b] c - presence[b]
 *   biased:                                                                       l <- l + its bias
 *   its bit of the row's mask is 0:                                               l <- -infinity
 *   logits     fp16 [T, V], rows ld >= V apart (any distance; multiples of 8 are faster);
 *   history    int32 [n_hist, ldh] (ldh up to 2^28): request b's tokens are row slot[b] (int32 [B]; NULL: row b; negative: none);
 *   hist_len   int32 [B];  prompt_len int32 [B] or NULL (zeros);
 *   fresh      int32 [T] or NULL: the tokens that the rows were computed from, where the history does not hold
 *              them yet: up to 64 a request, in the order of its rows.  A row's path is itself and its request's
 *              rows before it, or with tree (uint64 [T], as in tb_tree_attention) those whose bit its word has;
 *   repetition, presence, frequency  fp32 [B], each may be NULL (1, 0, 0);
 *   bias_start, bias_ids, bias_values  int32 [B + 1], int32 [n_bias], fp32 [n_bias]: request b's biased tokens
 *              (n_bias 0: none; unused pointers may then be NULL); of a token listed twice the last one counts;
 *   mask       uint32 [mask_rows, ceil(V/32)] or NULL, token v at bit v % 32 of word v / 32; row t reads row
 *              mask_row[t] (int32 [T]; NULL: row t; negative: no mask);
 *   out        [T, V] of out_type, rows ldo apart (out); may be logits where that is fp16 (with its distance), and
 *              must not overlap it otherwise.
 * Every step in fp32, rounded as written; one rounding to fp16.  A masked token gives -infinity whatever its logit
 * is.  Negative tokens are padding; rows of no request are not written (they are read).  T and B up to 65535
 * (TB_ERR_TOO_LARGE), V up to 2^24.  dev_status optional: TB_DEV_BAD_ID (a token, a history's or a mask's row past
 * its table: left out), TB_DEV_BAD_LEN (a length, a list or row starts that do not fit: cut, taken as empty, or
 * the row left out; more than 64 fresh tokens: the first 64).  The history's row, lengths and list are looked at of a
 * request without rows too, its tokens are not.
 */
int tb_logits_adjust(const uint16_t* logits, int64_t ld, int64_t T, int64_t V, const int32_t* row_start,
                     int64_t B, const int32_t* history, int64_t n_hist, int64_t ldh, const int32_t* slot,
                     const int32_t* hist_len, const int32_t* prompt_len, const int32_t* fresh,
                     const uint64_t* tree, const float* repetition, const float* presence,
                     const float* frequency, const int32_t* bias_start, const int32_t* bias_ids,
                     const float* bias_values, int64_t n_bias, const uint32_t* mask, int64_t mask_rows,
                     const int32_t* mask_row, void* out, int64_t ldo, int out_type,
                     int32_t* dev_status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TB_H */
