/*
 * bq.h -- C ABI of the low-bit weight-quantized decode QMV library (gfx950).
 *
 * Source of the method: the web article "oMLX Bonsai 自定义内核: Qwen 系列快速
 * QMV 路径完整解析" (cnnetsun.cn), section 二 (three kernel paths: qmv_fast,
 * qmv_wide with its symmetric variant, the t5 ternary format with its qmv,
 * qmv_wide and fused unpack+matmul qmm) and section 三 (an ABI probe guards
 * the native extension).
 *
 * Shared conventions of every entry point
 * ---------------------------------------
 *   x       fp16 [M][K] row-major activations (device memory).
 *   w       packed weights [N][row_bytes] (device memory), W[n][k] is the
 *           weight from input k to output n:
 *             bits = 1 or 2: uint32 words [N][K*bits/32]; code k of a row is
 *             bits (k*bits)%32 .. +bits-1 of word (k*bits)/32 (LSB first).
 *             bits = BQ_BITS_T5: uint8 [N][(K/gs)*ceil(gs/5)]; each group of
 *             gs weights owns ceil(gs/5) bytes (13 for gs=64, 26 for 128);
 *             code 5j+i of a group is base-3 digit i (least significant
 *             first) of the group's byte j; unused digits are 0; a byte
 *             above 242 is invalid (the result is then unspecified).
 *   scales  fp16 [N][K/gs], one per (output row, group along K).
 *   biases  fp16 [N][K/gs], or NULL where the call says so.  The weight is
 *           w = scale*q + bias (group-wise affine quantization).
 *   y       fp16 [M][N] row-major output, y[m][n] = sum_k x[m][k]*W[n][k],
 *           accumulated in fp32 and rounded to fp16 (nearest even) once.
 *           y is overwritten, never accumulated into.
 *   M, N, K sizes; K must be a positive multiple of group_size; N > 0.
 *   bits    1, 2, or BQ_BITS_T5 for the ternary format.
 *   group_size  64 or 128.
 *   stream  a hipStream_t (NULL = the default stream).  Every call only
 *           enqueues work on it and returns; there is no synchronization.
 *           The current HIP device has to be the stream's and the pointers'.
 *
 * Ownership: all pointers are device pointers owned by the caller.  The
 * library allocates nothing per call and keeps no mutable global state,
 * so calls from several host threads are safe.
 *
 * Errors: each entry point validates every argument before it launches
 * anything and returns BQ_OK (0) or a negative bq_status; bq_strerror()
 * names it.  A failed launch returns BQ_ERR_HIP.  Nothing aborts or throws
 * across this interface.
 *
 * Alignment: w needs 4-byte alignment (uint32 words for bits 1/2; dword
 * loads for t5).  The decode calls (qmv, qmv_wide, qmv_sym, t5_qmv,
 * t5_qmv_wide) read x, scales and biases as dwords and need them 4-byte
 * aligned (qmv_sym ignores the bias pointer).  bq_qmm and bq_t5_qmm stage x
 * with 16-byte loads that write LDS directly and need x 16-byte aligned,
 * scales and biases 2-byte aligned.  y needs 2-byte alignment everywhere
 * (bq_dequant uses 16-byte or dword stores when y allows them).  Fresh
 * allocations from hipMalloc or torch meet all of these.  t5 weights need
 * K to be a multiple of group_size only; rows need not be whole dwords
 * (bq_t5_repack alone needs K to be a multiple of 256).
 */
#ifndef BQ_H
#define BQ_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

#define BQ_ABI_VERSION 10
#define BQ_BITS_T5 0
#define BQ_MAX_WIDE_M 5

typedef enum bq_status {
  BQ_OK = 0,
  BQ_ERR_NULL = -1,       /* a required pointer is NULL */
  BQ_ERR_BITS = -2,       /* bits (or the logits dtype, or the cache format) not valid for this entry point */
  BQ_ERR_GROUP = -3,      /* group_size not 64 or 128 */
  BQ_ERR_SHAPE = -4,      /* N or K not positive, K % group_size != 0, K > 2^26,
                             or N * (packed row bytes) >= 2^30, or
                             N * (K / group_size) >= 2^29 (32-bit offsets), or
                             a decode call with K / group_size > 4092 (a
                             workgroup's scales must fit its LDS) */
  BQ_ERR_M = -5,          /* M outside the range this entry point accepts */
  BQ_ERR_ALIGN = -6,      /* a pointer is misaligned, or a t5 repack with K % 256 != 0 */
  BQ_ERR_HIP = -7,        /* the HIP runtime rejected a launch */
  BQ_ERR_FLAGS = -8,      /* bq_linear, bq_rope, bq_norm_rope, bq_kv_append,
                             bq_kv_append_norm, bq_kv_attn: flags holds
                             undefined bits (or a window without BQ_KV_CAUSAL) */
  BQ_ERR_WORKSPACE = -9,  /* bq_spec_decode_verify, bq_kv_fork / resize / compact:
                             workspace NULL or too small */
  BQ_ERR_SCRATCH = -10    /* bq_spec_decode_verify_noalloc: the call needs more than
                             BQ_SPEC_NOALLOC_SCRATCH_BYTES of scratch */
} bq_status;

/* bq_linear flags */
#define BQ_LINEAR_SYM 1   /* bias implied (-scale*ratio; t5: -scale), biases never read */
/* t5 calls of bq_linear with M >= BQ_T5_QMM_MIN_M take the fused qmm path
 * when the product has at least BQ_T5_QMM_MIN_TILES tiles of 32 x 64
 * outputs, or from BQ_T5_QMM_FEW_MIN_M rows at least BQ_T5_QMM_FEW_TILES
 * tiles (the small-M t5 product keeps four iterations of loads in flight,
 * which makes it faster than passes of five rows on fewer tiles than the
 * 1/2-bit product) */
#define BQ_T5_QMM_MIN_M 17
#define BQ_T5_QMM_MIN_TILES 64
#define BQ_T5_QMM_FEW_MIN_M 24
#define BQ_T5_QMM_FEW_TILES 16
/* 1/2-bit calls of bq_linear take bq_qmm when M >= BQ_QMM_MIN_M and the
 * product has at least BQ_QMM_MIN_TILES tiles of 32 x 64 outputs
 * (ceil(N/64)*ceil(M/32)), enough to occupy half the CUs */
#define BQ_QMM_MIN_M 17
#define BQ_QMM_MIN_TILES 128

typedef enum bq_route {
  BQ_ROUTE_QMV_WIDE = 1,  /* bits 1/2, stored bias: bq_qmv_wide per pass of <= 5 rows */
  BQ_ROUTE_QMV_SYM = 2,   /* bits 1/2, implied bias: bq_qmv_sym per pass of <= 5 rows */
  BQ_ROUTE_T5_WIDE = 3,   /* t5: bq_t5_qmv_wide per pass of <= 5 rows */
  BQ_ROUTE_T5_QMM = 4,    /* t5, M >= BQ_T5_QMM_MIN_M and tiles as below: one bq_t5_qmm */
  BQ_ROUTE_QMM = 5        /* bits 1/2, M and tiles as above: one bq_qmm */
} bq_route;

/* ABI version of the loaded library; callers must refuse to use a library
 * whose version differs from BQ_ABI_VERSION (the probe of section 三, but a
 * mismatch is an error here, never a silent fallback). */
int bq_abi_version(void);

/* Static, NUL-terminated description of a bq_status value. */
const char* bq_strerror(int status);

/* qmv -- section 二 path 1 (qmv_fast): bits 1 or 2, biases required, any
 * M >= 1.  Each activation row is an independent pass over W (W is read M
 * times); row m gives the same bits as a call with M = 1 on that row. */
int bq_qmv(const void* x, const void* w, const void* scales, const void* biases, void* y,
           int M, int N, int K, int bits, int group_size, void* stream);

/* qmv_wide -- section 二 path 2: bits 1 or 2, biases required,
 * 1 <= M <= 5; one read of W serves all M rows.  Row m gives the same
 * bits as bq_qmv on that row alone. */
int bq_qmv_wide(const void* x, const void* w, const void* scales, const void* biases, void* y,
                int M, int N, int K, int bits, int group_size, void* stream);

/* qmv_sym -- section 二 path 2, symmetric variant: bits 1 or 2,
 * 1 <= M <= 5; the bias is implied as -scale*(2^bits-1)/2 and the biases
 * argument is ignored and never read (it may be NULL).  Bit-identical to
 * bq_qmv_wide with an explicit fp16 bias equal to -scale*(2^bits-1)/2
 * whenever that value is exact in fp16. */
int bq_qmv_sym(const void* x, const void* w, const void* scales, const void* biases, void* y,
               int M, int N, int K, int bits, int group_size, void* stream);

/* t5_qmv -- section 二 path 3: bits must be BQ_BITS_T5, any M >= 1 (each
 * row an independent pass over W).  biases == NULL implies bias = -scale
 * (weights in {-s, 0, +s}) and no bias is read; non-NULL biases are read. */
int bq_t5_qmv(const void* x, const void* w, const void* scales, const void* biases, void* y,
              int M, int N, int K, int bits, int group_size, void* stream);

/* t5_qmv_wide -- section 二 path 3: as bq_t5_qmv with 1 <= M <= 5 and one
 * read of W for all rows. */
int bq_t5_qmv_wide(const void* x, const void* w, const void* scales, const void* biases, void* y,
                   int M, int N, int K, int bits, int group_size, void* stream);

/* t5_qmm -- section 二 path 3 (prefill, M > 16 intended; any M >= 1):
 * fused t5 unpack + matrix-core (MFMA, fp16 x fp16 -> fp32) product.  Each
 * t5 byte is unpacked once per weight tile; biases as in bq_t5_qmv. */
int bq_t5_qmm(const void* x, const void* w, const void* scales, const void* biases, void* y,
              int M, int N, int K, int bits, int group_size, void* stream);

/* qmm -- section 二 path 1 (1-bit prefill dequantizes to float16 and then
 * multiplies) and path 3 (the fused unpack + matrix multiply of t5): the
 * fused product for the uint32 formats, bits 1 or 2, any M >= 1 (prefill,
 * M > 16 intended).  Each code word is unpacked once per weight tile;
 * fp16 x fp16 -> fp32 on the matrix cores.  biases == NULL implies
 * -scale*(2^bits-1)/2 and no bias is read; non-NULL biases are read.  Each
 * weight enters the product as fp16_rne(scale*q + bias), as bq_dequant
 * writes it. */
int bq_qmm(const void* x, const void* w, const void* scales, const void* biases, void* y,
           int M, int N, int K, int bits, int group_size, void* stream);

/* K-split prefill -- section 二 path 3 (and path 1 for bits 1/2): the
 * products of bq_t5_qmm and bq_qmm with a caller-owned workspace.  At most
 * 32 rows give few output tiles (a 5120-column product has 80) for the
 * 256 CUs, so the K iterations of each tile are shared by up to 8
 * workgroups: each stores its fp32 partial tile to the workspace and a
 * second kernel adds the partials in a fixed order (same result every
 * call) and rounds once to fp16.  The sum order differs from the unsplit
 * product, so results may differ from bq_t5_qmm / bq_qmm in the last
 * bits (both are within the decode tolerance of the exact product).
 *
 * bq_qmm_workspace: *bytes := the workspace the split the library would
 * choose for (M, N, K, bits, group_size) needs; 0 when it would not split
 * (M > 32, or enough tiles).  bits 1, 2 or BQ_BITS_T5.  Host-only.
 *
 * bq_t5_qmm_ws / bq_qmm_ws: arguments as bq_t5_qmm / bq_qmm, plus
 * workspace (device memory, 16-byte aligned, or NULL) of workspace_bytes
 * bytes.  The split is taken only as far as the workspace holds its
 * partials; NULL or too small a workspace gives the unsplit product (no
 * error).  The workspace needs no initial contents; concurrent calls on
 * different streams must not share one.  BQ_ERR_ALIGN for a misaligned
 * workspace, else the errors of bq_t5_qmm / bq_qmm. */
int bq_qmm_workspace(int M, int N, int K, int bits, int group_size, size_t* bytes);
int bq_t5_qmm_ws(const void* x, const void* w, const void* scales, const void* biases, void* y,
                 int M, int N, int K, int bits, int group_size, void* workspace, size_t workspace_bytes,
                 void* stream);
int bq_qmm_ws(const void* x, const void* w, const void* scales, const void* biases, void* y,
              int M, int N, int K, int bits, int group_size, void* workspace, size_t workspace_bytes,
              void* stream);

/* dequant -- section 二 path 1 (1-bit prefill dequantizes to float16
 * before a matmul): y := fp16 [N][K], y[n][k] = fp16_rne(scale*q + bias)
 * computed exactly and rounded once.  x is ignored (may be NULL) and so is
 * M.  bits 1, 2 or BQ_BITS_T5.  biases == NULL implies -scale*(2^bits-1)/2
 * for bits 1/2 and -scale for t5. */
int bq_dequant(const void* x, const void* w, const void* scales, const void* biases, void* y,
               int M, int N, int K, int bits, int group_size, void* stream);

/* linear -- the routing of section 二 (the kernels are chosen by bits and
 * by the number of activation rows M) and section 三 (1/2-bit affine layers
 * in decode take the fast kernels): y = x * W^T for any M >= 1.
 *   bits 1/2: one bq_qmm when M >= BQ_QMM_MIN_M and the product has
 *             BQ_QMM_MIN_TILES tiles, else passes of up to 5 rows through
 *             bq_qmv_wide, or bq_qmv_sym when flags has BQ_LINEAR_SYM (each
 *             pass reads W once; M > 5 reads it ceil(M/5) times);
 *   t5:       bq_t5_qmm when M >= BQ_T5_QMM_MIN_M (the article's prefill
 *             rule, M > 16) and the product has BQ_T5_QMM_MIN_TILES tiles
 *             (or, from BQ_T5_QMM_FEW_MIN_M rows, BQ_T5_QMM_FEW_TILES
 *             tiles), else passes of up to 5 rows through bq_t5_qmv_wide.
 * Arguments as for the entry point a pass goes to; with BQ_LINEAR_SYM the
 * biases argument is ignored (may be NULL) and the bias is implied.
 * Results are those of the entry points the passes take; each pass is
 * validated before it launches, so an invalid argument fails before
 * anything runs.  Undefined flag bits: BQ_ERR_FLAGS. */
int bq_linear(const void* x, const void* w, const void* scales, const void* biases, void* y,
              int M, int N, int K, int bits, int group_size, int flags, void* stream);

/* linear with a workspace -- the routing of bq_linear, where a
 * workspace lets the fused prefill product split K (bq_t5_qmm_ws /
 * bq_qmm_ws): from BQ_T5_QMM_MIN_M (t5) or BQ_QMM_MIN_M (bits 1/2) rows
 * every product takes the fused route whatever its tile count, with
 * the workspace; fewer rows take the passes of bq_linear.  workspace ==
 * NULL: exactly bq_linear.  The fused route needs bq_qmm_workspace bytes
 * for its full split (less: a smaller split or none, see bq_qmm_ws);
 * workspace 16-byte aligned.  Arguments and errors otherwise as
 * bq_linear. */
int bq_linear_ws(const void* x, const void* w, const void* scales, const void* biases, void* y,
                 int M, int N, int K, int bits, int group_size, int flags, void* workspace,
                 size_t workspace_bytes, void* stream);

/* The route bq_linear takes for (M, N, bits, flags), a bq_route value, and
 * the number of kernel passes in *passes (may be NULL); BQ_ERR_M,
 * BQ_ERR_SHAPE (N < 1) or BQ_ERR_BITS for invalid arguments.  Host-only:
 * launches nothing. */
int bq_linear_route(int M, int N, int bits, int flags, int* passes);

/* sym detection -- section 二 path 2 (the symmetric variant applies when
 * bias = -scale * ratio holds): writes 1 to the device int *flag when every
 * stored fp16 bias equals -scale * ratio exactly (ratio (2^bits-1)/2, t5: 1),
 * else 0, asynchronously on stream.  scales and biases: fp16 [N][K/gs],
 * 2-byte aligned; flag: a caller-owned device int, 4-byte aligned.  A NaN
 * anywhere gives 0.  When it is 1, bq_qmv_sym (bq_linear with
 * BQ_LINEAR_SYM) gives the same bits as the affine call and skips the
 * bias read. */
int bq_sym_check(const void* scales, const void* biases, int N, int K, int bits, int group_size, int* flag,
                 void* stream);

/* t5 repack -- section 二, the t5 format (existing 1/2-bit weights are
 * repacked into t5 bytes): w holds uint32 code words [N][K*bits/32] (bits 1
 * or 2, the layout above); w_t5 receives t5 bytes [N][(K/gs)*ceil(gs/5)]
 * (the layout above).  Scales and biases stay as they are: s*q + b is the
 * same weight in both formats.  Writes 1 to the device int *flag when every
 * code is 0, 1 or 2 (the repack is exact), else 0; a code 3 is written as
 * digit 2.  K must be a multiple of 256 (whole dwords per t5 row); w, w_t5
 * and flag need 4-byte alignment.  Asynchronous on stream. */
int bq_t5_repack(const void* w, void* w_t5, int N, int K, int bits, int group_size, int* flag, void* stream);

/* speculative-decoding verification -- section 三 (spec_decode_verify:
 * comparing the draft tokens, counting the accepted length and producing the
 * correction token, fused into one kernel).  For each sequence b:
 *   t[i] = argmax over v of logits[b][i][v], i = 0..L (the largest value;
 *          equal values: the lowest v; -0 equals +0; a NaN is larger than
 *          every number and the first NaN wins);
 *   accepted[b] = the first i < L with draft[b][i] != t[i], else L;
 *   next_token[b] = t[accepted[b]] (the correction token, or the bonus token
 *          when every draft token is accepted);
 *   target_tokens[b][i] = t[i] when target_tokens is not NULL.
 * logits: [B][L+1][V] row-major, fp16 (BQ_DTYPE_F16) or fp32 (BQ_DTYPE_F32),
 * aligned to its element size; draft: int32 [B][L] (may be NULL when L = 0);
 * accepted, next_token: int32 [B]; target_tokens: int32 [B][L+1] or NULL;
 * all device memory owned by the caller, int arrays 4-byte aligned.
 * 1 <= B, 0 <= L <= BQ_SPEC_MAX_DRAFT, 1 <= V.
 * workspace: device memory of at least bq_spec_verify_workspace() bytes,
 * 8-byte aligned, all zero before its first use (e.g. hipMemset once);
 * every call leaves it zero again.  Calls that overlap in time on one
 * workspace race; give concurrent streams their own.  The library
 * allocates nothing.  Asynchronous on stream; one kernel launch. */
#define BQ_DTYPE_F16 1
#define BQ_DTYPE_F32 2
#define BQ_SPEC_MAX_DRAFT 1024

/* Workspace bytes bq_spec_decode_verify needs for B sequences of L draft
 * tokens (into *bytes).  Host-only. */
int bq_spec_verify_workspace(int B, int L, int V, size_t* bytes);

int bq_spec_decode_verify(const void* logits, int logits_dtype, const int* draft, int B, int L, int V,
                          int* accepted, int* next_token, int* target_tokens, void* workspace,
                          size_t workspace_bytes, void* stream);

/* bq_spec_decode_verify for callers that cannot allocate device memory (code
 * under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc): the same arguments and results without a workspace.  Its
 * scratch is a static device array of BQ_SPEC_NOALLOC_SCRATCH_BYTES inside
 * the library, one per GPU, held until the process ends; the call clears
 * what it uses (a kernel, no memset), then runs the verify kernel: two
 * launches, no allocation of any kind.  A call whose scratch,
 * bq_spec_verify_workspace(B, L), exceeds the array returns BQ_ERR_SCRATCH
 * before launching anything (e.g. B = 256 sequences of L = 15 draft tokens
 * need about 1.1 MB: 256 bytes per verified position, 128 per sequence).  Every call on a GPU shares that GPU's array: calls
 * that overlap in time on one GPU (several streams, several host threads)
 * race and give wrong results; serialize them.  Other errors as
 * bq_spec_decode_verify; BQ_ERR_HIP if the array's address cannot be
 * taken. */
#define BQ_SPEC_NOALLOC_SCRATCH_BYTES (2 * 1024 * 1024)
int bq_spec_decode_verify_noalloc(const void* logits, int logits_dtype, const int* draft, int B, int L, int V,
                                  int* accepted, int* next_token, int* target_tokens, void* stream);

/* ------------------------------------------------------------------------
 * Attention with a paged key/value cache held in 8 bits.
 *
 * The cache.  A page holds BQ_KV_PAGE = 64 tokens; every BQ_KV_BLOCK = 16
 * tokens of a page share one scale per head, for K and for V:
 *   k, v                 uint8 [layers][num_pages][kv_heads][64 * head_dim]
 *   k_scales, v_scales   fp32  [layers][num_pages][kv_heads][4]
 * value = scale * code.  format BQ_KV_I8: the code is an integer -127..127,
 * held as the byte code + 128; BQ_KV_E4M3: the byte is an OCP e4m3 number.
 * The bytes of a page lie in the order in which the matrix instructions take
 * them:
 *   K  [i: 4][c: head_dim/64][g: 4][t: 16][j: 16]  token 16i + t, dim 64c + 16g + j
 *   V  [n: head_dim/16][g: 4][d: 16][i: 4][j: 4]   token 16i + 4g + j, dim 16n + d
 * head_dim 64, 128, 192 or 256; kv_heads 1..1024; layers 1..4096; scales are
 * not negative; codes and scales 16-byte aligned.  layer selects one layer of
 * the arrays; page calls work on all.
 *
 * The batch of a call.  Sequence b has the rows cu[b] .. cu[b+1] - 1 of the
 * call's packed row arrays (cu: int32 [batch + 1], rising, cu[batch] =
 * total), holds lens[b] tokens, and its token t lies in page
 * table[b][t / 64] (int32 [batch][max_pages]).  Its rows are its last
 * tokens: row i of n stands at position lens[b] - n + i.  All three arrays
 * are device memory, read by the kernels only, so a captured call follows
 * what they hold at each replay.  Entries that do not fit (cu past total,
 * lens past 64 * max_pages, a page id outside 0 .. num_pages - 1) are never
 * followed: such rows, tokens and pages count as absent.
 *
 * Row arrays are fp16 [total][heads][head_dim] with a stride in elements
 * from row to row (at least heads * head_dim, a multiple of 8); pointers
 * 16-byte aligned.  total == 0 is a call that does nothing (its row arrays
 * may be NULL). */
#define BQ_KV_PAGE 64
#define BQ_KV_BLOCK 16
#define BQ_KV_I8 1
#define BQ_KV_E4M3 2
#define BQ_KV_MAX_PAGES (1 << 24)

typedef struct bq_kv_cache {
  void* k;
  void* v;
  float* k_scales;
  float* v_scales;
  int layers, num_pages, kv_heads, head_dim, format;
} bq_kv_cache;

/* rope -- rotary positions with several axes (time, height, width of images
 * and video; one axis for text).  Pair r of the first rot_dim dimensions of
 * every head turns by a = pos[axis[r]][token] * inv_freq[r]:
 *   y1 = x1 cos a - x2 sin a,  y2 = x2 cos a + x1 sin a,
 * x1, x2 = dimensions r and r + rot_dim/2, or 2r and 2r + 1 with
 * BQ_ROPE_ADJACENT; dimensions past rot_dim pass through.
 * x, y: rows as above, y may be x (with the same stride); head_dim a multiple of 16 up to
 * 1024, rot_dim a multiple of 16 up to head_dim (0: nothing turns, the
 * arrays may be NULL); up to 2^24 tokens fit any launch, a call that does not
 * is BQ_ERR_SHAPE; pos int32 [axes][tokens], inv_freq fp32
 * [rot_dim/2], axis int32 [rot_dim/2] (NULL: all 0; values outside 0 ..
 * axes - 1 are brought into it), 1 <= axes <= BQ_ROPE_MAX_AXES.  The angle
 * is exact to 2^-20 turns at any position.  Undefined flag bits:
 * BQ_ERR_FLAGS. */
#define BQ_ROPE_ADJACENT 1
#define BQ_ROPE_MAX_AXES 8
int bq_rope(const void* x, void* y, long long x_stride, long long y_stride, int tokens, int heads, int head_dim,
            const int* pos, const float* inv_freq, const int* axis, int rot_dim, int axes, int flags, void* stream);

/* kv_append -- rotates the new rows' k (and q, when q is not NULL, into
 * q_out) as bq_rope does and writes k and v to the cache as the last tokens
 * of their sequences; lens already counts them.  Every block that takes a
 * new token gets the scale
 *   max(largest |new value| / 127 (e4m3: / 448), its scale if it holds older tokens),
 * new values are coded as rne(value / scale), codes of the block's older
 * tokens are brought to the new scale (unchanged when it did not grow), and
 * tokens of the block past lens are cleared.  Infinities do not count for
 * the scale and are held as the largest code, NaN as 0.  Writing the same
 * rows again (after a rejected draft, say) replaces them.  Pages that
 * several sequences share must not be written: bq_kv_fork and bq_kv_resize
 * never leave a partly filled page shared. */
int bq_kv_append(const bq_kv_cache* cache, int layer, const void* k, const void* v, long long k_stride,
                 long long v_stride, const void* q, void* q_out, long long q_stride, long long q_out_stride,
                 int q_heads, const int* cu, const int* lens, const int* table, int batch, int max_pages, int total,
                 const int* pos, const float* inv_freq, const int* axis, int rot_dim, int axes, int flags,
                 void* stream);

/* kv_read -- the values held for the last tokens of each sequence, as
 * contiguous fp16 [total][kv_heads][head_dim] (one rounding of
 * scale * code); rows that no page holds are zero. */
int bq_kv_read(const bq_kv_cache* cache, int layer, void* k, void* v, const int* cu, const int* lens, const int* table,
               int batch, int max_pages, int total, void* stream);

/* kv_attn -- out[row][h] = sum_j p_j v_j / sum_j p_j, p_j = exp(scale *
 * q[row][h] . k_j), over the tokens j of the row's sequence that the row
 * sees, with the key/value head h / (q_heads / kv_heads).  With BQ_KV_CAUSAL
 * a row at position n sees j <= n, and with window > 0 only j > n - window;
 * without it every row sees all lens[b] tokens (an encoder's states).  A row
 * that sees nothing gives zeros; tokens that no page holds are not seen.
 * Scores, sums and outputs in fp32, codes exact.  Up to 16 rows of a
 * key/value head and sequence on average (rows times q_heads / kv_heads; 32
 * where head_dim <= 128) the probabilities, times V's scale, enter the product
 * with V as sums of two fp16 numbers; beyond that they are rounded to fp16
 * once and divided by the sum of the rounded ones.  What a term loses is at
 * most 2^-22 (rounded once: 2^-11) of it, or 2^-25 of the smallest scale
 * above 0 of the term's page, or 2^-31 of the page's largest term among the
 * rows taken together, whichever is most (times the code; a row's largest
 * probability taken as 1).
 *
 * workspace (device memory, 16-byte aligned, or NULL): lets the tokens of a
 * long sequence be shared by several workgroups.  Its first
 * BQ_KV_ATTN_COUNTER_BYTES must be zero before its first use; every call
 * leaves them zero again.  bq_kv_attn_workspace gives the size of the full
 * split; less gives a smaller split or none, with results that may differ
 * in the last bits.  Calls that overlap in time must not share a workspace.
 * The same bits on every call with the same arguments; one launch, two where
 * many rows are split (more past 32768 tiles of a head).  Rows of a call
 * whose cu falls somewhere may be left unwritten. */
#define BQ_KV_CAUSAL 1
#define BQ_KV_ATTN_COUNTER_BYTES 65536
int bq_kv_attn_workspace(const bq_kv_cache* cache, int q_heads, int batch, int total, size_t* bytes);
int bq_kv_attn(const bq_kv_cache* cache, int layer, const void* q, void* out, long long q_stride,
               long long out_stride, int q_heads, const int* cu, const int* lens, const int* table, int batch,
               int max_pages, int total, float scale, int window, int flags, void* workspace, size_t workspace_bytes,
               void* stream);

/* Pages.  table int32 [rows][max_pages], lens int32 [rows], refs int32
 * [num_pages]: the number of table entries that hold a page; a page is free
 * when it is 0.  Free pages are taken lowest first, in the order of the
 * call's rows.  All arrays are device memory and are updated there; status
 * (int32 [2], device) receives
 *   status[0]  0 done; -1 an argument array holds something invalid; n > 0:
 *              n more free pages are needed.  Unless 0, nothing was changed.
 *   status[1]  pages copied.
 * workspace: bq_kv_pages_workspace bytes, 16-byte aligned, no initial
 * contents needed; BQ_ERR_WORKSPACE when NULL or smaller.
 *
 * kv_fork    row dst[i] becomes a copy of row src[i] (n of each, int32,
 *            device; dst rows distinct and of length 0): whole pages are
 *            shared, a partly filled last page is copied.  1 <= n <= rows.
 * kv_resize  row i gets the length want[i] (int32 [rows], -1: as it is).
 *            Shorter: pages past it are let go, and a last page that is then
 *            partly filled and still shared is copied.  Longer: pages are
 *            taken; their contents are undefined until written.
 *            rows * max_pages < 2^31.
 * kv_compact moves pages so that those in use have the lowest ids: the ids in
 *            use from their number on, ascending, go to the free ids below
 *            it, ascending; table and refs follow.
 * kv_copy_pages  copies pages src[i] to dst[i] (int32 [n], device) over all
 *            layers; pairs outside 0 .. num_pages - 1 are skipped.  No page
 *            may be both, or twice in dst. */
int bq_kv_pages_workspace(const bq_kv_cache* cache, int rows, size_t* bytes);
int bq_kv_fork(const bq_kv_cache* cache, int* table, int* lens, int* refs, int rows, int max_pages, const int* src,
               const int* dst, int n, int* status, void* workspace, size_t workspace_bytes, void* stream);
int bq_kv_resize(const bq_kv_cache* cache, int* table, int* lens, int* refs, int rows, int max_pages, const int* want,
                 int* status, void* workspace, size_t workspace_bytes, void* stream);
int bq_kv_compact(const bq_kv_cache* cache, int* table, int* refs, int rows, int max_pages, int* status,
                  void* workspace, size_t workspace_bytes, void* stream);
int bq_kv_copy_pages(const bq_kv_cache* cache, const int* src, const int* dst, int n, void* stream);

/* ------------------------------------------------------------------------
 * A decoding step with a tree of drafted tokens, over the cache above.
 *
 * The tree of sequence b is its rows cu[b] .. cu[b+1] - 1: row 0 the last
 * token decided, every other row a drafted token behind its parent row.
 * parent, token and target are int32 [total] in device memory; parent[row] is
 * a row's number in its sequence, smaller than the row's own, or -1: a row
 * behind the context itself.  Any other value counts as -1.  Up to
 * BQ_TREE_MAX_ROWS rows of a sequence.  As above, arrays are read by the
 * kernels only, and what does not fit is never followed. */
#define BQ_TREE_MAX_WORDS 16
#define BQ_TREE_MAX_ROWS 1024

/* norm_rope -- a norm of each head's row and the rotation of bq_rope in one
 * pass: x * weight / sqrt(mean(x^2) + eps) over the head's dimensions, then
 * turned; fp32 inside, rounded once.  weight fp32 [head_dim], eps >= 0 and
 * finite (BQ_ERR_SHAPE); the rest as bq_rope, rot_dim 0 included (a norm
 * alone).  y may be x.  A row of zeros with eps 0, and a row that holds an
 * infinity or no number, give what the formula gives.
 *
 * kv_append_norm -- bq_kv_append with k normed by k_weight and q by q_weight
 * ahead of the rotation (each fp32 [head_dim], or NULL: not normed). */
int bq_norm_rope(const void* x, void* y, long long x_stride, long long y_stride, int tokens, int heads, int head_dim,
                 const float* weight, float eps, const int* pos, const float* inv_freq, const int* axis, int rot_dim,
                 int axes, int flags, void* stream);
int bq_kv_append_norm(const bq_kv_cache* cache, int layer, const void* k, const void* v, long long k_stride,
                      long long v_stride, const void* q, void* q_out, long long q_stride, long long q_out_stride,
                      int q_heads, const int* cu, const int* lens, const int* table, int batch, int max_pages,
                      int total, const float* k_weight, const float* q_weight, float eps, const int* pos,
                      const float* inv_freq, const int* axis, int rot_dim, int axes, int flags, void* stream);

/* kv_attn_sinks -- bq_kv_attn with BQ_KV_CAUSAL, where a row at position n
 * sees beside the window's tokens the first `sinks` of its sequence: j <= n
 * and (j > n - window or j < sinks).  window 0: all j <= n.  Pages that no row
 * sees are not read.
 *
 * kv_attn_tree -- bq_kv_attn where each sequence's rows are a tree: row i of n
 * sees the rows j of its sequence whose bit j % 64 of mask[row][j / 64] is set
 * (its own among them, if it is to see itself; bits from n on do not count),
 * and the context, the lens[b] - n tokens ahead of the tree: all of it, or
 * with window > 0 the last window - (rows it sees of the tree) of its tokens
 * and the first `sinks`.  mask uint64 [total][mask_words], 8-byte aligned, 1
 * <= mask_words <= BQ_TREE_MAX_WORDS; rows past 64 * mask_words of a sequence
 * are seen by none.  A row that sees nothing gives zeros.  bq_tree_plan makes
 * the masks of a tree; a mask need not be one of a tree.  The sinks end with the
 * context: rows of the tree are seen as the mask says and not otherwise.  A
 * chain over a context shorter than `sinks`, longer than the window and with the
 * masks of bq_tree_plan, so sees fewer of its own first tokens than the same
 * rows in bq_kv_attn_sinks, until they are context.
 *
 * Both: arguments, workspace, numerics and errors otherwise as bq_kv_attn
 * (sinks < 0: BQ_ERR_SHAPE). */
int bq_kv_attn_sinks(const bq_kv_cache* cache, int layer, const void* q, void* out, long long q_stride,
                     long long out_stride, int q_heads, const int* cu, const int* lens, const int* table, int batch,
                     int max_pages, int total, float scale, int window, int sinks, void* workspace,
                     size_t workspace_bytes, void* stream);
int bq_kv_attn_tree(const bq_kv_cache* cache, int layer, const void* q, void* out, long long q_stride,
                    long long out_stride, int q_heads, const int* cu, const int* lens, const int* table, int batch,
                    int max_pages, int total, const void* mask, int mask_words, float scale, int window, int sinks,
                    void* workspace, size_t workspace_bytes, void* stream);

/* tree_plan -- of every row the rows that it sees, itself and those above it
 * (with window > 0 only the nearest `window` of them), as mask uint64
 * [total][mask_words] for bq_kv_attn_tree, and its position for the rotation,
 * pos int32 [total]: lens[b] - n (at least 0) + the number of rows above it.
 * mask or pos may be NULL (not both).  Rows past 64 * mask_words of a sequence see
 * nothing and stand at its first row's position.
 *
 * tree_accept -- the path that the target tokens take from row 0 on: of the
 * rows whose parent is the last row taken, the first whose token is that
 * row's target is taken next (rows behind it in the sequence only).  target[row]
 * is the token that the target model has after the row: its most likely one
 * (bq_logprobs) or one that the caller drew.  For each sequence:
 *   path [batch][max_path]  the rows taken, rising, then -1; path[0] = 0
 *   kept [batch]            their number, at most max_path
 *   next_token [batch]      the target behind the last of them
 *   want [batch]            lens[b] - n + kept, the length for bq_kv_resize (of
 *                           fewer tokens than rows: kept, lens[b] at most)
 * A sequence without rows: kept 0, next_token -1, want lens[b].  Rows past
 * BQ_TREE_MAX_ROWS are never taken.  1 <= max_path <= BQ_TREE_MAX_ROWS.
 *
 * kv_keep -- over all layers, keys and values of the rows path[b][i], i <
 * kept[b], go to the places of the rows i: with bq_kv_resize to `want` they
 * are then the sequence's last tokens.  A block that takes a token gets the
 * largest of its own scale and its tokens' scales, and the codes of tokens that
 * had a smaller one are brought to it (rne).  So tokens of the block that no
 * other replaces keep their values only where its scale did not grow; where it
 * did, they are rounded once more, by half a step of the new scale at most, as
 * kv_append rounds the older tokens of a block.  Blocks that take no token stay
 * as they are.  lens still counts all n rows.  A sequence whose
 * path does not rise from row to row inside 0 .. n - 1, or that holds fewer
 * tokens than rows, is left as it is; a row whose page, or whose place's, is
 * missing is not moved.  Pages that are written must not be
 * shared (as for bq_kv_append). */
int bq_tree_plan(const int* parent, const int* cu, const int* lens, int batch, int total, int mask_words, int window,
                 void* mask, int* pos, void* stream);
int bq_tree_accept(const int* target, const int* token, const int* parent, const int* cu, const int* lens, int batch,
                   int total, int max_path, int* path, int* kept, int* next_token, int* want, void* stream);
int bq_kv_keep(const bq_kv_cache* cache, const int* cu, const int* lens, const int* table, int batch, int max_pages,
               const int* path, int max_path, const int* kept, void* stream);

/* logprobs -- of each row of logits [rows][V] (fp16 or fp32; row_stride in
 * elements, at least V; aligned to the element) under p = softmax(row):
 *   logprob [rows][count]       log p of the given tokens (int32 [rows][count];
 *                               a token outside 0 .. V - 1: -inf)
 *   entropy [rows]              -sum p log p
 *   top_tokens, top_logprobs    the `top` largest, [rows][top], in
 *   [rows][top]                 bq_spec_decode_verify's order: equal values,
 *                               lowest token first; -0 equals 0; NaN first
 * fp32 and int32 arrays, 4-byte aligned; tokens and logprob may be NULL with
 * count 0, entropy may be NULL, top_tokens and top_logprobs with top 0; at
 * least one is asked for.  Sums in fp32, one read of the logits.  Logits of
 * -inf have probability 0; with top > V the places behind V hold token -1 and
 * -inf.  A row with a NaN or +inf, and one of -inf alone, has no
 * probabilities: its logprob, entropy and top_logprobs are NaN, its top_tokens
 * are by value all the same.  0 <= count <= BQ_LOGPROBS_MAX_COUNT, 0 <= top <=
 * BQ_LOGPROBS_MAX_TOP, 0 <= rows < 2^24, 1 <= V < 2^28.
 * workspace: as bq_kv_attn's (its first BQ_LOGPROBS_COUNTER_BYTES zero before
 * the first use, zero again after every call; 16-byte aligned, NULL allowed):
 * it lets several workgroups share a row, bq_logprobs_workspace gives the size
 * for as many as the library would take, less gives fewer.  Calls that overlap
 * in time must not share one; one that serves bq_kv_attn serves here too.
 * Results may differ in the last bits by the number of workgroups, and are the
 * same on every call with the same arguments.  One launch. */
#define BQ_LOGPROBS_MAX_TOP 64
#define BQ_LOGPROBS_MAX_COUNT 1024
#define BQ_LOGPROBS_COUNTER_BYTES 65536
int bq_logprobs_workspace(int rows, int V, int logits_dtype, int top, size_t* bytes);
int bq_logprobs(const void* logits, int logits_dtype, long long row_stride, int rows, int V, const int* tokens,
                int count, float* logprob, float* entropy, int top, int* top_tokens, float* top_logprobs,
                void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* BQ_H */
