/*
 * fp4.h -- C ABI of libfp4: FP4 (E2M1) block-scaled quantisation and matrix
 * multiply on AMD Instinct MI355X (gfx950).
 *
 * The operation, as the sources state it:
 *   - E2M1 elements {0, ±0.5, ±1, ±1.5, ±2, ±3, ±4, ±6}, one scale per block
 *     chosen so the block's largest magnitude maps to 6 (Ultralytics glossary
 *     "FP4", "How FP4 works");
 *   - MXFP4: 32-value blocks, power-of-two E8M0 scale; NVFP4: 16-value blocks,
 *     E4M3 scale plus one FP32 per-tensor scale (NVFP4 video transcript,
 *     prism.simon-ai.net; glossary "How FP4 works");
 *   - the GEMM accumulates in FP32 and multiplies by the product of the scales,
 *     C = (A_fp4 * B_fp4) * (scaleA * scaleB) ("Rubin FP4 GEMM deep dive",
 *     yfxerp.com, §1.1, §3.1, §4.2);
 *   - two FP4 values per byte with an explicitly fixed order, scales stored in
 *     the order the kernel tiles read them (same page, §4.2, §5.2);
 *   - weights and activations may take different precisions, FP8 activations
 *     beside FP4 weights (same page, §3.4), here MXFP8: E4M3 elements under
 *     the MXFP4 block scales (§3.1 names MXFP8 among the MX formats).
 *
 * Conventions for every entry point:
 *   - All data pointers are DEVICE pointers (hipMalloc'd or equivalent) unless
 *     stated otherwise; `stream` is a hipStream_t passed as void* (NULL = the
 *     null stream).  Every call is asynchronous on `stream`: it enqueues work
 *     and returns; nothing is copied to or from the host, no call synchronises.
 *   - The caller owns and allocates every buffer, workspace included.  The
 *     library never allocates or frees memory and keeps no global mutable
 *     state, with one exception: fp4_quantize_noalloc's scratch array, a
 *     static device array of 256 bytes on each GPU the library runs on.
 *   - Argument errors return a negative fp4_status before any HIP call is made,
 *     so they are reported synchronously and leave the stream untouched.  A
 *     failed kernel launch returns FP4_ERR_HIP.  Faults inside a kernel surface
 *     at the caller's next synchronisation.  Debug mode (fp4_set_debug,
 *     FP4_DEBUG) adds checks that make HIP calls and synchronise.
 *   - Format, dtype, output, activation and operation arguments are declared
 *     int and take the values of the enums below.  A C enum's underlying type
 *     is up to the compiler (-fshort-enums makes it one byte), while int is the
 *     same for every compiler and for foreign-function callers; any other value
 *     is refused with FP4_ERR_FMT, FP4_ERR_DTYPE or FP4_ERR_FLAGS.
 *   - Matrices are row-major.  A quantised matrix of `rows` x `K` values is
 *       codes:  rows * K/2 bytes; element k of a row is in byte k/2, bits 0-3
 *               for even k and bits 4-7 for odd k; a code is sign<<3 | magnitude
 *               with magnitude 0..7 -> 0, 0.5, 1, 1.5, 2, 3, 4, 6;
 *       scales: fp4_scale_bytes(fmt, rows, K) bytes in the tiled layout below;
 *       tensor scale (NVFP4 only): one FP32 in device memory.
 *     MXFP8 codes are rows * K bytes instead, one E4M3 byte per element
 *     (sign<<7 | exponent<<3 | mantissa, bias 7, largest value 448; the NaN
 *     patterns 0x7F / 0xFF are never written and not supported as input).
 *   - Element value: MXFP4  E2M1(code) * 2^(scale_byte - 127);
 *                    MXFP8  E4M3(code) * 2^(scale_byte - 127);
 *                    NVFP4  E2M1(code) * E4M3(scale_byte) * tensor_scale.
 *
 * Tiled scale layout (identical for A and B operands; both are "rows x K").
 *   Scales are grouped in tiles of 32 rows x 256 K values, stored row-tile
 *   major: tile (rt, kt) starts at byte T * (rt * ceil(K/256) + kt), with tile
 *   size T = 256 (MXFP4 and MXFP8: 8 blocks of 32) or 512 (NVFP4: 16 blocks
 *   of 16).
 *   Inside a tile, row i (0..31) and 32-value K chunk c (0..7) belong to lane
 *   L = 32 * (c % 2) + i and sub-step s = c / 2 -- the lane order of the 32x32
 *   matrix-core operand, where lane 32*j + i carries row i's chunk j of each
 *   64-value K sub-step:
 *     MXFP4, MXFP8: lane L owns bytes 4L..4L+3; byte 4L + s is the chunk's
 *            E8M0 scale;
 *     NVFP4: lane L owns bytes 8L..8L+7; bytes 8L + 2s and 8L + 2s + 1 are the
 *            E4M3 scales of the chunk's first and second 16-value block.
 *   One dword (MXFP4) or two (NVFP4) per lane thus carry a wavefront's scales
 *   for four K sub-steps.  Bytes of rows >= `rows` or of blocks past K are
 *   padding: the quantiser writes them as 0, and the GEMMs rely on that (a
 *   zero scale makes the codes read past the end of K contribute nothing), so
 *   hand-built scale buffers must keep padding bytes 0.  E8M0 byte 0xFF (NaN)
 *   is never produced and not supported as input.
 */
#ifndef FP4_H_
#define FP4_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Block format. */
enum fp4_fmt {
    FP4_MXFP4 = 0,     /* 32-blocks, E8M0; exponent = smallest e with amax <= 6*2^e */
    FP4_NVFP4 = 1,     /* 16-blocks, E4M3 (bias 7, max 448) + FP32 tensor scale      */
    FP4_MXFP4_OCP = 2, /* 32-blocks, E8M0; exponent = floor(log2 amax) - 2, saturate */
    FP4_MXFP8 = 3,     /* 32-blocks, E8M0, E4M3 elements; smallest e with amax <= 448*2^e */
    FP4_MXFP8_OCP = 4  /* 32-blocks, E8M0, E4M3 elements; floor(log2 amax) - 8, saturate */
};

/* Element type of unquantised inputs and of outputs. */
enum fp4_dtype { FP4_F32 = 0, FP4_BF16 = 1 };

/* Operation selector for fp4_workspace_size. */
enum fp4_op { FP4_OP_QUANTIZE = 0, FP4_OP_GEMM = 1, FP4_OP_GEMM_GROUPED = 2 };

/* Output of fp4_gemm_ex: FP32 or BF16 (the fp4_dtype values), or the product
 * quantised again to MXFP4 along N (ceil or OCP exponent rule, as
 * FP4_MXFP4 / FP4_MXFP4_OCP) or to NVFP4 along N under a given tensor scale. */
enum fp4_out { FP4_OUT_F32 = 0, FP4_OUT_BF16 = 1, FP4_OUT_MXFP4 = 2, FP4_OUT_MXFP4_OCP = 3, FP4_OUT_NVFP4 = 4 };

/* Activation of fp4_gemm_ex. */
enum fp4_act { FP4_ACT_NONE = 0, FP4_ACT_RELU = 1 };

/* Flags for fp4_quantize. */
#define FP4_TS_GIVEN 1u /* NVFP4: read the tensor scale from *tensor_scale instead of computing it */
/* More flags for fp4_quantize_ex. */
#define FP4_Q_SR 2u     /* round the elements stochastically (as fp4_quantize_sr)          */
#define FP4_Q_2D 4u     /* NVFP4 only: one block scale per 16 x 16 patch (2-D scaling)      */

enum fp4_status {
    FP4_OK = 0,
    FP4_ERR_NULL = -1,      /* a required pointer is NULL                          */
    FP4_ERR_SHAPE = -2,     /* negative size, K not a multiple of the block, ...   */
    FP4_ERR_ALIGN = -3,     /* a pointer is not aligned as documented              */
    FP4_ERR_FMT = -4,       /* unknown fmt, or fmt not supported by this operation */
    FP4_ERR_DTYPE = -5,     /* unknown dtype                                       */
    FP4_ERR_WORKSPACE = -6, /* workspace missing or smaller than required          */
    FP4_ERR_HIP = -7,       /* a HIP launch failed                                 */
    FP4_ERR_FLAGS = -8,     /* unknown flag bits                                   */
    FP4_ERR_BOUNDS = -9     /* debug mode only: a buffer is not memory of the      */
                            /* current device or smaller than the call needs, or   */
                            /* a group offset or token index is out of range       */
};

/* Debug mode, for callers hunting a fault or a wrong result: on when the
 * environment variable FP4_DEBUG is set to anything but "0" when the library
 * is first used, or after fp4_set_debug(1).  Then every entry point, after its argument checks:
 *   - checks that each buffer it reads or writes lies wholly inside one device
 *     allocation of the current device (hipMemGetAddressRange; a caching
 *     allocator's block counts as one allocation), else FP4_ERR_BOUNDS;
 *   - fp4_gemm_grouped waits for the stream, copies group_off and row_idx to
 *     the host and checks them as documented there, else FP4_ERR_BOUNDS;
 *   - waits for its kernels (hipStreamSynchronize), so that a launch or
 *     execution error is returned by the call that caused it (FP4_ERR_HIP).
 * The checks make HIP calls and synchronise, and the grouped check allocates
 * host memory; none of this happens with debug mode off.  Returns the previous
 * setting (0 or 1).  Host-only; the setting is process-wide. */
int fp4_set_debug(int on);

/* Size in bytes of the tiled scale buffer of a rows x K matrix, or a negative
 * fp4_status for an invalid fmt or shape.  Host-only, no HIP call. */
int64_t fp4_scale_bytes(int fmt, int64_t rows, int64_t K);

/* Workspace bytes an operation needs (0 if none).  For FP4_OP_QUANTIZE, M is
 * the row count; for FP4_OP_GEMM_GROUPED, E is the expert count and M the total
 * routed rows.  NVFP4 quantisation that computes its own tensor scale needs 16
 * bytes (the running amax and two workgroup counters); fp4_gemm returns 0.
 * FP4_OP_GEMM_GROUPED returns the size of an OPTIONAL workspace (MXFP4
 * formats; 0 for NVFP4): given one, fp4_gemm_grouped first copies the routed
 * token rows into expert order there, which makes the GEMM faster; it needs
 * no zero-fill (it holds no control words).  Operations keep their control words at the start of the
 * workspace.  A workspace must be zero-filled once before its first use; every
 * call leaves the control words zero again when its work on the stream
 * completes, so one zero-filled workspace of the largest size needed serves
 * any sequence of calls, of these and of the operators below; all keep what
 * else they leave there behind the first 2 KB.  The one exception is
 * fp4_gemm_grouped's copy, which begins at the workspace's first byte: an
 * operation with control words needs them zero-filled again after it.  Calls that
 * share one workspace must be ordered (same stream, or events); calls that
 * overlap on one workspace race.  Host-only. */
size_t fp4_workspace_size(int op, int fmt, int64_t M, int64_t N, int64_t K, int32_t E);

/* Quantise a rows x K matrix x (K contiguous) of `in_dtype` (FP32 or BF16).
 *   Per block: MXFP4 picks an E8M0 exponent from the block's largest magnitude
 *   (MXFP8: the same rules with 448 in place of 6, elements y = x * 2^-e
 *   rounded to the nearest E4M3 value, ties to even, saturating at 448);
 *   NVFP4 takes r = (amax_block / 6) / tensor_scale, rounds it to E4M3 (nearest
 *   even, saturating at 448), and divides by d = E4M3(r) * tensor_scale (FP32).
 *   Each element is then rounded to the nearest E2M1 value, ties to even,
 *   saturating at 6; the sign bit is copied (-0 gives code 8).
 *   NVFP4 tensor scale: unless flags has FP4_TS_GIVEN, computed over the whole
 *   matrix as s_t = amax / 2688 (6 * 448), s_t = 1 for an all-zero matrix and
 *   s_t >= FLT_MIN, and written to *tensor_scale.  With FP4_TS_GIVEN the caller's
 *   value is used (it must be a positive, finite, normal FP32).
 *   (Sources: glossary "How FP4 works"; NVFP4 video transcript.)
 * Requirements: K % bs == 0 (32 for MXFP4 and MXFP8, 16 for NVFP4); x 16-byte
 *   aligned; codes 4-byte (MXFP8: 8-byte) and block_scales 4-byte aligned.  tensor_scale must be non-NULL for NVFP4 and
 *   is ignored for MXFP4.  NVFP4 without FP4_TS_GIVEN needs a workspace of
 *   fp4_workspace_size(FP4_OP_QUANTIZE, ...) bytes; otherwise workspace may be NULL.
 *   (Inputs of at most 256 KB take a single launch in which every workgroup
 *   reduces the maximum itself and the workspace is left untouched; up to 1 MB,
 *   a single launch whose workgroups exchange the maximum through the
 *   workspace and wait for each other (a bounded wait, after which a
 *   workgroup reduces the whole maximum itself); larger ones reduce across
 *   workgroups through the workspace, then quantise.  All give the same
 *   bits.  A test hook: the environment variable FP4_TEST_NV_GRID_SPIN, a
 *   positive count, caps that wait, so that tests reach the path of a
 *   workgroup that stops waiting.)
 * rows == 0 or K == 0 is a no-op. */
int fp4_quantize(const void* x, int fmt, uint8_t* codes, uint8_t* block_scales, float* tensor_scale,
                 int64_t rows, int64_t K, int in_dtype, unsigned flags, void* workspace,
                 size_t workspace_bytes, void* stream);

/* fp4_quantize for callers that cannot allocate device memory: code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc.
 * Same arguments, rules, errors and bits as fp4_quantize (flags:
 * FP4_TS_GIVEN only), without the workspace: where fp4_quantize would use one
 * (NVFP4 computing its own tensor scale over more than 256 KB of input), the
 * running maximum and workgroup counters live in a scratch array the library
 * holds, a static device array of 256 bytes on each GPU (held until the
 * process ends).  The call allocates nothing and calls no allocating
 * routine.
 *   The first call on a device looks the array up for that device (which must
 *   be current) and enqueues a one-workgroup kernel on `stream` that clears
 *   it; every later call leaves its control words zero when its work
 *   completes.
 *   All calls on one GPU share that GPU's array: calls that may run at the
 *   same time on one GPU (different streams, no ordering between them) race
 *   and give wrong tensor scales.  Order them, or use fp4_quantize with a
 *   workspace per stream.
 * Errors: as fp4_quantize; FP4_ERR_WORKSPACE if the operation needed more
 * than the array's 256 bytes (no format needs more than 16 today);
 * FP4_ERR_HIP if the array cannot be located on the current device or the
 * clearing kernel fails to launch. */
int fp4_quantize_noalloc(const void* x, int fmt, uint8_t* codes, uint8_t* block_scales, float* tensor_scale,
                         int64_t rows, int64_t K, int in_dtype, unsigned flags, void* stream);

/* fp4_quantize with stochastic rounding of the elements (NVFP4 video
 * transcript, the training recipe's fourth part: a value between two
 * representable points goes up with probability equal to its distance from
 * the lower one, so the expectation is kept -- meant for gradients).  The
 * block and tensor scales are chosen exactly as by fp4_quantize; only the
 * E2M1 rounding of each scaled value y changes:
 *   lo = the largest grid value <= |y| (|y| >= 6 gives 6), hi the next one;
 *   the code is hi iff u * (hi - lo) < |y| - lo, with u = (w >> 8) * 2^-24 and
 *   w the element's 32-bit random word; the sign bit is copied.
 * Random words: Philox4x64-10 (Salmon et al., "Parallel random numbers: as
 * easy as 1, 2, 3", SC 2011) with key (seed, 0); element i of the matrix
 * (row-major, i = r * K + k) takes word (i mod 8) / 2 of the block with
 * counter (i / 8, 0, 0, 0), its low 32 bits for even i.  The result is a
 * function of (x, seed) alone.  FP4 formats only (MXFP8: FP4_ERR_FMT).
 * Arguments and errors as fp4_quantize. */
int fp4_quantize_sr(const void* x, int fmt, uint8_t* codes, uint8_t* block_scales, float* tensor_scale,
                    int64_t rows, int64_t K, int in_dtype, unsigned flags, uint64_t seed, void* workspace,
                    size_t workspace_bytes, void* stream);

/* fp4_quantize with options (flags may combine):
 *   FP4_TS_GIVEN: as in fp4_quantize.
 *   FP4_Q_SR: stochastic rounding of the elements with `seed`, exactly as
 *     fp4_quantize_sr.
 *   FP4_Q_2D (NVFP4 only, else FP4_ERR_FMT): 2-D block scaling (NVFP4 video
 *     transcript, the training recipe's second part: a weight matrix is used
 *     as W forward and as W^T backward, so one scale serves a 16 x 16 patch
 *     and both directions quantise alike).  The patch of rows 16p..16p+15
 *     (those inside the matrix) and columns 16b..16b+15 takes the E4M3 scale
 *     of its largest magnitude, written for each of its rows in the usual
 *     layout; rows past the matrix keep scale byte 0.  W and W^T then
 *     dequantise to exact transposes of each other (rows and K multiples of
 *     16).  The tensor scale is the usual one.
 * seed is ignored without FP4_Q_SR.  Arguments and errors otherwise as
 * fp4_quantize. */
int fp4_quantize_ex(const void* x, int fmt, uint8_t* codes, uint8_t* block_scales, float* tensor_scale,
                    int64_t rows, int64_t K, int in_dtype, unsigned flags, uint64_t seed, void* workspace,
                    size_t workspace_bytes, void* stream);

/* Random Hadamard transform (NVFP4 video transcript, the training recipe's
 * third part: values are mixed within a block so that an outlier no longer
 * sets the block scale alone; the transform is orthogonal, so norms and dot
 * products survive).  On every 16-value block along K of the rows x K matrix
 * x: y = (1/4) H16 D x, where D holds the signs of the columns (-1 where the
 * top bit of column k's Philox4x64-10 word under `seed` -- the word
 * fp4_quantize_sr gives element k of a one-row matrix -- is set), and H16 is
 * the 16-point Walsh-Hadamard matrix evaluated as FP32 butterflies
 * (a + b, a - b) of distance 1, 2, 4, 8 in that order; the 1/4 is exact.
 * Two matrices transformed with one seed keep their products along K, so
 * transforming both GEMM operands leaves the product unchanged up to
 * rounding.  x: FP32 or BF16 (in_dtype); y: FP32 or BF16 (out_dtype, round to
 * nearest even), may equal x when the dtypes agree.  K % 16 == 0; x and y
 * 16-byte aligned.  rows == 0 or K == 0 is a no-op. */
int fp4_hadamard16(const void* x, int in_dtype, void* y, int out_dtype, int64_t rows, int64_t K, uint64_t seed,
                   void* stream);

/* Dequantise codes + scales (+ NVFP4 tensor scale) to a rows x K matrix of
 * `out_dtype` (value = E2M1 code x block scale, x tensor scale for NVFP4:
 * Ultralytics glossary "FP4", "How FP4 works"; "Rubin FP4 GEMM deep dive"
 * §3.1; NVFP4 video transcript).  MXFP4 values are exact; NVFP4 computes (E2M1 * E4M3), exact,
 * times tensor_scale with one FP32 rounding; BF16 output is the round-to-
 * nearest-even of that FP32 value.  MXFP8 values are exact.  Same alignment
 * rules as fp4_quantize. */
int fp4_dequantize(const uint8_t* codes, const uint8_t* block_scales, const float* tensor_scale, int fmt,
                   void* out, int out_dtype, int64_t rows, int64_t K, void* stream);

/* C[M x N] = (sum_k A[m,k] * B[n,k]) * tsA * tsB, accumulated in FP32
 * ("Rubin FP4 GEMM deep dive" §3.1-§3.2, §4.2: products of the block-scaled
 * FP4 operands, FP32 accumulation, the scales applied to the result; §4.4 the
 * interface; §1.2, §6.2 decode streams the weights).
 *   A: M x K quantised (codes + scales), B: N x K quantised (each row of B is one
 *   output column, i.e. B is the weight matrix stored K-contiguous).
 *   tsA, tsB: device FP32 tensor scales; required for NVFP4, optional (NULL = 1)
 *   for MXFP4.  C: M x N row-major, FP32 or BF16 (round to nearest even).
 *   MXFP4 runs on the gfx950 block-scaled FP4 matrix core with the E8M0 scales
 *   applied inside the instruction; NVFP4 decodes E2M1 * E4M3 exactly to FP16
 *   and runs the FP16 matrix core, with the tensor scales in the epilogue.
 *   NVFP4 with M <= 32 (decode shapes) takes a bandwidth-first path with
 *   sums in a fixed order (results do not depend on timing) and no workspace.
 *   M = 1 with K <= 8192 runs on the vector ALU (16 weight rows per
 *   workgroup, each thread one 32-value chunk of every row, exact block sums
 *   from FP16 dot products); otherwise one workgroup per 32 weight rows, K
 *   split over its wavefronts.  For M <= 8 the FP4 x FP4 matrix core forms each pair of 16-value blocks'
 *   exact dot product and the E4M3 scales multiply those block sums in FP32
 *   (K up to 8192 at M = 5..8, 16384 at M = 2..4, 32768 at M = 1); otherwise
 *   the weights are decoded to FP16 while the activation fits the
 *   workgroup's staging memory (for example M <= 8 with K <= 8960, or any
 *   M <= 32 with K <= 8192); larger shapes take the tiled kernel.
 * Formats: the FP4 ones (MXFP8 operands: fp4_gemm_w4a8).
 * Requirements: K % 32 == 0 (both formats); codes 16-byte aligned; scales
 *   4-byte aligned; C aligned to its element size.  M, N >= 0 arbitrary, as
 *   long as each operand's scale buffer stays below 4 GiB (at K = 8192:
 *   2^24 rows for MXFP4, 2^23 for NVFP4).
 *   workspace: fp4_workspace_size(FP4_OP_GEMM, fmt, M, N, K, 0) bytes,
 *   zero-filled before first use (0 bytes -> NULL is fine).
 * M == 0 or N == 0 is a no-op; K == 0 writes zeros. */
int fp4_gemm(const uint8_t* A, const uint8_t* sA, const uint8_t* B, const uint8_t* sB, const float* tsA,
             const float* tsB, void* C, int64_t M, int64_t N, int64_t K, int fmt, int out_dtype,
             void* workspace, size_t workspace_bytes, void* stream);

/* Grouped GEMM for mixture-of-experts layers (glossary "Inference and training
 * in FP4": MXFP4 expert weights).
 *   A: A_rows x K quantised token rows.  row_idx[total_rows] (device int32):
 *   output row r reads token row row_idx[r] of A.  group_off[E+1] (device int32,
 *   non-decreasing, group_off[0] = 0, group_off[E] = total_rows): rows
 *   group_off[e] .. group_off[e+1]-1 belong to expert e.  B: E expert matrices,
 *   each N x K quantised, codes N*K/2 bytes apart and scales
 *   fp4_scale_bytes(fmt, N, K) bytes apart.  C: total_rows x N, row r =
 *   (A[row_idx[r]] . B_e^T) * tsA * tsB for its expert e.
 *   Group sizes stay on the device; the kernel builds its own tile list: a
 *   group's last tile is only as high as its rows need (32 to 256 rows, the
 *   rest of the workgroup idles), and tiles of at most 128 rows run after
 *   the others.  Every row_idx entry must lie in [0, A_rows).
 * Formats: FP4_MXFP4, FP4_MXFP4_OCP and FP4_NVFP4.  NVFP4: tsA is the token
 *   matrix's tensor scale (one device FP32) and tsB holds E device FP32
 *   values, expert e's tensor scale at tsB[e] (each expert quantised on its
 *   own); both required (FP4_ERR_NULL).  MXFP4: both ignored, may be NULL.
 * Requirements as fp4_gemm, and A's codes (A_rows * K/2 bytes) below 4 GiB.
 * workspace (optional, MXFP4 formats): NULL, or at least
 *   fp4_workspace_size(FP4_OP_GEMM_GROUPED, fmt, total_rows, N, K, E) bytes,
 *   16-byte aligned (else FP4_ERR_WORKSPACE / FP4_ERR_ALIGN), with the
 *   gathered codes (total_rows * K/2 bytes) below 4 GiB.  With it, the call
 *   first copies row_idx's token rows (codes and scales) into expert order
 *   there and the GEMM reads them as contiguous rows; the result has the same
 *   bits.  Ignored for NVFP4.  Calls sharing one workspace must be ordered. */
int fp4_gemm_grouped(const uint8_t* A, const uint8_t* sA, int64_t A_rows, const int32_t* row_idx,
                     const int32_t* group_off, int32_t E, const uint8_t* B, const uint8_t* sB,
                     const float* tsA, const float* tsB, void* C, int64_t total_rows, int64_t N, int64_t K,
                     int fmt, int out_dtype, void* workspace, size_t workspace_bytes, void* stream);

/* Decode-shape NVFP4 GEMM with the activation quantised inside the call (one
 * kernel): C[M x N] = (X^ . W^T) * s_x * tsW, where X^, s_x are what
 * fp4_quantize(X, FP4_NVFP4, ...) would produce -- the tensor scale from X's
 * largest magnitude (s_x = amax / 2688, 1 for an all-zero X, at least FLT_MIN)
 * unless flags has FP4_TS_GIVEN, 16-value blocks with E4M3 scales, E2M1 codes
 * -- and W^ the NVFP4 weights (codes, scales, tensor scale tsW).  Same
 * arithmetic as fp4_quantize followed by fp4_gemm ("Rubin FP4 GEMM deep dive"
 * §1.2, §6.2: decoding moves every weight once per token, so the activation
 * work is folded into the weight stream); the quantised X is not stored.
 *   X: M x K, FP32 or BF16 (x_dtype), K contiguous, 16-byte aligned.
 *   x_tensor_scale: with FP4_TS_GIVEN, the given s_x (device FP32, required);
 *   otherwise, if non-NULL, receives the computed s_x.
 *   W, sW, tsW: as B, sB, tsB of fp4_gemm.  C: M x N, FP32 or BF16.
 * Applies to small activations (each workgroup stages all of X: for example
 * M <= 8 with K = 8192); fp4_gemm_nvfp4_act_supported says whether a shape
 * is; otherwise FP4_ERR_SHAPE (use fp4_quantize + fp4_gemm).  The result has
 * the same bits as fp4_quantize + fp4_gemm (both take the same decode kernel).
 * Each workgroup re-reads and re-quantises all of X, so beyond M = 2 the two
 * calls are faster (measured at 8192 x 8192). 
 * Requirements: K % 32 == 0.  M == 0 or N == 0 is a no-op. */
int fp4_gemm_nvfp4_act(const void* X, int x_dtype, float* x_tensor_scale, unsigned flags, const uint8_t* W,
                       const uint8_t* sW, const float* tsW, void* C, int64_t M, int64_t N, int64_t K, int out_dtype,
                       void* stream);

/* 1 if fp4_gemm_nvfp4_act takes this shape and X dtype, else 0.  Host-only. */
int fp4_gemm_nvfp4_act_supported(int64_t M, int64_t N, int64_t K, int x_dtype);

/* Dense GEMM with the whole epilogue in the same kernel ("Rubin FP4 GEMM deep
 * dive" §3.2: scale the FP32 result, add bias, apply the activation, convert
 * to FP4 if wanted; §4.2: C = (A.B) * (sA * sB) + bias, fused so that C makes
 * one trip to memory).  Per element, each step one FP32 rounding:
 *   v = acc * tsA * tsB;  v = v + bias[n] (bias != NULL);
 *   v = v > 0 ? v : +0 (act == FP4_ACT_RELU; -0 becomes +0).
 * Output (out):
 *   FP4_OUT_F32 / FP4_OUT_BF16: C is M x N of that type, as fp4_gemm.
 *   FP4_OUT_MXFP4 / FP4_OUT_MXFP4_OCP: v is quantised along N exactly as
 *     fp4_quantize(v, FP4_MXFP4 / FP4_MXFP4_OCP) quantises an M x N matrix
 *     (rows = M, K = N): codes into C (M x N/2 bytes), scale tiles into C_scales
 *     (fp4_scale_bytes(fmt, M, N) bytes, padding included), so the result feeds
 *     the next fp4_gemm as its A operand.  Requires N % 32 == 0 and C 16-byte
 *     aligned.
 *   FP4_OUT_NVFP4: likewise, quantised exactly as fp4_quantize(v, FP4_NVFP4)
 *     with the given tensor scale *C_tensor_scale (flag FP4_TS_GIVEN; NVFP4
 *     video transcript: 16-value blocks, E4M3 block scales, one FP32 tensor
 *     scale).  The scale is the caller's because the one fp4_quantize would
 *     compute needs the maximum of all of C, i.e. a second pass over it.
 *     The result feeds the next fp4_gemm with that tensor scale.
 *   A, sA, B, sB, tsA, tsB, fmt (FP4_MXFP4, FP4_MXFP4_OCP or FP4_NVFP4), K: as
 *   fp4_gemm (always the tiled kernel, any M).  bias: N device FP32 values,
 *   16-byte aligned, or NULL.  C_scales: required (4-byte aligned) for FP4
 *   output, ignored otherwise.  C_tensor_scale: one device FP32 (finite,
 *   > 0), 4-byte aligned, required for FP4_OUT_NVFP4 (FP4_ERR_NULL), ignored
 *   otherwise.  No workspace.
 * M == 0 or N == 0 is a no-op; K == 0 gives v = 0 (+ bias, activation). */
int fp4_gemm_ex(const uint8_t* A, const uint8_t* sA, const uint8_t* B, const uint8_t* sB, const float* tsA,
                const float* tsB, const float* bias, int act, void* C, uint8_t* C_scales,
                const float* C_tensor_scale, int64_t M, int64_t N, int64_t K, int fmt, int out, void* stream);

/* Mixed-format GEMM, W4A8 ("Rubin FP4 GEMM deep dive" §3.4: activations
 * kept in FP8 while the weights go to FP4):
 *   C[m,n] = sum_k A[m,k] * B[n,k], accumulated in FP32, then
 *   v = v + bias[n] (bias != NULL) and v = v > 0 ? v : +0 (act ==
 *   FP4_ACT_RELU), each step one FP32 rounding, stored as FP32 or BF16
 *   (out_dtype, round to nearest even).
 *   A: M x K MXFP8 (codes M * K bytes, scales fp4_scale_bytes(FP4_MXFP8, M, K)
 *   bytes), as fp4_quantize(FP4_MXFP8 or FP4_MXFP8_OCP) writes them.
 *   B: N x K MXFP4 (either exponent rule), as for fp4_gemm.
 * The gfx950 block-scaled matrix core multiplies E4M3 by E2M1 directly, both
 * E8M0 scales applied inside the instruction (at the FP8 rate, half the FP4
 * rate).
 * Requirements: K % 32 == 0, K <= 2^23; codes 16-byte aligned; scales 4-byte
 *   aligned; bias 16-byte aligned or NULL; C aligned to its element size.
 *   M, N >= 0 arbitrary.  No workspace.
 * M == 0 or N == 0 is a no-op; K == 0 gives v = 0 (+ bias, activation). */
int fp4_gemm_w4a8(const uint8_t* A, const uint8_t* sA, const uint8_t* B, const uint8_t* sB, const float* bias,
                  int act, void* C, int64_t M, int64_t N, int64_t K, int out_dtype, void* stream);

/* ---- decode-step operators: paged key-value cache, attention, eviction, log
 * probabilities (the rest of a decode step beside the linear layers above;
 * "Rubin FP4 GEMM deep dive" §1.2, §6.2: decoding is bound by the bytes it
 * streams, so the cache takes the block-scaled formats too). ---- */

/* Row formats of a cache.  A row is one token's D key (or value) values of one
 * head: FP4_KV_BF16 2*D bytes; FP4_KV_MXFP8 D E4M3 bytes and FP4_KV_MXFP4 D/2
 * bytes of E2M1 codes (element order as above), each with D/32 E8M0 scale
 * bytes, the scale of every 32 values as fp4_quantize chooses it for FP4_MXFP8
 * / FP4_MXFP4. */
enum fp4_kv_fmt { FP4_KV_BF16 = 0, FP4_KV_MXFP8 = 1, FP4_KV_MXFP4 = 2 };

/* A pool of cache pages (a host struct; the pointers are device pointers the
 * caller owns).  Row of page p, head h, slot s: row number
 * (p * kv_heads + h) * page_size + s, rows dense in that order in k and v, and
 * likewise the D/32 scale bytes of each row in k_scales and v_scales (MX
 * formats; else ignored).  page_size: a power of two from 16 to 4096.
 * head_dim: 64, 128, 192 or 256.  k, v 16-byte, scales 8-byte aligned.
 *   A page table (device int32, sequences x table_width, dense) maps token t
 * of sequence b to slot t % page_size of page table[b][t / page_size].
 * Sequences may share pages.  The calls below check every entry they use: a
 * page outside [0, pages) is never touched (its tokens count as masked). */
typedef struct fp4_kv_cache {
    void* k;
    void* v;
    uint8_t* k_scales;
    uint8_t* v_scales;
    int64_t pages;
    int32_t page_size;
    int32_t kv_heads;
    int32_t head_dim;
    int32_t fmt; /* enum fp4_kv_fmt */
} fp4_kv_cache;

/* Write new keys and values into the cache, converted to its format (BF16:
 * round to nearest even; MX formats: bit for bit what fp4_quantize gives).
 *   k, v: `rows` rows of kv_heads x head_dim values of in_dtype, row i at
 *   element i * k_stride (v_stride), the heads dense within a row; 16-byte
 *   aligned, strides a multiple of 16 bytes and >= kv_heads * head_dim.
 *   Row i becomes token pos[i] of sequence seq[i] (device int32).  A row with
 *   seq outside [0, seqs), pos outside the table or a page outside the pool is
 *   skipped (seq = -1 pads a batch).  Two rows for one token race.
 * rows == 0 is a no-op. */
int fp4_kv_append(const fp4_kv_cache* cache, const void* k, const void* v, int in_dtype, int64_t k_stride,
                  int64_t v_stride, const int32_t* page_table, int64_t table_width, int64_t seqs,
                  const int32_t* seq, const int32_t* pos, int64_t rows, void* stream);

/* Workspace bytes of fp4_attn_decode (0: none needed).  As for the operations
 * above it must be zero-filled once; calls leave its control words zero.
 * weights: whether weights_out will be given.  0 for invalid arguments. */
size_t fp4_attn_decode_workspace(const fp4_kv_cache* cache, int64_t B, int64_t q_heads, int64_t max_len, int weights);

/* Attention of one new token per sequence over the paged cache.  For query
 * head h of sequence b (reading kv head h / (q_heads / kv_heads)) over the
 * tokens t of [max(0, len - window), len), len = min(lens[b], max_len):
 *   s_t = scale * sum_d q[b,h,d] K[t,d];  p = softmax(s);
 *   out[b,h,:] = sum_t p_t V[t,:];  lse[b,h] = log sum_t exp s_t.
 *   A row with no tokens (length 0, or all pages masked) gives out = 0 and
 *   lse = -inf.  Slots outside the range never influence the result, whatever
 *   bits they hold.  A NaN score in the range gives a NaN row, a NaN lse and NaN
 *   weights of the tokens attended to; masked tokens' weights stay as they are.
 *   q: B x q_heads x head_dim of q_dtype, sequence b at element b * q_stride
 *   (heads dense; 16-byte aligned, stride a multiple of 16 bytes).  out: B x
 *   q_heads x head_dim of out_dtype, dense, 16-byte aligned.  lse: B x q_heads
 *   FP32 or NULL.  q_heads a multiple of kv_heads.
 *   lens: B device int32 (negative reads as 0).  max_len <= table_width *
 *   page_size bounds the lengths (and sizes the workspace); B * kv_heads *
 *   ceil(q_heads / kv_heads / 16) * (max_len / 32 + 32) < 2^32, B < 2^16.  window: 0 for
 *   none.  scale: of magnitude 2^127 at most (0 and below 0 too).
 *   weights_out (optional): FP32 B x kv_heads x weights_stride, receives for
 *   every t < len  weights_in[b,kv,t] + sum over the kv head's query heads of
 *   p_t  (weights_in NULL: 0; it may equal weights_out); entries t >= len are
 *   left alone.  weights_stride >= max_len.
 *   Scores, softmax and sums in FP32.  The probabilities enter the product with
 *   V as three BF16 terms (FP32's 24 bits), with BF16 q and out over an MX
 *   cache as two (relative error 2^-17); q in FP32, or with FP32 out, as three.
 *   Sums are in a fixed order: results do not depend on timing.  The order
 *   follows the lengths of all sequences of the call, so a sequence's last bits
 *   may differ beside other sequences.
 * B == 0 or q_heads == 0 is a no-op; max_len == 0 writes the empty result. */
int fp4_attn_decode(const fp4_kv_cache* cache, const void* q, int q_dtype, int64_t q_stride,
                    const int32_t* page_table, int64_t table_width, const int32_t* lens, int64_t B, int64_t q_heads,
                    int64_t max_len, int64_t window, float scale, void* out, int out_dtype, float* lse,
                    const float* weights_in, float* weights_out, int64_t weights_stride, void* workspace,
                    size_t workspace_bytes, void* stream);

/* Workspace bytes of fp4_kv_evict (zero-filled once; 0: none needed, also
 * for invalid arguments).  max_len: the longest sequence's length. */
size_t fp4_kv_evict_workspace(const fp4_kv_cache* cache, int64_t B, int64_t max_len, int64_t budget);

/* Evict by accumulated attention weight: every (sequence, kv head) with more
 * than `budget` tokens keeps budget of them -- the last min(recent, budget),
 * and of the others those with the largest weights[b,kv,t] (ties to the lowest
 * token; +0 equals -0; a NaN counts as largest) -- and one with at most budget
 * keeps all.  The kept tokens, in their order, become tokens 0, 1, ... of
 * dst_table's pages in dst (which may be the same pool; the destination pages
 * must not be pages the call reads, so pages shared with other sequences stay
 * whole and the old ones can be freed afterwards).
 *   weights: FP32 B x kv_heads x weights_stride; weights_stride >= max_len,
 *   the bound of lens (longer ones read as max_len).
 *   out_lens[b] = min(lens[b], budget).  out_weights: FP32 B x kv_heads x
 *   out_stride, the kept tokens' weights (-0 as +0), then zeros; out_stride >= budget.
 *   kept: int32 B x kv_heads x budget, the kept tokens' old numbers, then -1.
 *   No output may overlap an input (other than the pools, as said).
 *   dst has src's fmt, heads, head_dim and page_size; dst_width * page_size >=
 *   min(budget, max_len).  A kept token whose page (old or new) is outside the
 *   pool is not copied.
 * B == 0 is a no-op. */
int fp4_kv_evict(const fp4_kv_cache* src, const int32_t* src_table, int64_t src_width, const int32_t* lens,
                 const float* weights, int64_t weights_stride, const fp4_kv_cache* dst, const int32_t* dst_table,
                 int64_t dst_width, int32_t* out_lens, float* out_weights, int64_t out_stride, int32_t* kept,
                 int64_t B, int64_t max_len, int64_t budget, int64_t recent, void* workspace,
                 size_t workspace_bytes, void* stream);

/* Workspace bytes of fp4_logprobs (zero-filled once; 0: none needed, also for
 * invalid arguments). */
size_t fp4_logprobs_workspace(int64_t N, int64_t V, int32_t top_k);

/* Log probabilities of given tokens under softmax(y), y = scale * x, with the
 * entropy and the largest alternatives, in one pass over the logits:
 *   lse[n] = log sum_i exp y[n,i];  logp[n,j] = y[n, tokens[n,j]] - lse[n];
 *   entropy[n] = lse[n] - sum_i p_i y_i  (p_i = 0 contributes 0);
 *   top_index[n,:] / top_logp[n,:]: the top_k largest x (ties to the lowest
 *   index, NaN above all, +0 equal to -0) and their log probabilities, in
 *   that order; past V entries: index -1, log probability -inf.
 *   A token outside [0, V) is padding: its logp is 0.  A row whose logits are
 *   all -inf has lse -inf, log probabilities -inf and entropy 0; a NaN or
 *   +inf logit gives NaN.
 *   x: N rows of V values of dtype, row n at element n * stride (stride >= V),
 *   aligned to its element size only.  tokens: int32 N x M, dense (M <= 1024).  entropy
 *   and lse may be NULL; top_k 0..32; 0 < scale <= 2^127.  All sums in
 *   FP32.
 * N == 0 is a no-op; V >= 1. */
int fp4_logprobs(const void* x, int dtype, int64_t stride, int64_t N, int64_t V, float scale, const int32_t* tokens,
                 int32_t M, float* logp, float* entropy, float* lse, int32_t top_k, float* top_logp,
                 int32_t* top_index, void* workspace, size_t workspace_bytes, void* stream);

/* Gradient of fp4_logprobs with respect to x, given lse (and entropy) as it
 * returned them, the gradients g_logp (N x M FP32) and g_entropy (N FP32, or
 * NULL for none; then entropy is not read):
 *   dx_i = scale * (sum_{j: tokens_j = i} g_j
 *                   - p_i * (sum_j g_j + g_entropy * (log p_i + entropy))),
 *   padding tokens' g_j left out, p_i = 0 giving 0 for the second term (so a
 *   row of -inf logits gives 0 there).  dx: N rows of V values of dtype, row
 *   n at element n * dx_stride; rounded once.  dx must not overlap x. */
int fp4_logprobs_backward(const void* x, int dtype, int64_t stride, int64_t N, int64_t V, float scale,
                          const int32_t* tokens, int32_t M, const float* lse, const float* entropy,
                          const float* g_logp, const float* g_entropy, void* dx, int64_t dx_stride, void* stream);

/* ---- Between the projections and the cache: norms of queries and keys for
 * each head, and rotary positions. ---- */

/* Pairs of values (2i, 2i + 1) are turned; otherwise (i, i + rot_dim / 2). */
#define FP4_ROPE_INTERLEAVED 1u
/* Several axes take the pairs in turns (0, 1, 2, 0, 1, 2, ...; one whose section
 * is used up is passed over); otherwise axis 0 the first sections[0] pairs, axis 1
 * the next, and so on. */
#define FP4_ROPE_CYCLIC 2u

/* Rotary positions (a host struct).  Pair i of a head's first rot_dim values is
 * turned by the angle pos[axis(i)] * freq[i], worked out in FP64. */
typedef struct fp4_rope {
    const float* freq;   /* device, rot_dim / 2 radians a position           */
    int32_t rot_dim;     /* a multiple of 8, 0 (no rotation) to head_dim     */
    int32_t axes;        /* 1 to 4 (e.g. 3: time, height, width)             */
    int32_t sections[4]; /* pairs of each axis, rot_dim / 2 together (axes > 1) */
    uint32_t flags;      /* FP4_ROPE_INTERLEAVED, FP4_ROPE_CYCLIC            */
} fp4_rope;

/* For every row and head of q and k, with x its head_dim values:
 *   y = x * (mean x^2 + eps)^-1/2 * weight   (weight NULL: y = x),
 * then the rotation, (a, b) -> (a cos - b sin, b cos + a sin); FP32
 * throughout, rounded once to dtype.
 *   q, k: `rows` rows of q_heads (k_heads) x head_dim values of dtype, row i at
 *   element i * q_stride (k_stride), the heads dense within a row; outputs
 *   likewise.  16-byte aligned, strides multiples of 16 bytes and no less
 *   than a row.  An output may be its input (same address and stride); it must
 *   not overlap an input otherwise.  Either may have no heads.
 *   head_dim: a multiple of 8 from 32 to 256.  q_weight, k_weight: head_dim FP32
 *   or NULL.  eps >= 0; mean x^2 + eps has to lie in FP32's normal range (a head
 *   of zeros with eps 0 gives NaN).  pos: device int32, axes x rows, dense, any
 *   values.
 *   rope NULL: no rotation.  rows < 2^25.
 * rows == 0 is a no-op. */
int fp4_qk_norm_rope(const fp4_rope* rope, const int32_t* pos, const void* q, int64_t q_stride, int64_t q_heads,
                     const void* k, int64_t k_stride, int64_t k_heads, int64_t head_dim, int dtype,
                     const float* q_weight, const float* k_weight, float eps, void* q_out, int64_t q_out_stride,
                     void* k_out, int64_t k_out_stride, int64_t rows, void* stream);

/* Workspace bytes of fp4_qk_norm_rope_backward (0: none needed, also for
 * invalid arguments); enough for any smaller call too.  No zero-fill needed; the
 * control words of others are left alone. */
size_t fp4_qk_norm_rope_workspace(int64_t rows, int64_t q_heads, int64_t k_heads, int64_t head_dim);

/* Gradient of fp4_qk_norm_rope: from the gradients gq, gk of its outputs and
 * its inputs q, k (strided as there), dq and dk (of dtype, rounded once) and,
 * of each weight given, its gradient dq_weight, dk_weight (head_dim FP32,
 * required; sums over rows and heads in a fixed order; 0 for rows == 0).  q (k)
 * is not read without its weight.  dq may be gq or q, dk gk or k. */
int fp4_qk_norm_rope_backward(const fp4_rope* rope, const int32_t* pos, const void* gq, int64_t gq_stride,
                              const void* gk, int64_t gk_stride, const void* q, int64_t q_stride, int64_t q_heads,
                              const void* k, int64_t k_stride, int64_t k_heads, int64_t head_dim, int dtype,
                              const float* q_weight, const float* k_weight, float eps, void* dq, int64_t dq_stride,
                              void* dk, int64_t dk_stride, float* dq_weight, float* dk_weight, int64_t rows,
                              void* workspace, size_t workspace_bytes, void* stream);

/* ---- Around fp4_gemm_grouped: the choice of experts, the tokens' order by
 * expert, and rows there and back. ---- */

/* The top_k largest logits of each token, in order (ties to the lowest expert,
 * NaN above all, +0 equal to -0), and their weights: the softmax over the
 * chosen logits (renormalise != 0), or the softmax over all experts at them.
 * FP32.  A logit of -inf has weight 0 (a row of them only: all weights 0); a NaN
 * or +inf logit makes weights of the row NaN.
 *   logits: T rows of E values of dtype, row t at element t * stride, aligned
 *   to its element size.  1 <= top_k <= min(E, 16); E <= 512.  ids (int32),
 *   weights (FP32): T x top_k, dense.
 * T == 0 is a no-op. */
int fp4_moe_route(const void* logits, int dtype, int64_t stride, int64_t T, int64_t E, int32_t top_k, int renormalise,
                  int32_t* ids, float* weights, void* stream);

/* Gradient of fp4_moe_route's weights with respect to the logits, given the ids
 * it returned and the weights' gradient g (T x top_k FP32):
 *   dlogits_e = p_e (G_e - sum_i p_i G_i),
 * p the softmax over the chosen experts (renormalise; 0 elsewhere) or over all,
 * G_e the sum of g at e's places in ids.  dlogits: T x E of dtype, dense, every
 * element written.  Ids outside [0, E) count for nothing. */
int fp4_moe_route_backward(const void* logits, int dtype, int64_t stride, int64_t T, int64_t E, int32_t top_k,
                           int renormalise, const int32_t* ids, const float* g, void* dlogits, void* stream);

/* Workspace bytes of fp4_moe_sort (0: none needed, also for invalid
 * arguments); enough for any smaller call too.  No zero-fill needed; the control
 * words of others are left alone. */
size_t fp4_moe_sort_workspace(int64_t T, int32_t top_k, int64_t E);

/* The T * top_k entries of ids (T x top_k, device int32) in the order of their
 * experts, equal ids in the order of the entries:
 *   group_off (int32, E + 1) and row_idx (int32, T * top_k: the token of every
 *   row) as fp4_gemm_grouped takes them;
 *   pos (int32, T x top_k): the row of every entry.
 * An entry whose id is outside [0, E) (-1 pads a batch) is taken by no expert:
 * its row r lies behind all the others and pos has -1 - r.  So that group_off[E]
 * is T * top_k, those rows count to the last group; the calls below leave
 * them out.
 *   1 <= E <= 512, 0 <= top_k <= 64, T * top_k <= 2^30. */
int fp4_moe_sort(const int32_t* ids, int64_t T, int32_t top_k, int64_t E, int32_t* group_off, int32_t* row_idx,
                 int32_t* pos, void* workspace, size_t workspace_bytes, void* stream);

/* Rows in expert order: out[r] = x[t] for every entry (t, j), r = pos[t,j] (or
 * -1 - pos[t,j] where that is negative: every row is written).
 *   x: T rows of H values of dtype, row t at element t * stride; out: `rows` rows
 *   of H, dense.  16-byte aligned, H and stride multiples of 16 bytes.  An entry
 *   whose r is no row (r >= rows) is skipped; two entries for one row race.  out
 *   must not overlap x.
 *   0 <= top_k <= 64; T < 2^24 and T * (H rounded up to 1 KB) below 2^32 * 16 bytes,
 *   for this call and the two below.  Its gradient is fp4_moe_combine without weights.
 * T == 0 is a no-op. */
int fp4_moe_gather(const void* x, int dtype, int64_t stride, const int32_t* pos, int64_t T, int32_t top_k, int64_t H,
                   int64_t rows, void* out, void* stream);

/* Rows joined back: out[t] = sum_j weights[t,j] * y[pos[t,j]], j in order, FP32
 * sums, rounded once to dtype.  Entries with pos outside [0, rows) count for
 * nothing (a token without any: 0).  weights: T x top_k FP32, or NULL for 1.
 *   y: `rows` rows of H values of dtype, dense; out: T rows of H, row t at element
 *   t * stride.  Alignment as above.  out must not overlap y.
 * T == 0 is a no-op. */
int fp4_moe_combine(const void* y, int dtype, const int32_t* pos, const float* weights, int64_t T, int32_t top_k,
                    int64_t H, int64_t rows, void* out, int64_t stride, void* stream);

/* Gradient of fp4_moe_combine (with weights) from that of its output, g (T rows
 * of H values of dtype, row t at element t * stride): dy[pos[t,j]] =
 * weights[t,j] * g[t] (rows of dtype, dense), dweights[t,j] = g[t] . y[pos[t,j]]
 * (T x top_k FP32).  An entry that no expert takes (pos negative) has dweights 0
 * and its row -1 - pos in dy zeros; one that names no row of y has dweights 0.
 * Two entries for one row race in dy; rows that no entry names stay as they are.
 * dy must not overlap y or g. */
int fp4_moe_combine_backward(const void* g, int64_t stride, const void* y, int dtype, const int32_t* pos,
                             const float* weights, int64_t T, int32_t top_k, int64_t H, int64_t rows, void* dy,
                             float* dweights, void* stream);

/* ---- Behind the head: drafted tokens. ---- */

/* Workspace bytes of fp4_verify_drafts (0: none needed, for B == 0 and invalid
 * arguments); enough for any smaller call too, with and without draft logits.  It
 * must be zero-filled once; calls leave its control words zero. */
size_t fp4_verify_drafts_workspace(int64_t B, int64_t G, int64_t V);

/* Verify up to G drafted tokens of each of B sequences against the target's
 * distribution, from given random numbers.  p_i, q_i: the softmaxes of the
 * target's and the draft's logits of position i over the sequence's temperature.
 *   tokens[b,i] is kept while u[b,i] * q_i(token) < p_i(token).  At the first
 *   position i that is not kept one token is drawn from max(p_i - q_i, 0) (from
 *   p_i where that is 0 everywhere), past the last draft (i = G, or a token
 *   outside [0, V), which ends a sequence's drafts) from p_i: the smallest t with
 *   sum_{s <= t} r_s > u[b,G] * sum_s r_s.
 *   draft NULL: q_i is 1 at tokens[b,i] (drafts that were not drawn).
 *   temperature[b] (FP32, or NULL for 1) 0, below or NaN: greedy; a token is kept
 *   if it is p_i's largest logit (ties to the lowest), else that one is emitted.
 *   out (int32 B x (G + 1)): the drafts kept, the token drawn, then -1.
 *   accepted (int32 B): the number of drafts kept.  chance (FP32 B x G): the
 *   probability of keeping each draft were it reached, min(1, p_i / q_i); 0
 *   where there is none.
 *   A target row without a distribution (a NaN or +inf logit, or all -inf) ends
 *   the drafts before it and draws nothing (-1); with such a draft row a token
 *   is never kept, and q_i counts as 0.
 *   target: B x (G + 1) rows, draft: B x G rows of V values of dtype, row i of
 *   sequence b at element b * seq_stride + i * row_stride, aligned to the element
 *   size.  tokens: int32 B x G, u: FP32 B x (G + 1), in [0, 1), dense.
 *   B < 2^16, 0 <= G <= 32, 1 <= V <= 2^24, B * (2G + 1) * V <= 2^40.
 *   Exponentials and sums in FP64, in a fixed order; an exponential below 2^-1000
 *   of its row's largest counts as 0.
 * B == 0 is a no-op. */
int fp4_verify_drafts(const void* target, int64_t target_seq_stride, int64_t target_row_stride, const void* draft,
                      int64_t draft_seq_stride, int64_t draft_row_stride, int dtype, int64_t B, int64_t G, int64_t V,
                      const int32_t* tokens, const float* u, const float* temperature, int32_t* out,
                      int32_t* accepted, float* chance, void* workspace, size_t workspace_bytes, void* stream);

/* Static string naming a status code. */
const char* fp4_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* FP4_H_ */
