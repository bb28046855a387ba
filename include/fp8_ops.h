/* C ABI of the 8-bit operators of a pre-norm projection on GB300 (sm_103a):
 *
 *   fp8_gemm_*           D = A * B^T of two quantised matrices, fp32 sums, bf16 or fp32 D
 *   fp8_quantize         bf16 or fp32 matrix -> quantised matrix, along rows, columns or both
 *   fp8_rmsnorm          residual addition + root-mean-square norm, quantised output
 *   fp8_rmsnorm_backward its gradients
 *
 * A quantised matrix of R rows and K columns is two device arrays:
 *   codes   R rows of ldq bytes (ldq >= K, a multiple of 16; a multiple of 128
 *           is fastest), the first K of each an e4m3 number;
 *   scales  ceil(K/512) x R words of 4 bytes: byte j of word [i][r] is the biased
 *           exponent e (e8m0: the scale is 2^(e-127)) of row r's block 4i+j of
 *           128 columns.  Bytes past the last block are written as 127 and
 *           have no effect.
 * The value of an element is its code times its block's scale.  The quantisers
 * take the least scale with |value| / scale <= 448 for the block's finite values
 * (at least 2^-127), round to nearest even, and turn infinities and NaN into NaN codes.
 *
 * Calls return a status code, never throw, and only enqueue work on `stream` (a
 * cudaStream_t) of the calling thread's current device (the handle's device
 * for fp8_gemm_*); argument errors are returned before anything is enqueued.
 * Sizes of zero are allowed where a result of that size makes sense: a matrix
 * with no rows launches nothing, a product over K = 0 is zero. */
#ifndef FP8_OPS_H
#define FP8_OPS_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define FP8_API __attribute__((visibility("default")))
#else
#define FP8_API
#endif

typedef enum fp8_status {
    FP8_OK = 0,
    FP8_ERR_INVALID_ARG = -1,    /* null pointer, negative or too large size, pitch below the width, rows
                                    written over part of rows that are read */
    FP8_ERR_ALIGNMENT = -2,      /* a base or pitch that the call documents as aligned is not */
    FP8_ERR_NOT_PLANNED = -3,    /* fp8_gemm_run before fp8_gemm_plan */
    FP8_ERR_CUDA = -4,           /* a CUDA runtime call failed */
    FP8_ERR_TENSORMAP = -5,      /* TMA tensor-map encoding failed */
    FP8_ERR_DEVICE_TIMEOUT = -6, /* a barrier wait ran out; the kernel returned early */
    FP8_ERR_UNSUPPORTED = -7     /* device other than compute capability 10.3, or a size beyond the limit */
} fp8_status;

typedef enum fp8_type { FP8_BF16 = 0, FP8_FP32 = 1 } fp8_type;

typedef enum fp8_gemm_option {
    FP8_GEMM_OPT_CTA_GROUP = 1,   /* 0 = automatic, 1 = one SM per tile, 2 = SM pairs */
    FP8_GEMM_OPT_TRANSPOSED = 2,  /* 0 = automatic, 1 = A's rows on the MMA's row side, 2 = B's rows */
    FP8_GEMM_OPT_WIDTH = 3,       /* 0 = automatic, else the tile's width on the MMA's column side:
                                     a multiple of 16 (32 for SM pairs), at most 224 (192 for an fp32 D
                                     with K > 4096) */
    FP8_GEMM_OPT_SPLIT = 4,       /* tiles that would leave SMs idle are split along K: 1 = among clusters of CTAs or
                                     through global memory (default), 2 = through global memory only, 0 = never */
    FP8_GEMM_OPT_WATCHDOG_NS = 5, /* limit of any wait inside the kernel (default 2e9, 1e5 to 6e10) */
    FP8_GEMM_OPT_FAULT_SKIP_LOAD = 6, /* test hook: each producer leaves out this load (-1 = none), so that
                                         a bounded wait runs out and the call reports DEVICE_TIMEOUT */
    FP8_GEMM_OPT_RASTER_GROUP = 7 /* tiles are walked in bands of this many row tiles; 0 = automatic */
} fp8_gemm_option;

typedef struct fp8_gemm *fp8_gemm_t;

typedef struct fp8_gemm_plan_info_s {
    int64_t tiles;
    int64_t k_blocks;        /* ceil(K / 128) */
    int32_t grid_ctas;
    int32_t cta_group;
    int32_t transposed;      /* 1: B's rows on the MMA's row side */
    int32_t width;           /* tile width on the column side */
    int32_t stages;
    int32_t split_tiles;     /* tiles split along K */
    int32_t smem_bytes;
    int32_t regs_per_thread;
    int32_t cluster;         /* CTAs of a cluster that share a tile (1: none) */
} fp8_gemm_plan_info_t;

FP8_API const char *fp8_strerror(int status);
FP8_API const char *fp8_version(void);

/* ---- product of two quantised matrices ---------------------------------- */

/* A handle bound to CUDA device `device` (-1 = the current one).  It holds plans,
 * the watchdog's status word and, for fp8_gemm_run, a workspace: launches by
 * fp8_gemm_run of one handle share it, so they must run one after another (one
 * stream, or events), replays of graphs that captured them among them.  Use a
 * handle per stream and per graph, or fp8_gemm_run_in, otherwise. */
FP8_API int fp8_gemm_create(int device, fp8_gemm_t *out);
/* Frees the handle's memory, which may wait for the device's work.  No launch of the
 * handle may come after it, nor a replay of a graph that captured one: the launches hold the
 * address of the handle's status word (and of its workspace).  NULL is accepted. */
FP8_API int fp8_gemm_destroy(fp8_gemm_t h);
FP8_API int fp8_gemm_set_option(fp8_gemm_t h, int key, int64_t value);
FP8_API int fp8_gemm_get_option(fp8_gemm_t h, int key, int64_t *value);

/* Host-only check of a problem.  lda, ldb: bytes per row of codes (multiples of
 * 16); ldd: elements per row of D (any value >= N). */
FP8_API int fp8_gemm_check_problem(int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb, int64_t ldd,
                                   int out_type);
/* Picks tile, grid and split; launches nothing. */
FP8_API int fp8_gemm_plan(fp8_gemm_t h, int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb, int64_t ldd,
                          int out_type);
FP8_API int fp8_gemm_plan_info(fp8_gemm_t h, fp8_gemm_plan_info_t *info);
/* D[m][n] = sum_b sa[m][b] sb[n][b] sum_{k in block b} a[m][k] b[n][k], summed
 * in fp32 and rounded once to D's type.  A, B: 16-byte aligned codes; SA, SB:
 * their scales (4-byte aligned); D: aligned to its element.  Only the M x N
 * sub-matrix of D is written.  May be captured into a CUDA graph. */
FP8_API int fp8_gemm_run(fp8_gemm_t h, const void *A, const void *SA, const void *B, const void *SB, void *D,
                         void *stream);
/* Bytes of workspace that a launch of the handle's plan needs: 0 unless tiles are
 * split along K through global memory. */
FP8_API int fp8_gemm_workspace(fp8_gemm_t h, int64_t *bytes);
/* fp8_gemm_run with a workspace of the caller's (16-byte aligned, whatever it holds,
 * held until the work has run): launches with workspaces of their own may overlap. */
FP8_API int fp8_gemm_run_in(fp8_gemm_t h, const void *A, const void *SA, const void *B, const void *SB, void *D,
                            void *workspace, int64_t workspace_bytes, void *stream);
/* Waits for the handle's device (so not while a stream is being captured);
 * DEVICE_TIMEOUT with *detail = the watchdog's word if a wait ran out in any
 * launch of the handle, on whatever stream or from a graph, since the last call,
 * and clears it. */
FP8_API int fp8_gemm_device_status(fp8_gemm_t h, uint32_t *detail);

/* ---- quantiser ----------------------------------------------------------- */

/* y[r][c] = x[r][c] * row_factor[r] * column_factor[c] (either may be NULL),
 * quantised.  x: R rows of ldx elements of x_type.
 *   codes, scales      (or both NULL) y with blocks of 128 along its rows
 *   codes_t, scales_t  (or both NULL) y's transpose, C rows of R codes, with
 *                      blocks of 128 along those (down y's columns)
 *   tile != 0: one scale for each 128 x 128 tile of y, in both outputs
 * row_factor: fp32; column_factor: column_type.  codes and codes_t 16-byte
 * aligned with pitches that are multiples of 16, scales 4-byte aligned. */
FP8_API int fp8_quantize(const void *x, int x_type, int64_t ldx, int64_t R, int64_t C, int tile,
                         const float *row_factor, const void *column_factor, int column_type, void *codes, int64_t ldq,
                         void *scales, void *codes_t, int64_t ldqt, void *scales_t, void *stream);

/* ---- norm ---------------------------------------------------------------- */

#define FP8_NORM_MAX_COLUMNS 32768

/* h[r] = bf16(x[r] + residual[r])  (h = x where residual is NULL; nothing is stored then)
 * rstd[r] = 1 / sqrt(mean_c h[r][c]^2 + eps);  y[r][c] = h[r][c] * rstd[r] * weight[c]
 * and y is quantised along its rows into codes and scales.  x, residual, h:
 * bf16; weight: weight_type; rstd: fp32, R values, or NULL.  h may be x or
 * residual itself; rows of h over part of theirs are refused (INVALID_ARG).  C <= FP8_NORM_MAX_COLUMNS. */
FP8_API int fp8_rmsnorm(const void *x, int64_t ldx, const void *residual, int64_t ldr, const void *weight,
                        int weight_type, int64_t R, int64_t C, float eps, void *h, int64_t ldh, void *codes,
                        int64_t ldq, void *scales, float *rstd, void *stream);

/* Bytes of workspace that fp8_rmsnorm_backward needs for these sizes (on the
 * calling thread's current device). */
FP8_API int fp8_rmsnorm_backward_workspace(int64_t R, int64_t C, int64_t *bytes);
/* With g = dy * weight and n = h * rstd:
 *   dx[r][c] = rstd[r] * (g[r][c] - n[r][c] * mean_c(g[r] * n[r])) (+ dresidual[r][c])
 *   dweight[c] = sum_r dy[r][c] * n[r][c]
 * dx is the gradient of both x and residual.  dy, h, dresidual (or NULL), dx:
 * bf16 (dx may be dy or dresidual itself; rows of dx over part of theirs or of h's
 * are refused); dweight: fp32, C values, summed in a
 * fixed order.  workspace: 16-byte aligned, held until the work has run. */
FP8_API int fp8_rmsnorm_backward(const void *dy, int64_t lddy, const void *h, int64_t ldh, const void *weight,
                                 int weight_type, const float *rstd, const void *dresidual, int64_t lddr, void *dx,
                                 int64_t lddx, float *dweight, int64_t R, int64_t C, void *workspace,
                                 int64_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif
