/* C ABI of the bf16 operators of a feed-forward block on GB300 (sm_103a):
 *
 *   ffn_linear           z = x W^T + bias;  y = act(z) + residual
 *   ffn_linear_backward  dz = dy act'(z);  dx = dz W, dW = dz^T x, dbias = sum of dz
 *   ffn_gated            g = x Wg^T, u = x Wu^T;  h = act(g) u, and g and u kept in bf16 or 8 bits
 *   ffn_gated_backward   of y = h Wd^T: dh = dy Wd;  dg = dh u act'(g), du = dh act(g), h = act(g) u;
 *                        dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x, dWd = dy^T h
 *
 * Matrices are bf16 with contiguous rows, `ld` elements apart; sums are fp32.  Those of an
 * fp32 result, and those that are kept in 8 bits, are rounded to nearest every 512 (1024)
 * terms at least, so that their error does not grow with their length; a bf16 result's may be
 * added up in the tensor core alone, whose additions truncate: 1e-9 of the sum a term.
 *
 * Any base and pitch will do; rows at multiples of 128 bytes are fastest.  An operand of a
 * product whose rows do not start at multiples of 16 bytes is copied to the workspace first,
 * by every call, as is a large one whose rows do not at multiples of 128: weights that are
 * used again and again are better laid out so once.  dz, and dg, du and h of
 * ffn_gated_backward, are rounded to bf16, in which the products that follow take them.
 *
 * Calls return a status code, never throw, and only enqueue work on `stream` (a
 * cudaStream_t) of the calling thread's current device; argument errors are returned
 * before anything is enqueued.  Results must lie apart from what a call reads and from
 * each other, but for y, which may be the residual's rows themselves.  A call's
 * workspace (256-byte aligned, whatever it holds) is the caller's until the work has
 * run: calls with workspaces of their own may overlap, and calls may be captured into
 * CUDA graphs.  Sizes of zero are allowed: an empty sum is zero. */
#ifndef FFN_OPS_H
#define FFN_OPS_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define FFN_API __attribute__((visibility("default")))
#else
#define FFN_API
#endif

typedef enum ffn_status {
    FFN_OK = 0,
    FFN_ERR_INVALID_ARG = -1,    /* null pointer, negative or too large size, pitch below the width, no such
                                    activation or type, a result over what is read */
    FFN_ERR_ALIGNMENT = -2,      /* a base or pitch that the call documents as aligned is not */
    FFN_ERR_WORKSPACE = -3,      /* the workspace is missing or too small */
    FFN_ERR_CUDA = -4,           /* a CUDA runtime call failed */
    FFN_ERR_TENSORMAP = -5,      /* TMA tensor-map encoding failed */
    FFN_ERR_DEVICE_TIMEOUT = -6, /* a barrier wait ran out; the kernel returned early */
    FFN_ERR_UNSUPPORTED = -7     /* device other than compute capability 10.3, or a size beyond the limit */
} ffn_status;

typedef enum ffn_type { FFN_BF16 = 0, FFN_FP32 = 1 } ffn_type;

typedef enum ffn_activation {
    FFN_ACT_NONE = 0,
    FFN_ACT_RELU = 1,
    FFN_ACT_SILU = 2,      /* z / (1 + exp(-z)) */
    FFN_ACT_GELU = 3,      /* z Phi(z) */
    FFN_ACT_GELU_TANH = 4  /* z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2 */
} ffn_activation;

/* Settings of the calling thread's products; 0 leaves the choice to the plan. */
typedef enum ffn_option {
    FFN_OPT_CTA_GROUP = 1,   /* 1 = one SM per tile, 2 = SM pairs */
    FFN_OPT_TRANSPOSED = 2,  /* 1 = the result's rows on the MMA's row side, 2 = its columns */
    FFN_OPT_WIDTH = 3,       /* the tile's width on the MMA's column side: a multiple of 16 (32 for SM pairs), at
                                most 256 (128 for a transposed ffn_gated, whose width is fixed otherwise; for
                                long sums of an fp32 result 192 stands for more, but for pairs not transposed) */
    FFN_OPT_SPLIT = 4,       /* tiles that would leave SMs idle are split along K: 1 = among clusters of CTAs or
                                through global memory (default), 2 = through global memory only, 0 = never */
    FFN_OPT_WATCHDOG_NS = 5, /* limit of any wait inside a kernel (default 2e9, 1e5 to 6e10) */
    FFN_OPT_FAULT_SKIP_LOAD = 6, /* test hook: each producer leaves out this load (-1 = none), so that a bounded
                                    wait runs out and ffn_device_status reports DEVICE_TIMEOUT */
    FFN_OPT_RASTER_GROUP = 7, /* tiles are walked in bands of this many row tiles */
    FFN_OPT_STREAM = 9,       /* products of few tokens on the kernels that stream the weights: 1 = up to 32
                                 tokens, 16 in a gradient, 2 = never */
    FFN_OPT_TOGETHER = 10,    /* a gradient's products that need none of each other in one launch: 1 = always, 2 =
                                 never */
    FFN_OPT_REPACK = 8        /* operands whose rows do not start at multiples of 128 bytes: 1 = copied first, 2 =
                                 read as they are where a tensor map can describe them */
} ffn_option;

typedef struct ffn_plan_info_s {
    int64_t tiles;        /* 0: a kernel that streams the weights, for few tokens */
    int64_t k_blocks;     /* of 64 */
    int32_t grid_ctas;
    int32_t cta_group;
    int32_t transposed;   /* 1: the result's columns on the MMA's row side */
    int32_t width;        /* tile width on the column side */
    int32_t stages;
    int32_t split_tiles;  /* tiles split along K */
    int32_t cluster;      /* CTAs of a cluster that share a tile (1: none) */
    int32_t packed;       /* operands copied to the workspace first */
    int32_t products;     /* of the launch */
    int32_t reserved;
} ffn_plan_info_t;

/* Rows of bf16 (or, where a type is named, of that), `ld` elements apart. */
typedef struct ffn_matrix {
    void *data;
    int64_t ld;
} ffn_matrix;

/* An 8-bit matrix in the format of fp8_ops.h: rows of `ld` e4m3 codes (16-byte aligned, a multiple of
 * 16; of 128 where it is written) and one e8m0 byte per row and block of 128 columns, in ceil(columns / 512)
 * x rows words of four. */
typedef struct ffn_quantized {
    void *codes;
    int64_t ld;
    void *scales;
} ffn_quantized;

FFN_API const char *ffn_strerror(int status);
FFN_API const char *ffn_version(void);

FFN_API int ffn_set_option(int key, int64_t value);
FFN_API int ffn_get_option(int key, int64_t *value);
/* The plan of the calling thread's last product (the first of its launch). */
FFN_API int ffn_plan_info(ffn_plan_info_t *info);

/* ---- product with bias, activation and residual -------------------------- */

typedef struct ffn_linear_args {
    int64_t M, N, K;
    ffn_matrix x;         /* M x K */
    ffn_matrix weight;    /* N x K */
    const void *bias;     /* N values of bias_type, or NULL */
    int32_t bias_type;
    int32_t activation;
    ffn_matrix residual;  /* M x N, or NULL */
    ffn_matrix y;         /* M x N of y_type */
    int32_t y_type;
    int32_t reserved;
    ffn_matrix z;         /* M x N, or NULL */
} ffn_linear_args;

FFN_API int ffn_linear_workspace(const ffn_linear_args *args, int64_t *bytes);
FFN_API int ffn_linear(const ffn_linear_args *args, void *workspace, int64_t workspace_bytes, void *stream);

/* dx, dweight and dbias may each be NULL (not computed).  z may be NULL without an activation.
 * The bias's gradient is the sum of dz before it is rounded, in a fixed order. */
typedef struct ffn_linear_backward_args {
    int64_t M, N, K;
    ffn_matrix dy;       /* M x N */
    ffn_matrix x;        /* M x K */
    ffn_matrix weight;   /* N x K */
    ffn_matrix z;        /* M x N */
    int32_t activation;
    int32_t dweight_type;
    ffn_matrix dx;       /* M x K */
    ffn_matrix dweight;  /* N x K of dweight_type */
    float *dbias;        /* N values */
} ffn_linear_backward_args;

FFN_API int ffn_linear_backward_workspace(const ffn_linear_backward_args *args, int64_t *bytes);
FFN_API int ffn_linear_backward(const ffn_linear_backward_args *args, void *workspace, int64_t workspace_bytes,
                                void *stream);

/* ---- gated block --------------------------------------------------------- */

typedef struct ffn_gated_args {
    int64_t M, F, C;
    ffn_matrix x;             /* M x C */
    ffn_matrix w_gate, w_up;  /* F x C */
    int32_t activation;
    int32_t reserved;
    ffn_matrix h;             /* M x F */
    ffn_matrix g, u;          /* M x F, both or neither */
    ffn_quantized qg, qu;     /* the same in 8 bits, instead; blocks of 128 of the fp32 sums */
} ffn_gated_args;

FFN_API int ffn_gated_workspace(const ffn_gated_args *args, int64_t *bytes);
FFN_API int ffn_gated(const ffn_gated_args *args, void *workspace, int64_t workspace_bytes, void *stream);

/* g and u from bf16, or from 8 bits (h is then made of what these stand for). */
typedef struct ffn_gated_backward_args {
    int64_t M, F, C, N;               /* y is M x N */
    ffn_matrix dy;                    /* M x N */
    ffn_matrix x;                     /* M x C */
    ffn_matrix g, u;                  /* M x F, or NULL: then qg and qu */
    ffn_quantized qg, qu;
    ffn_matrix w_gate, w_up;          /* F x C */
    ffn_matrix w_down;                /* N x F */
    int32_t activation;
    int32_t dweight_type;             /* of the three gradients below */
    ffn_matrix dx;                    /* M x C */
    ffn_matrix dw_gate, dw_up;        /* F x C */
    ffn_matrix dw_down;               /* N x F */
} ffn_gated_backward_args;

FFN_API int ffn_gated_backward_workspace(const ffn_gated_backward_args *args, int64_t *bytes);
FFN_API int ffn_gated_backward(const ffn_gated_backward_args *args, void *workspace, int64_t workspace_bytes,
                               void *stream);

/* Waits for the calling thread's current device (so not while a stream is being captured);
 * DEVICE_TIMEOUT with *detail = the watchdog's word if a wait ran out in any call on it, on
 * whatever stream or from a graph, since the last query, and clears it. */
FFN_API int ffn_device_status(uint32_t *detail);

#ifdef __cplusplus
}
#endif
#endif
