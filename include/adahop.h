/*
 * adahop.h -- C ABI of the AdaHOP per-GEMM hot path on MI355X (gfx950).
 *
 * The method is the one of "AdaHOP: Fast and Accurate Low-Precision Training
 * via Outlier-Pattern-Aware Rotation" (arXiv 2604.02525). Its Fig. 9 and the
 * appendix list of its kernels give four stages per GEMM:
 *   1. FOID: the outlier lines of one operand, chosen by the variance of their
 *      first 64 elements (adahop_detect);
 *   2. IHT and quantization: zero those lines, rotate the residual by a
 *      32-point Hadamard transform along the inner dimension, quantize to
 *      MXFP4 (adahop_iht_quant);
 *   3. the fused MXFP4 + BF16 GEMM: the residual product on FP4 matrix cores
 *      and the outlier product in bf16 (adahop_gemm_mx);
 *   4. the fused scatter-add of the outlier product into the result (inside
 *      adahop_gemm_mx's epilogue).
 * Fig. 5 routes each of a linear layer's three products (forward, input
 * gradient, weight gradient) by its operand pattern pair to IHT, OE-Left,
 * OE-Right or BF16 (adahop_route); adahop_gemm runs the whole path for one
 * product.
 *
 * Conventions
 *   - Every tensor pointer is a DEVICE pointer owned by the caller. The
 *     library never allocates, frees or synchronizes device memory; scratch
 *     space is the caller's workspace (adahop_detect_noalloc alone uses a
 *     static device array of the library instead). Every launch is enqueued
 *     on `stream` (a hipStream_t, NULL = the null stream) and the call
 *     returns at once.
 *   - bf16 tensors are uint16 bit patterns, row-major, leading dimension `ld`
 *     in elements (ld >= cols). A bf16 input quantized along its rows
 *     (contraction along columns) must have 16-byte aligned rows: base
 *     pointer 16-byte aligned and ld % 8 == 0. Packed code buffers must be
 *     16-byte aligned.
 *   - Textbook frame of a product: C[m,n] = A[m,K] * B[K,n], K the inner
 *     (contraction) dimension.
 *   - MXFP4 operand (OCP Microscaling v1.0 MXFP4): 4-bit E2M1 codes, two per
 *     byte, element 2j in the low nibble, stored [outer][K/2]; one E8M0 scale
 *     byte per 32 consecutive K-elements, stored [outer][K/32]. K runs
 *     contiguously. For A, outer = m (its rows); for B, outer = n (its
 *     columns).
 *   - Outlier index sets are int32, ascending, unique, on the device.
 *   - Errors: argument errors are found on the host before any launch and
 *     return ADAHOP_ERR_INVALID (or ADAHOP_ERR_UNSUPPORTED for a valid but
 *     unimplemented case) with a message in adahop_last_error(); a too-small
 *     workspace returns ADAHOP_ERR_WORKSPACE; a failed launch returns
 *     ADAHOP_ERR_HIP. Non-finite inputs are not supported (results
 *     unspecified). Outputs must not alias inputs.
 *   - Thread safety: calls on different streams may run concurrently;
 *     adahop_last_error() is per host thread.
 *   - adahop_gemm with OE_LEFT or OE_RIGHT quantizes the operand FOID does
 *     not scan beside FOID: in FOID's own launch when FOID's selection takes
 *     at most two levels (k <= 256, up to 16384 candidates at k = 64);
 *     otherwise, when the two operands exceed 96 MB of bf16, on a second
 *     stream the library creates once per device (default priority), forked
 *     from `stream` with an event and joined back before the GEMM;
 *     otherwise after FOID on `stream`. The call's completion stays ordered
 *     on `stream`.
 */
#ifndef ADAHOP_H
#define ADAHOP_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define ADAHOP_API __attribute__((visibility("default")))

typedef enum {
  ADAHOP_OK = 0,
  ADAHOP_ERR_INVALID = 1,     /* bad argument (detected before any launch) */
  ADAHOP_ERR_UNSUPPORTED = 2, /* valid but not implemented (alignment, sizes) */
  ADAHOP_ERR_WORKSPACE = 3,   /* workspace missing or too small */
  ADAHOP_ERR_HIP = 4          /* a HIP runtime call or launch failed */
} adahop_status;

/* Outlier pattern of a stored tensor (Table 1's R / C / N). */
typedef enum { ADAHOP_PAT_NONE = 0, ADAHOP_PAT_ROW = 1, ADAHOP_PAT_COL = 2 } adahop_pattern;

/* The three products of a linear layer Y = X W^T (Table 1's columns):
 * FWD   Y  [T,Dout]    = X [T,Din] * W^T       (lhs X,  rhs W [Dout,Din])
 * DGRAD dX [T,Din]     = GY [T,Dout] * W       (lhs GY, rhs W [Dout,Din])
 * WGRAD dW [Dout,Din]  = GY^T * X              (lhs GY, rhs X [T,Din]) */
typedef enum { ADAHOP_OP_FWD = 0, ADAHOP_OP_DGRAD = 1, ADAHOP_OP_WGRAD = 2 } adahop_op;

/* Path of one product (Fig. 5). OE_INNER extracts inner-dimension lines of
 * both operands into a dense rank-k bf16 term; MXFP4 is plain quantization
 * without rotation or extraction (a baseline). */
typedef enum {
  ADAHOP_ROUTE_AUTO = -1,
  ADAHOP_ROUTE_BF16 = 0,
  ADAHOP_ROUTE_IHT = 1,
  ADAHOP_ROUTE_OE_LEFT = 2,
  ADAHOP_ROUTE_OE_RIGHT = 3,
  ADAHOP_ROUTE_OE_INNER = 4,
  ADAHOP_ROUTE_MXFP4 = 5
} adahop_route_t;

typedef enum { ADAHOP_AXIS_ROWS = 0, ADAHOP_AXIS_COLS = 1 } adahop_axis;
typedef enum { ADAHOP_OUT_BF16 = 0, ADAHOP_OUT_F32 = 1 } adahop_out_dtype;

/* Layout of packed MXFP4 operands in an adahop_gemm workspace.
 *   ROWS  : codes [outer][K/2], scales [outer][K/32] (as adahop_iht_quant).
 *   KCHUNK: K cut into chunks of 128: codes [K/128][outer][64] and scales
 *           [K/128][outer][4], i.e. chunk c of row r holds K-elements
 *           128 c .. 128 c + 127 of that row, each chunk of all rows
 *           contiguous -- the order in which the GEMM streams them. A
 *           chunk's four scale bytes are its blocks' in the order 0, 2, 1, 3. */
typedef enum { ADAHOP_LAYOUT_ROWS = 0, ADAHOP_LAYOUT_KCHUNK = 1 } adahop_layout;

ADAHOP_API const char* adahop_status_string(int status);
/* Detail of the last failure on this host thread ("" if none). */
ADAHOP_API const char* adahop_last_error(void);
ADAHOP_API int adahop_version(void);

/* ---------------------------------------------------------------------------
 * Routing (host only, pure). Fig. 5 routes each product by the pattern pair
 * of its operands; Fig. 2 and the abstract say IHT (mixing along the inner
 * dimension) suppresses outliers that lie along the inner dimension and not
 * those along the outer one. Rule, in the textbook frame: A is hurt if its
 * outlier lines are rows, B if its outlier lines are columns; neither -> IHT,
 * A only -> OE_LEFT, B only -> OE_RIGHT, both -> BF16. Patterns are given in
 * each tensor's storage frame (as in Table 1); a tensor used transposed swaps
 * ROW and COL. Returns ADAHOP_ROUTE_AUTO for an invalid op or pattern. */
ADAHOP_API adahop_route_t adahop_route(adahop_op op, adahop_pattern pat_lhs,
                                       adahop_pattern pat_rhs);

/* ---------------------------------------------------------------------------
 * Pattern calibration (Table 1 names the three patterns; Fig. 4 and Fig. 8
 * show them on real tensors, and the pages give no numeric test). Reading
 * used here: a tensor is Row-wise when a few rows carry far more energy than
 * the typical row, Column-wise likewise for columns, None otherwise,
 * measured with FOID's own line score.
 *
 * adahop_line_scores writes each line's FOID score (the probe variance
 * defined below for adahop_detect, bit for bit) to scores_out, a DEVICE
 * array of fp64 [rows] (axis ROWS) or [cols] (axis COLS). Enqueued on
 * `stream`; no workspace. Errors as adahop_detect's argument checks.
 *
 * adahop_classify_pattern (host only, pure) takes HOST copies of a tensor's
 * row scores and column scores and compares, per axis, r = max / median
 * (the median is the lower one: the element of rank (n - 1) / 2 in
 * ascending order): if the larger r is below `threshold` the pattern is
 * NONE, else ROW when r_rows >= r_cols and COL otherwise. A zero median with
 * a positive maximum counts as an infinite ratio; an all-zero axis as 1.
 * Returns ADAHOP_PAT_NONE for null pointers or empty arrays. */
ADAHOP_API adahop_status adahop_line_scores(const uint16_t* t, int64_t rows, int64_t cols,
                                            int64_t ld, adahop_axis axis, int32_t probe,
                                            double* scores_out, void* stream);
ADAHOP_API adahop_pattern adahop_classify_pattern(const double* row_scores, int64_t rows,
                                                  const double* col_scores, int64_t cols,
                                                  double threshold);

/* ---------------------------------------------------------------------------
 * FOID (appendix, kernel 1; Fig. 9). Candidates are the rows (axis ROWS:
 * statistics over t[r, 0:P]) or the columns (axis COLS: t[0:P, c]) of the
 * bf16 tensor t [rows, cols], P = min(probe, line length). Each candidate's
 * score is the population variance of those P values, computed in fp64 in
 * index order (sum, mean, then sum of squared deviations). The k candidates
 * with the largest score (ties: lower index first) are written to idx_out
 * (device int32[k]) in ascending order. Deterministic. Needs
 * adahop_detect_workspace_size(...) bytes of workspace: none up to 1024
 * candidates (4096 when k > 256), else the survivor lists of the selection
 * levels (k scores and indices per chunk of candidates: 256 or 512 when the
 * first level's survivors then fit in 1024 entries, else 1024, or 4096
 * when k > 256; two lists) and 256 bytes for a counter; ws may be NULL when
 * the size is 0.
 * Errors: INVALID if t/idx_out is NULL, rows/cols < 1, ld < cols, probe < 1,
 * k < 1 or k > number of candidates; UNSUPPORTED if k > 1024. */
ADAHOP_API size_t adahop_detect_workspace_size(int64_t rows, int64_t cols, adahop_axis axis,
                                               int32_t k);
ADAHOP_API adahop_status adahop_detect(const uint16_t* t, int64_t rows, int64_t cols,
                                       int64_t ld, adahop_axis axis, int32_t probe,
                                       int32_t k, int32_t* idx_out, void* ws,
                                       size_t ws_bytes, void* stream);

/* FOID without a workspace, for callers that cannot allocate device memory
 * (code under HIP graph capture, tight serving loops, harnesses that forbid
 * allocation). Same arguments, checks and result as adahop_detect; the
 * selection's scratch (what adahop_detect_workspace_size reports) lives in a
 * static device array of adahop_detect_noalloc_max_bytes() bytes (1 MiB),
 * one per GPU, that the library holds until the process ends. The call
 * itself allocates nothing and clears what must start at zero with a kernel,
 * not a memset. Errors: as adahop_detect, and UNSUPPORTED when the
 * selection needs more scratch than that (e.g. k = 1024 over more than about
 * 170 000 candidates; k = 64 over more than about 1.4 million). Every call
 * on one GPU shares that GPU's array: calls that overlap in time on one GPU
 * (different streams or host threads without ordering) race and give
 * unspecified indices; order them on one stream. */
ADAHOP_API size_t adahop_detect_noalloc_max_bytes(void);
ADAHOP_API adahop_status adahop_detect_noalloc(const uint16_t* t, int64_t rows, int64_t cols,
                                               int64_t ld, adahop_axis axis, int32_t probe,
                                               int32_t k, int32_t* idx_out, void* stream);

/* ---------------------------------------------------------------------------
 * Zero + gather + IHT + MXFP4 quantization (appendix, kernel 2; abstract).
 * src is bf16 [rows, cols]. contract COLS: 32-blocks run along each row
 * (K = cols, outer = rows); contract ROWS: 32-blocks run down each column
 * (K = rows, outer = cols). K must be a multiple of 32.
 * Zeroing: the nzero lines zero_idx (device, ascending, unique) -- rows of
 * src if zero_axis is ROWS, columns if COLS -- are treated as +0 (the
 * residual with the outliers removed). gathered (device, may be NULL when
 * nzero > 0 and the lines are not needed) receives a compact bf16 copy of
 * those lines, one line per row: [nzero][cols] for rows, [nzero][rows] for
 * columns.
 * Rotation: hadamard_block 32 applies the orthonormal 32-point Walsh-Hadamard
 * transform (Sylvester order, fp32 butterflies with strides 1,2,4,8,16, then
 * one multiply by fp32(1/sqrt(32))) to each block; 0 applies none.
 * Quantization (OCP MX v1.0): scale exponent s = floor(log2(block amax)) - 2,
 * clamped to [-127, 127], stored as the byte s + 127 (0x00 for an all-zero
 * block); each element's code is the sign bit and the E2M1 magnitude nearest
 * to |y| / 2^s, ties to the even code, saturating at 6.
 * Output codes [outer][K/2] and scales [outer][K/32] (device).
 * Errors: INVALID for NULL src/codes/scales, bad sizes, K % 32 != 0,
 * hadamard_block not in {0, 32}, nzero < 0, or zero_idx NULL with nzero > 0;
 * UNSUPPORTED if codes or gathered are not 16-byte aligned, (contract COLS)
 * src rows are not 16-byte aligned, or nzero > 1024. Indices are not
 * validated on the device: unsorted or repeated zero_idx gives unspecified
 * results, out-of-range entries are ignored. */
ADAHOP_API adahop_status adahop_iht_quant(const uint16_t* src, int64_t rows, int64_t cols,
                                          int64_t ld, adahop_axis contract,
                                          int32_t hadamard_block, const int32_t* zero_idx,
                                          int32_t nzero, adahop_axis zero_axis,
                                          uint8_t* codes, uint8_t* scales, uint16_t* gathered,
                                          void* stream);

/* ---------------------------------------------------------------------------
 * Fused MXFP4 + BF16 GEMM with the scatter-add epilogue (appendix, kernels 3
 * and 4). */
typedef struct {
  const uint8_t* codes;   /* [outer][K/2] */
  const uint8_t* scales;  /* [outer][K/32] */
  int64_t outer;          /* m for A, n for B */
  int64_t K;
} adahop_mx_operand;

/* A bf16 factor of the outlier product, seen as [outer][inner]: element
 * (r, t) sits at ptr[r * ld + t] if inner_contiguous, else ptr[t * ld + r]. */
typedef struct {
  const uint16_t* ptr;
  int64_t ld;
  int32_t inner_contiguous;
  int32_t reserved;
} adahop_bf16_view;

/* The outlier (OE) term, P = a * b^T contracted over the views' inner index:
 *   OE_LEFT : a = the k extracted rows of A ([k][K]), b = B in bf16 ([n][K]);
 *             C[idx[p], j] += P[p][j].
 *   OE_RIGHT: a = A in bf16 ([m][K]), b = the k extracted columns of B
 *             ([k][K]); C[i, idx[p]] += P[i][p].
 *   OE_INNER: a = A's k extracted columns ([m][k]), b = B's k extracted rows
 *             ([n][k]); C[i, j] += P[i][j].
 * The add happens on fp32 values before the single rounding of C. */
typedef struct {
  adahop_route_t route;   /* OE_LEFT, OE_RIGHT or OE_INNER */
  int32_t k;
  const int32_t* idx;     /* device [k]; unused (may be NULL) for OE_INNER */
  adahop_bf16_view a;
  adahop_bf16_view b;
} adahop_oe;

/* C[m,n] (row-major, leading dim ldc, bf16 or fp32) = deq(A) * deq(B)^T with
 * fp32 accumulation, plus the OE term if oe != NULL. Needs
 * adahop_gemm_mx_workspace_size(...) bytes of 16-byte aligned workspace: the
 * outlier product's partial sums (OE_LEFT/OE_RIGHT) and, when K is a multiple
 * of 512, a copy of both scale arrays reordered for the GEMM plus, when the
 * last round of 256 x 256 tiles is split along K (at most half a round left
 * over from whole rounds of one tile per compute unit of the current device
 * -- 256 on an MI355X --, K / 128 a multiple of 8 and at least 32),
 * 256 KB of fp32 partial sums per tile part (0 when none applies; ws may then
 * be NULL). Its contents after the call are unspecified.
 * Errors: INVALID for NULL pointers, K mismatch, K % 32 != 0, ldc < n, a bad
 * out_dtype, bad OE descriptors; WORKSPACE for a missing or short workspace;
 * UNSUPPORTED for k > 1024, codes not 16-byte aligned or a misaligned
 * workspace. */
ADAHOP_API size_t adahop_gemm_mx_workspace_size(int64_t m, int64_t n, int64_t K,
                                                const adahop_oe* oe);
ADAHOP_API adahop_status adahop_gemm_mx(const adahop_mx_operand* A,
                                        const adahop_mx_operand* B, const adahop_oe* oe,
                                        void* C, int64_t ldc, adahop_out_dtype out_dtype,
                                        void* ws, size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * One AdaHOP product end to end: route, FOID on the operand and axis the route
 * extracts, zero + gather + IHT + MXFP4 on both operands (along each one's
 * contraction axis), the fused GEMM and the scatter-add.
 *   FWD  : lhs X [T,Din],  rhs W [Dout,Din] -> out Y  [T,Dout]
 *   DGRAD: lhs GY [T,Dout], rhs W [Dout,Din] -> out dX [T,Din]
 *   WGRAD: lhs GY [T,Dout], rhs X [T,Din]    -> out dW [Dout,Din]
 * lhs, rhs and out are contiguous row-major. route AUTO applies adahop_route
 * to (pat_lhs, pat_rhs); oe_rank is the number of extracted lines (64 on the
 * pages, Fig. 10). The contraction length (Din, Dout or T) must be a
 * multiple of 32. The workspace holds, after the call, the quantized
 * operands and the outlier lines at the offsets adahop_gemm_plan reports;
 * the operands are in the plan's layout (KCHUNK when the contraction length
 * is a multiple of 512 and each packed operand is under 2 GiB, else ROWS).
 * Errors: as for the stage calls; INVALID for a bad op or route, or an OE
 * route with oe_rank < 1 or above the number of candidate lines.
 * Route BF16 (both operands hurt) computes the plain product on bf16 matrix
 * cores with fp32 accumulation and no packed operands (oe_rank is ignored).
 * When the contraction length is a multiple of 128 an operand not
 * contiguous along K (DGRAD: W; WGRAD: GY and X) is read in place if its
 * row length is a multiple of 8 and it is under 2 GiB; the workspace holds
 * K-major bf16 copies of the others, for a forward with 8192 or more rows on
 * one side a copy across K of the other operand (read faster that way), and
 * the fp32 parts of tiles split along K. Otherwise it needs none. With an
 * operand or the workspace not 16-byte aligned it runs on a slower tile
 * kernel instead. */
typedef struct {
  adahop_route_t route;   /* resolved route */
  int64_t m, n, K;        /* textbook-frame sizes */
  int32_t k;              /* extracted lines (0 without OE) */
  int32_t scan_tensor;    /* 0 = lhs, 1 = rhs, -1 = no FOID */
  adahop_axis scan_axis;  /* candidate lines: rows or columns of that tensor */
  adahop_layout layout;   /* layout of the packed operands below */
  size_t ws_bytes;        /* workspace the call needs */
  /* Byte offsets into the workspace (SIZE_MAX if absent): */
  size_t off_idx;         /* int32 [k] FOID indices */
  size_t off_a_codes, off_a_scales;   /* A packed (outer = m) in `layout` */
  size_t off_b_codes, off_b_scales;   /* B packed (outer = n) in `layout` */
  size_t off_lhs_lines;   /* bf16 lines gathered from lhs (layout as adahop_iht_quant) */
  size_t off_rhs_lines;   /* bf16 lines gathered from rhs */
  int32_t oe_in_quant;    /* 1: the outlier product is formed in the other operand's
                             quantization (asked for with adahop_gemm_options) */
} adahop_plan;

ADAHOP_API adahop_status adahop_gemm_plan(adahop_op op, int64_t T, int64_t Din, int64_t Dout,
                                          adahop_pattern pat_lhs, adahop_pattern pat_rhs,
                                          adahop_route_t route, int32_t oe_rank,
                                          adahop_plan* plan);
ADAHOP_API size_t adahop_gemm_workspace_size(adahop_op op, int64_t T, int64_t Din,
                                             int64_t Dout, adahop_pattern pat_lhs,
                                             adahop_pattern pat_rhs, adahop_route_t route,
                                             int32_t oe_rank);
ADAHOP_API adahop_status adahop_gemm(adahop_op op, const uint16_t* lhs, const uint16_t* rhs,
                                     int64_t T, int64_t Din, int64_t Dout,
                                     adahop_pattern pat_lhs, adahop_pattern pat_rhs,
                                     adahop_route_t route, int32_t oe_rank, void* out,
                                     adahop_out_dtype out_dtype, void* ws, size_t ws_bytes,
                                     void* stream);

/* Options of adahop_gemm_plan_ex and adahop_gemm_ex (NULL: all defaults,
 * which is adahop_gemm's behaviour). reserved must be zero.
 * oe_in_quant = 1: with OE_LEFT or OE_RIGHT, when the operand FOID does not
 * scan is quantized down its columns (contracted along its rows: DGRAD's W,
 * both WGRAD operands) and k <= 64, that operand's quantization also forms
 * the outer outlier product -- its rank-k product with the extracted lines,
 * fp32 partial sums per group of 128-row tiles, then their sum in group
 * order -- so the operand is read once (appendix, kernels 2 and 3: the
 * outlier product beside the quantization's single pass). The stages then
 * run one after another on `stream`: FOID, the scanned operand's
 * quantization (which gathers the lines), the other's with the partial
 * sums, their sum, the GEMM, whose epilogue adds the sum to the extracted
 * lines before the single rounding. The plan reports whether it applies
 * (plan.oe_in_quant); where it does not, the call runs as adahop_gemm. The
 * default path, which quantizes that operand beside FOID and forms the
 * outlier product inside the GEMM launch, measured faster on the workloads
 * here; this one exists for the one-read schedule and its measurement.
 * Errors: INVALID for oe_in_quant not 0 or 1 or a reserved field not 0;
 * otherwise as adahop_gemm_plan / adahop_gemm_timed (stage_events may be
 * NULL). */
typedef struct {
  int32_t oe_in_quant;
  int32_t reserved[7];
} adahop_gemm_options;

ADAHOP_API adahop_status adahop_gemm_plan_ex(adahop_op op, int64_t T, int64_t Din, int64_t Dout,
                                             adahop_pattern pat_lhs, adahop_pattern pat_rhs,
                                             adahop_route_t route, int32_t oe_rank,
                                             const adahop_gemm_options* opts,
                                             adahop_plan* plan);
ADAHOP_API adahop_status adahop_gemm_ex(adahop_op op, const uint16_t* lhs, const uint16_t* rhs,
                                        int64_t T, int64_t Din, int64_t Dout,
                                        adahop_pattern pat_lhs, adahop_pattern pat_rhs,
                                        adahop_route_t route, int32_t oe_rank,
                                        const adahop_gemm_options* opts, void* out,
                                        adahop_out_dtype out_dtype, void* ws, size_t ws_bytes,
                                        void* stream, void* const* stage_events);

/* ---------------------------------------------------------------------------
 * Saved forward context (appendix, kernel 2: for the activation of the
 * forward path, the quantized residual and the bf16 outlier tensor are kept
 * for backpropagation). The only backward product that reads the activation
 * X [T, Din] is the weight gradient dW = GY^T X, contracting over T, so the
 * context keeps X in the form that product consumes: the k columns its FOID
 * extracts (route OE_RIGHT), the residual with those columns zeroed, rotated
 * (FWHT-32, not for route MXFP4) and MXFP4-quantized along T, and those
 * columns in bf16 -- 17/32 bytes per element plus 2 k T for the lines, up to
 * 3.76x less than X in bf16. adahop_gemm_wgrad_ctx then computes the weight
 * gradient from GY and the context alone, bit for bit what adahop_gemm
 * (WGRAD, GY, X, ...) computes from X.
 *
 * pat_gy, pat_x, route and oe_rank are those of the weight gradient
 * (route AUTO applies adahop_route(WGRAD, pat_gy, pat_x)); the context
 * holds X for routes IHT, MXFP4 and OE_RIGHT. Routes BF16, OE_LEFT and
 * OE_INNER read X in bf16 in the backward (the outlier product of OE_LEFT
 * multiplies GY's lines by the whole of X) and return UNSUPPORTED.
 *
 * The context is one caller-owned device buffer of ctx_bytes (16-byte
 * aligned) at the plan's offsets: idx int32 [k] (SIZE_MAX without
 * extraction), codes and scales of X's residual with outer = Din, K = T in
 * the plan's layout (KCHUNK when T is a multiple of 512, as adahop_gemm's
 * weight gradient packs it), lines bf16 [k][T] (X's extracted columns, one
 * per row). adahop_ctx_save needs save_ws_bytes of workspace (FOID's
 * selection scratch; 0: ws may be NULL), adahop_gemm_wgrad_ctx
 * wgrad_ws_bytes (GY's packed form, the outlier product's partial sums and
 * the GEMM's scratch). Errors as adahop_gemm; INVALID for a context smaller
 * than its plan. stage_events: as adahop_gemm_timed (NULL for none); the FOID
 * and rhs stages are empty. */
typedef struct {
  adahop_route_t route;   /* the weight gradient's resolved route */
  int64_t T, Din, Dout;
  int32_t k;              /* extracted columns of X (0 without extraction) */
  adahop_layout layout;   /* layout of the kept codes and scales */
  size_t ctx_bytes;
  size_t off_idx, off_codes, off_scales, off_lines;   /* SIZE_MAX if absent */
  size_t save_ws_bytes;   /* workspace of adahop_ctx_save */
  size_t wgrad_ws_bytes;  /* workspace of adahop_gemm_wgrad_ctx */
} adahop_ctx_plan_t;

ADAHOP_API adahop_status adahop_ctx_plan(int64_t T, int64_t Din, int64_t Dout,
                                         adahop_pattern pat_gy, adahop_pattern pat_x,
                                         adahop_route_t route, int32_t oe_rank,
                                         adahop_ctx_plan_t* plan);
ADAHOP_API adahop_status adahop_ctx_save(const uint16_t* X, int64_t T, int64_t Din,
                                         int64_t Dout, adahop_pattern pat_gy,
                                         adahop_pattern pat_x, adahop_route_t route,
                                         int32_t oe_rank, void* ctx, size_t ctx_bytes,
                                         void* ws, size_t ws_bytes, void* stream);
ADAHOP_API adahop_status adahop_gemm_wgrad_ctx(const uint16_t* GY, const void* ctx,
                                               size_t ctx_bytes, int64_t T, int64_t Din,
                                               int64_t Dout, adahop_pattern pat_gy,
                                               adahop_pattern pat_x, adahop_route_t route,
                                               int32_t oe_rank, void* out,
                                               adahop_out_dtype out_dtype, void* ws,
                                               size_t ws_bytes, void* stream,
                                               void* const* stage_events);

/* As adahop_gemm, and if stage_events is not NULL it must hold
 * ADAHOP_STAGE_EVENTS created hipEvent_t handles: events[0] is recorded on
 * `stream` before the first launch and events[1..6] after the FOID, lhs
 * quantization, rhs quantization (which ends with reordering both scale
 * arrays for the GEMM), outlier product, GEMM main kernel and GEMM tail
 * stages (a stage that does not run records its event right after the
 * previous one). The tail is what finishes the main kernel's output: the
 * fixup of a split last round of tiles and, when the outlier product ran
 * inside the main kernel, its scatter into the extracted lines. With
 * OE_LEFT and OE_RIGHT the operand FOID does not scan is quantized in
 * FOID's launch (the FOID stage then holds both, and that operand's stage is
 * empty), on a second stream (its stage is empty here, the ROWS-layout scale
 * reordering falls in the GEMM stage, and the other stages overlap with it)
 * or in its own stage after FOID, as the notes at the top say. With route
 * BF16 the lhs and rhs stages are the operands' K-major copies, if any.
 * With the outlier product formed in the quantization (adahop_gemm_ex,
 * oe_in_quant), the stages follow that order: with OE_RIGHT the lhs stage is
 * empty and the lhs's quantization with the partial sums falls in the
 * outlier product's stage, with their sum. */
#define ADAHOP_STAGE_EVENTS 7
ADAHOP_API adahop_status adahop_gemm_timed(adahop_op op, const uint16_t* lhs,
                                           const uint16_t* rhs, int64_t T, int64_t Din,
                                           int64_t Dout, adahop_pattern pat_lhs,
                                           adahop_pattern pat_rhs, adahop_route_t route,
                                           int32_t oe_rank, void* out,
                                           adahop_out_dtype out_dtype, void* ws,
                                           size_t ws_bytes, void* stream,
                                           void* const* stage_events);

/* ---------------------------------------------------------------------------
 * Around the products: RMS norm, the linear layer on microscaled operands with
 * its epilogue, and their gradients. They share the conventions above (device
 * pointers, the caller's workspace, launches on `stream`, host checks before
 * any launch), except that infinities and NaNs are supported: they propagate.
 *
 * MXFP8 (OCP Microscaling v1.0): E4M3 codes, one byte each, [rows][ld_codes],
 * and one E8M0 scale byte per 32 consecutive elements of a row,
 * [rows][ld_scales]. Conversion to MXFP8 here: the scale exponent is the least
 * e with (block amax) <= 448 * 2^e, clamped to [-127, 127] and stored as the
 * byte e + 127 (0x00 for an all-zero block), so no element saturates; the
 * codes are v / 2^e rounded to nearest even. A block that holds an infinity
 * or a NaN gets the scale byte 0xFF and codes 0x7F (NaN).
 *
 * bf16 and fp32 matrices here may start at any element-aligned address and
 * have any leading dimension >= their columns (elements). Matrices with 0
 * rows are allowed: nothing is read, and column sums over them are 0. */
typedef enum { ADAHOP_MX_E2M1 = 0, ADAHOP_MX_E4M3 = 1 } adahop_mx_format;

/* MXFP8 codes and scales of src [rows, cols] (bf16 or fp32, `dtype`), and the
 * values that codes and scales stand for, in bf16 (where the values are exact
 * down to bf16's smallest subnormal) or fp32. cols must be a multiple of 32.
 * Errors: INVALID for NULL pointers (rows > 0), rows < 0, cols < 1 or not a
 * multiple of 32, a leading dimension too small, a bad dtype. */
ADAHOP_API adahop_status adahop_mx8_quant(const void* src, adahop_out_dtype dtype, int64_t rows,
                                          int64_t cols, int64_t ld, uint8_t* codes,
                                          int64_t ld_codes, uint8_t* scales, int64_t ld_scales,
                                          void* stream);
ADAHOP_API adahop_status adahop_mx8_dequant(const uint8_t* codes, int64_t ld_codes,
                                            const uint8_t* scales, int64_t ld_scales,
                                            int64_t rows, int64_t cols, void* dst,
                                            adahop_out_dtype dtype, int64_t ld, void* stream);

/* RMS norm of a residual stream. With a residual r (bf16 or fp32, the type of
 * the stream): h = x + r rounded to r's type, written to h (which may be r
 * itself); without (residual NULL): h = x, nothing is written. Then
 *   rstd = 1 / sqrt(mean_j h_j^2 + eps),   y_j = h_j * rstd * gain_j,
 * sums in fp32 (a row whose squares overflow it, from about 1.8e19 on, gets
 * rstd 0). y goes to codes and scales (MXFP8) and / or to y (bf16); at least
 * one is required. rstd (fp32 [rows]) may be NULL.
 * Errors: INVALID for missing pointers, cols < 1, rows < 0, leading dimensions
 * too small, a bad dtype, cols % 32 != 0 with an MXFP8 output, eps negative or
 * not finite, reserved not 0; UNSUPPORTED for cols > 32768 or more than
 * 2^31 - 1 rows. */
typedef struct {
  int64_t rows, cols;
  const void* x; int64_t ld_x;
  const void* residual; int64_t ld_residual;     /* NULL: none */
  const void* gain;                              /* [cols] */
  void* h; int64_t ld_h;                         /* required with a residual */
  uint16_t* y; int64_t ld_y;                     /* bf16, or NULL */
  uint8_t* codes; int64_t ld_codes;              /* MXFP8, or NULL */
  uint8_t* scales; int64_t ld_scales;
  float* rstd;
  int32_t x_dtype, residual_dtype, gain_dtype;   /* adahop_out_dtype */
  float eps;
  int32_t reserved[4];
} adahop_rmsnorm_args;

ADAHOP_API adahop_status adahop_rmsnorm(const adahop_rmsnorm_args* args, void* stream);

/* Gradient of the norm at h, given dy (the gradient of y; the MXFP8 rounding
 * is passed through) and, if not NULL, dh (the gradient that reaches h along
 * the residual stream), with n = h * rstd and u = gain * dy:
 *   dx = dh + rstd * (u - n * mean_j(u_j n_j)),   dgain = sum_rows dy * n.
 * dx is the gradient of x and of the residual alike; dx and dh have h's type,
 * and dx may be dh, dy or h itself (where the types agree). dgain is fp32
 * [cols], or NULL; its sums are taken in a fixed order and need
 * adahop_rmsnorm_backward_workspace_size(rows, cols) bytes of workspace (none
 * without dgain). Errors: as adahop_rmsnorm, and WORKSPACE. */
typedef struct {
  int64_t rows, cols;
  const void* dy; int64_t ld_dy;
  const void* h; int64_t ld_h;
  const void* gain;
  const float* rstd;
  const void* dh; int64_t ld_dh;                 /* NULL: none */
  void* dx; int64_t ld_dx;
  float* dgain;
  int32_t dy_dtype, h_dtype, gain_dtype;
  int32_t reserved[5];
} adahop_rmsnorm_backward_args;

ADAHOP_API size_t adahop_rmsnorm_backward_workspace_size(int64_t rows, int64_t cols);
ADAHOP_API adahop_status adahop_rmsnorm_backward(const adahop_rmsnorm_backward_args* args, void* ws,
                                                 size_t ws_bytes, void* stream);

/* Activations of a linear layer. GELU is z * Phi(z); GELU_TANH its tanh form
 * z / 2 * (1 + tanh(sqrt(2 / pi) * (z + 0.044715 z^3))). */
typedef enum {
  ADAHOP_ACT_NONE = 0,
  ADAHOP_ACT_RELU = 1,
  ADAHOP_ACT_SILU = 2,
  ADAHOP_ACT_GELU = 3,
  ADAHOP_ACT_GELU_TANH = 4
} adahop_act;

/* How a linear layer's products are formed. EXACT: exactly, on bf16 matrix
 * cores. SCALED: on the scaled matrix cores, which drop, within 8 products, what
 * lies under 2^-13 of the largest: within about 5e-5 of the result, root mean
 * square, on operands with outlier columns; a bf16 output's rounding hides
 * that, in an MXFP8 output it moves about one code in a thousand to its
 * neighbour. Both sum in fp32. EXACT reads B again for every 32 rows, so it is
 * for few rows above all; SCALED takes tiles. AUTO: EXACT for MXFP8 outputs of up to 32768 values (m * n),
 * SCALED for larger ones and for bf16. */
typedef enum {
  ADAHOP_PRODUCTS_AUTO = 0,
  ADAHOP_PRODUCTS_SCALED = 1,
  ADAHOP_PRODUCTS_EXACT = 2
} adahop_products;

/* Linear layer on microscaled operands:
 *   z = deq(A) * deq(B)^T + bias                             [m, N]
 *   out = act(z) + residual                                  [m, n], n = N
 *   gated: out = act(z[:, :n]) * z[:, n:] + residual         [m, n], n = N / 2
 * A: MXFP8 [m, K]. B: MXFP8 or MXFP4 [N, K] (MXFP4: codes as
 * adahop_iht_quant writes them, two to a byte, rows ld_b_codes bytes apart;
 * gated: the n gate rows, then the n up rows). The products are formed as
 * `products` says; sums over K, bias, activation and residual are in fp32, with
 * one rounding to the output: bf16 (out, ld_out elements) or, with out_scales
 * not NULL, MXFP8 (out: codes, ld_out bytes; n a multiple of 32). z (bf16
 * [m, N], or NULL) keeps z for adahop_act_backward. residual is bf16 and may be
 * out itself.
 * Needs up to adahop_linear_mx_workspace_size(...) bytes of 16-byte aligned
 * workspace, whatever the output's type (0 for few rows, else the scales in
 * another order and, where K is split, the parts' sums); none with EXACT
 * products.
 * Errors: INVALID for NULL operands or out (m > 0), m < 0, N or K < 1, K not
 * a multiple of 32, leading dimensions too small, N odd with gated, n not a
 * multiple of 32 with an MXFP8 output, a bad format, dtype, activation or products,
 * reserved not 0; UNSUPPORTED for codes of A or B that are not 16-byte
 * aligned or whose leading dimension is not a multiple of 16, for m, N or K of
 * 2^30 and more, a gated layer's N above 2^30 - 64, and for leading dimensions
 * of B's codes or scales of 2^25 bytes and more; WORKSPACE. */
typedef struct {
  int64_t m, N, K;
  const uint8_t* a_codes; int64_t ld_a_codes;
  const uint8_t* a_scales; int64_t ld_a_scales;
  const uint8_t* b_codes; int64_t ld_b_codes;
  const uint8_t* b_scales; int64_t ld_b_scales;
  const void* bias;                              /* [N], or NULL */
  const uint16_t* residual; int64_t ld_residual; /* NULL: none */
  void* out; int64_t ld_out;
  uint8_t* out_scales; int64_t ld_out_scales;    /* NULL: out is bf16 */
  uint16_t* z; int64_t ld_z;                     /* NULL: not kept */
  int32_t b_format;                              /* adahop_mx_format */
  int32_t bias_dtype;                            /* adahop_out_dtype */
  int32_t act;                                   /* adahop_act */
  int32_t gated;                                 /* 0 or 1 */
  int32_t products;                              /* adahop_products */
  int32_t reserved[3];
} adahop_linear_args;

ADAHOP_API size_t adahop_linear_mx_workspace_size(int64_t m, int64_t N, int64_t K,
                                                  adahop_mx_format b_format, int32_t gated);
/* What one call needs of it: 0 where its output's type and products need none
 * (and for arguments that adahop_linear_mx refuses). */
ADAHOP_API size_t adahop_linear_mx_args_workspace_size(const adahop_linear_args* args);
ADAHOP_API adahop_status adahop_linear_mx(const adahop_linear_args* args, void* ws,
                                          size_t ws_bytes, void* stream);

/* Gradient of that epilogue: from dout [m, n] (bf16 or fp32) and the kept z
 * (bf16 [m, N]) to dz (bf16 [m, N], the GY of adahop_gemm's DGRAD and WGRAD;
 * may be z itself)
 *   dz = dout * act'(z);   gated: dz = [dout * z_up * act'(z_gate),
 *                                       dout * act(z_gate)]
 * and, if not NULL, dbias = sum_rows dz (fp32 [N], summed before dz is
 * rounded, in a fixed order; it needs
 * adahop_act_backward_workspace_size(m, N, gated) bytes of workspace). The
 * residual's gradient is dout. Relu's slope at 0 is 0.
 * Errors: INVALID for NULL dout, z or dz (m > 0), m < 0, N < 1, N odd with
 * gated, leading dimensions too small, a bad dtype or activation;
 * UNSUPPORTED for m or N of 2^30 and more; WORKSPACE. */
ADAHOP_API size_t adahop_act_backward_workspace_size(int64_t m, int64_t N, int32_t gated);
ADAHOP_API adahop_status adahop_act_backward(const void* dout, adahop_out_dtype dout_dtype,
                                             int64_t ld_dout, const uint16_t* z, int64_t ld_z,
                                             int64_t m, int64_t N, adahop_act act, int32_t gated,
                                             uint16_t* dz, int64_t ld_dz, float* dbias, void* ws,
                                             size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Gradients from activations kept in MXFP8, as adahop_mx8_quant or a layer's
 * MXFP8 output writes them (checkpoints of 33 bytes in 32 elements). They are the
 * gradients of the functions at the kept values.
 *
 * adahop_act_backward's, from z [m, N] in MXFP8 (N a multiple of 32), and, if
 * `out` is not NULL, the layer's output made again beside it, so that it need
 * not be kept:
 *   out = act(z)   [m, n], n = N;   gated: act(z[:, :n]) * z[:, n:],  n = N / 2
 * in bf16 (without the residual). dz bf16 [m, N]; dbias fp32 [N] or NULL, with
 * adahop_act_backward_workspace_size(m, N, gated) bytes of workspace.
 * Errors: as adahop_act_backward, and INVALID for N not a multiple of 32 (gated:
 * n a multiple of 16 then), reserved not 0. */
typedef struct {
  int64_t m, N;
  const void* dout; int64_t ld_dout;             /* [m, n] */
  const uint8_t* z_codes; int64_t ld_z_codes;
  const uint8_t* z_scales; int64_t ld_z_scales;
  uint16_t* dz; int64_t ld_dz;
  uint16_t* out; int64_t ld_out;                 /* NULL: not wanted */
  float* dbias;                                  /* NULL: not wanted */
  int32_t dout_dtype;                            /* adahop_out_dtype */
  int32_t act, gated;
  int32_t reserved[5];
} adahop_act_backward_mx8_args;

ADAHOP_API adahop_status adahop_act_backward_mx8(const adahop_act_backward_mx8_args* args, void* ws,
                                                 size_t ws_bytes, void* stream);

/* adahop_rmsnorm_backward's, from h in MXFP8 (cols a multiple of 32) and the rstd
 * of the forward pass. dx and dh have the type dx_dtype; dx may be dh, or dy where
 * the types agree. Workspace as adahop_rmsnorm_backward's.
 * Errors: as adahop_rmsnorm_backward, and INVALID for cols not a multiple of 32. */
typedef struct {
  int64_t rows, cols;
  const void* dy; int64_t ld_dy;
  const uint8_t* h_codes; int64_t ld_h_codes;
  const uint8_t* h_scales; int64_t ld_h_scales;
  const void* gain;
  const float* rstd;
  const void* dh; int64_t ld_dh;                 /* NULL: none */
  void* dx; int64_t ld_dx;
  float* dgain;                                  /* NULL: not wanted */
  int32_t dy_dtype, dx_dtype, gain_dtype;
  int32_t reserved[5];
} adahop_rmsnorm_backward_mx8_args;

ADAHOP_API adahop_status adahop_rmsnorm_backward_mx8(const adahop_rmsnorm_backward_mx8_args* args,
                                                     void* ws, size_t ws_bytes, void* stream);

/* Weight gradient of a linear layer from its MXFP8 input X [T, Din] as it was
 * kept (the A operand of adahop_linear_mx), without a bf16 copy of it:
 *   dW [Dout, Din] = GY^T * X,   GY bf16 [T, Dout]
 * X's values are taken in bf16 as adahop_mx8_dequant gives them (those below
 * bf16's normal range, 2^-126, may count as 0), products are exact, sums fp32,
 * dW (bf16 or fp32) is rounded once. T is any; T = 0 gives zeros. Needs
 * adahop_gemm_wgrad_mx8_workspace_size(T, Din, Dout) bytes of 16-byte aligned
 * workspace (the parts of products split along T).
 * Errors: INVALID for T < 0, Din or Dout < 1, NULL GY, codes or scales (T > 0) or
 * out, leading dimensions too small, Din not a multiple of 32, a bad dtype,
 * reserved not 0; UNSUPPORTED for Dout or ld_gy that is not a multiple of 8,
 * ld_x_codes not a multiple of 16, GY or codes not 16-byte aligned, rows 8 MB or
 * more apart, T, Din or Dout of 2^30 and more, Din * Dout of 2^46 and more;
 * WORKSPACE. */
typedef struct {
  int64_t T, Din, Dout;
  const uint16_t* gy; int64_t ld_gy;
  const uint8_t* x_codes; int64_t ld_x_codes;
  const uint8_t* x_scales; int64_t ld_x_scales;
  void* out; int64_t ld_out;
  int32_t out_dtype;                             /* adahop_out_dtype */
  int32_t reserved[5];
} adahop_gemm_wgrad_mx8_args;

ADAHOP_API size_t adahop_gemm_wgrad_mx8_workspace_size(int64_t T, int64_t Din, int64_t Dout);
ADAHOP_API adahop_status adahop_gemm_wgrad_mx8(const adahop_gemm_wgrad_mx8_args* args, void* ws,
                                               size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Softmax cross entropy over a vocabulary, from hidden states h [T, D] and the
 * output layer's weights w [V, D], without keeping the logits:
 *   z = scale * h * w^T                                      [T, V]
 *   lse_t = log(sum_v exp(z_tv)),   loss_t = lse_t - z_t,y(t)
 * A target outside 0 .. V - 1 leaves its row out: loss 0; its lse is written.
 * Products of bf16 values are exact, sums, exponentials and logits fp32.
 * Infinities and NaNs propagate (a row of -inf has lse -inf).
 * Needs adahop_xent_workspace_size(rows, vocab) bytes of 16-byte aligned
 * workspace (32 bytes a row for every 256 entries of the vocabulary).
 * Errors: INVALID for rows < 0, vocab or dim < 1, NULL h, w, targets, loss or
 * lse (rows > 0), leading dimensions below dim, a bad target_dtype, a scale that
 * is not finite, reserved not 0; UNSUPPORTED for dim or a leading dimension of
 * h or w that is not a multiple of 8, h or w not 16-byte aligned, rows 8 MB or
 * more apart, rows or vocab of 2^30 and more, or rows * vocab of 2^46 and
 * more; WORKSPACE. */
typedef enum { ADAHOP_INDEX_I32 = 0, ADAHOP_INDEX_I64 = 1 } adahop_index_dtype;

typedef struct {
  int64_t rows, vocab, dim;                      /* T, V, D */
  const uint16_t* h; int64_t ld_h;               /* bf16 [T, D] */
  const uint16_t* w; int64_t ld_w;               /* bf16 [V, D] */
  const void* targets;                           /* [T] */
  float* loss;                                   /* [T] */
  float* lse;                                    /* [T] */
  float scale;
  int32_t target_dtype;                          /* adahop_index_dtype */
  int32_t reserved[4];
} adahop_xent_args;

ADAHOP_API size_t adahop_xent_workspace_size(int64_t rows, int64_t vocab);
ADAHOP_API adahop_status adahop_xent(const adahop_xent_args* args, void* ws, size_t ws_bytes,
                                     void* stream);

/* How the gradient of the logits, g, is held between its products. SPLIT: as the
 * sum of two bf16 numbers, off by at most 2^-16 of each element. BF16: as the
 * nearest bf16, off by at most 2^-8 of each element, with three fifths of the
 * operations (2.3e-3 to 2.6e-3 of dh and dw in the root mean square, where bf16
 * outputs' own rounding is 1.7e-3). */
typedef enum { ADAHOP_XENT_G_SPLIT = 0, ADAHOP_XENT_G_BF16 = 1 } adahop_xent_g;

/* Its gradient, from dloss (fp32 [T], the gradient of each row's loss) and, if
 * not NULL, dlse (fp32 [T], that of each row's lse, as a penalty on the
 * normalizer gives it), with the lse that adahop_xent returned:
 *   g_tv = scale * ((dloss_t + dlse_t) * exp(z_tv - lse_t) - dloss_t * [v = y(t)])
 *   dh = g * w   [T, D],      dw = g^T * h   [V, D]
 * dloss of a row that is left out does not count; its dlse does. dh and dw are
 * bf16 or fp32; either may be NULL. The logits are formed again, `piece` entries
 * of the vocabulary at a time (0: as many as keep g within 1 GiB, but 256, which
 * take more past 2^20 rows (BF16: 2^21); rounded up to a multiple of 256); g of a piece is held as `g` says, sums are fp32,
 * dh and dw are rounded once. Where SPLIT's second numbers meet an infinity of h
 * or w, the sum may be a NaN instead of an infinity. Needs
 * adahop_xent_backward_args_workspace_size(args) bytes of 16-byte aligned
 * workspace (0 for arguments that the call refuses): 4 (BF16: 2) * rows * piece
 * (rows rounded up to a multiple of 64) for g, dh
 * in fp32 where there are several pieces, and the parts of products split over
 * their sums.
 * Errors: as adahop_xent, and INVALID for NULL lse or dloss (rows > 0), dh and dw
 * both NULL (rows > 0), ld_dh or ld_dw below dim, a bad dtype or g, piece < 0; UNSUPPORTED for
 * rows of 2^22 and more. */
typedef struct {
  int64_t rows, vocab, dim;
  const uint16_t* h; int64_t ld_h;
  const uint16_t* w; int64_t ld_w;
  const void* targets;
  const float* lse;
  const float* dloss;
  const float* dlse;                             /* NULL: none */
  void* dh; int64_t ld_dh;                       /* NULL: not wanted */
  void* dw; int64_t ld_dw;
  int64_t piece;
  float scale;
  int32_t target_dtype;
  int32_t dh_dtype, dw_dtype;                    /* adahop_out_dtype */
  int32_t g;                                     /* adahop_xent_g */
  int32_t reserved[3];
} adahop_xent_backward_args;

ADAHOP_API size_t adahop_xent_backward_args_workspace_size(const adahop_xent_backward_args* args);
ADAHOP_API adahop_status adahop_xent_backward(const adahop_xent_backward_args* args, void* ws,
                                              size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* ADAHOP_H */
