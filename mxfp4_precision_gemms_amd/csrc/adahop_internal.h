// Internal declarations of the AdaHOP HIP library (gfx950). Not installed.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>
#include <string>

#include "../../include/adahop.h"
#include "linear_plan.h"

namespace adahop {

// Per-thread error detail, set by fail().
void set_error(const std::string& msg);
adahop_status fail(adahop_status st, const std::string& msg);
adahop_status check_launch(const char* what);

inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
constexpr size_t kAlign = 256;
constexpr int kMaxK = 1024;  // largest outlier rank (FOID top-k, OE lines)

// ---- FOID -----------------------------------------------------------------
size_t foid_workspace_bytes(int64_t ncand, int32_t k);
// Whether foid_launch's grid fits (false: it would return UNSUPPORTED).
bool foid_fits(int64_t ncand, int32_t k);
// FOID's score of every candidate line, fp64 [ncand], on the device.
adahop_status line_scores_launch(const uint16_t* t, int64_t rows, int64_t cols, int64_t ld, int axis,
                                 int32_t probe, double* out, hipStream_t stream);
// The quantization (IHT over blocks of 32, MXFP4) of an operand with no
// extracted lines that FOID may run in its own launch. contract ROWS (blocks
// down the columns): src [K][outer]; contract COLS (blocks along the rows):
// src [outer][K]; row stride ld; codes and scales as iht_quant_launch writes
// them for that layout; stream_src as there.
struct QuantBeside {
  const uint16_t* src;
  int64_t K, outer, ld;
  uint8_t* codes;
  uint8_t* scales;
  int layout;
  int contract;
  bool stream_src;
};
// Whether FOID's selection over ncand candidates fits one launch of
// 256-thread workgroups (k <= 256, at most two levels) that also runs q's
// quantization (q suits the vectorized quantizer tiles of its direction).
bool foid_beside_fits(int64_t ncand, int32_t k, const QuantBeside& q);
// With `beside` and foid_beside_fits, the selection's workgroups and that
// quantization's share one launch and *beside_done is set; otherwise FOID
// runs as without it and the caller quantizes the operand itself.
adahop_status foid_launch(const uint16_t* t, int64_t rows, int64_t cols, int64_t ld, int axis,
                          int32_t probe, int32_t k, int32_t* idx_out, void* ws, size_t ws_bytes,
                          hipStream_t stream, const QuantBeside* beside = nullptr,
                          bool* beside_done = nullptr);

// ---- zero + gather + IHT + MXFP4 ------------------------------------------
// Whether iht_quant_launch's grid fits (false: it would return UNSUPPORTED).
bool iht_quant_fits(int64_t rows, int64_t cols, int contract);
// stream_src: load the source non-temporally (it is read once); false keeps
// it in the caches for a kernel that reads it again soon after (the outer
// outlier product's wide factor).
adahop_status iht_quant_launch(const uint16_t* src, int64_t rows, int64_t cols, int64_t ld,
                               int contract, int32_t hadamard_block, const int32_t* zero_idx,
                               int32_t nzero, int zero_axis, uint8_t* codes, uint8_t* scales,
                               uint16_t* gathered, int layout, hipStream_t stream,
                               bool stream_src = true);

// The one-read variant of OE_LEFT / OE_RIGHT: the operand FOID does not scan,
// quantized down its columns (contract ROWS, K = rows), also forms the outer
// outlier product's partial sums P_s = (its columns) x lines^T over group s
// of K, fp32, in `partials` ([groups][cols][k], or [groups][k][cols] with
// by_line), from the k extracted lines ([k][K] bf16, 16-byte aligned).
// iht_quant_oe_groups returns the number of groups (0 if k > 64 or the
// sizes do not fit).
int iht_quant_oe_groups(int64_t K, int64_t outer, int32_t k, int* tiles_per_wg);
adahop_status iht_quant_oe_launch(const uint16_t* src, int64_t rows, int64_t cols, int64_t ld,
                                  uint8_t* codes, uint8_t* scales, int layout,
                                  const uint16_t* lines, int32_t k, int by_line, float* partials,
                                  hipStream_t stream);

// ---- outlier product (bf16 MFMA) ------------------------------------------
// P_s[x][y] = sum over t in split s of X(x, t) * Y(y, t), fp32, for s < splits,
// laid out [splits][nx][ny] in `partials`, followed by their sum P [nx][ny]
// (so `partials` holds (splits + 1) * nx * ny floats).
struct Bf16View {
  const uint16_t* ptr;
  int64_t ld;
  int inner_contiguous;
};
int oe_splits(int64_t nx, int64_t ny, int64_t K);
// Whether the outlier product's grid fits (false: oe_product_launch would
// return UNSUPPORTED).
bool oe_product_fits(int64_t nx, int64_t ny);
adahop_status oe_product_launch(Bf16View X, Bf16View Y, int64_t nx, int64_t ny, int64_t K,
                                int splits, float* partials, hipStream_t stream);
// P = sum over s < splits of partials[s] (each `count` floats), in the order
// s = 0, 1, ..., written right after the partials.
adahop_status oe_reduce_launch(float* partials, int splits, int64_t count, hipStream_t stream);
// Full bf16 product written to C (the BF16 route): C[i][j] = sum_t X(i,t) Y(j,t).
adahop_status bf16_gemm_launch(Bf16View X, Bf16View Y, int64_t m, int64_t n, int64_t K,
                               void* C, int64_t ldc, int out_f32, hipStream_t stream);
// The same product on the FP4 GEMM's ring kernel with bf16 matrix cores,
// K % 128 == 0 (bf16_ring_ok). Each operand is 16-byte aligned and either
// along K (a [m, K] row-major, row stride K) or, with *_across, stored
// across K (a [K, lda] row-major holding a(i, t) at t * lda + i; lda % 8 ==
// 0 and under 2 GiB: bf16_ring_across_ok). `scratch` holds
// bf16_ring_scratch_bytes(m, n, K) bytes (the split tiles' fp32 parts,
// 16-byte aligned).
bool bf16_ring_ok(int64_t m, int64_t n, int64_t K);
bool bf16_ring_across_ok(int64_t K, int64_t ld);
size_t bf16_ring_scratch_bytes(int64_t m, int64_t n, int64_t K);
adahop_status bf16_ring_launch(const uint16_t* a, int a_across, int64_t lda, const uint16_t* b,
                               int b_across, int64_t ldb, int64_t m, int64_t n, int64_t K, void* C,
                               int64_t ldc, int out_f32, void* scratch, size_t scratch_bytes,
                               hipStream_t stream, hipEvent_t main_done = nullptr);
// dst [cols, rows] (leading dim rows) = transpose of src [rows, cols]
// (leading dim ld).
adahop_status bf16_transpose_launch(const uint16_t* src, int64_t rows, int64_t cols, int64_t ld,
                                    uint16_t* dst, hipStream_t stream);
bool bf16_transpose_fits(int64_t rows, int64_t cols);

// ---- FP4 GEMM with the OE epilogue ----------------------------------------
struct OeEpilogue {
  int mode;                 // 0 none, ADAHOP_ROUTE_OE_LEFT / _OE_RIGHT / _OE_INNER
  int32_t k;
  const int32_t* idx;       // OE_LEFT / OE_RIGHT
  const float* partials;    // OE_LEFT: [splits][k][n]; OE_RIGHT: [splits][m][k]; then P
  int splits;
  Bf16View a, b;            // OE_INNER factors: a [m][k], b [n][k]; OE_LEFT / OE_RIGHT:
                            // the outlier product's factors, as for oe_product_launch
  // OE_LEFT / OE_RIGHT computed inside the GEMM launch (fused_parts > 0, from
  // oe_fused_parts): `fused_ws` holds oe_fused_bytes(...) bytes, 16-byte
  // aligned, for the partial sums and the extracted lines' residual.
  int fused_parts;
  float* fused_ws;
};
// K-parts of the outer outlier product (OE_LEFT / OE_RIGHT, X = a, Y = b as
// in oe_product_launch) when it runs as work items of the main GEMM kernel,
// or 0 when it runs as oe_product_kernel before the GEMM: k <= 64, the main
// kernel applies to (m, n, K), the wide factor (a for OE_RIGHT, b for
// OE_LEFT) is stored across K with a row of a multiple of 8 elements under
// 2 GiB, the lines (the other factor) run along K in rows of a multiple of 8
// elements; with check_ptrs, both 16-byte aligned.
int oe_fused_parts(int64_t m, int64_t n, int64_t K, int mode, int32_t k, Bf16View a, Bf16View b,
                   bool check_ptrs);
// Whether gemm_mx_launch runs the main (ring) kernel for these operands.
bool gemm_mx_ring_used(const uint8_t* a_codes, const uint8_t* a_scales, const uint8_t* b_codes,
                       const uint8_t* b_scales, int64_t m, int64_t n, int64_t K, int layout);
// Workspace of the fused outlier product: parts x wide x k partial sums plus
// wide x k residuals, fp32.
size_t oe_fused_bytes(int64_t m, int64_t n, int mode, int32_t k, int parts);
// Workspace the GEMM needs for (m, n, K) in `layout`, when the main kernel
// applies (K % 512 == 0), else 0: for ROWS, stage-major copies of both scale
// arrays ([K/128][rows] words; gemm_mx_stage_scales writes them), then, for
// both layouts, the fp32 parts of the tiles the main kernel splits along K
// in its last round (256 KB per part).
size_t gemm_mx_scratch_bytes(int64_t m, int64_t n, int64_t K, int layout);
// Whether (m, n, K) operands may be packed K-chunked (ADAHOP_LAYOUT_KCHUNK):
// the main kernel applies and stage offsets fit 31 bits.
bool gemm_mx_kchunk_ok(int64_t m, int64_t n, int64_t K);
// Whether the GEMM's tile count fits (false: gemm_mx_launch would return
// UNSUPPORTED).
bool gemm_mx_fits(int64_t m, int64_t n);
adahop_status gemm_mx_stage_scales(const uint8_t* a_codes, const uint8_t* a_scales,
                                   const uint8_t* b_codes, const uint8_t* b_scales, int64_t m,
                                   int64_t n, int64_t K, void* scratch, size_t scratch_bytes,
                                   hipStream_t stream);
// layout ROWS: scales reordered by gemm_mx_stage_scales into `scratch` when
// the main kernel applies; KCHUNK: operands as ADAHOP_LAYOUT_KCHUNK. `scratch`
// holds gemm_mx_scratch_bytes(m, n, K, layout) bytes.
adahop_status gemm_mx_launch(const uint8_t* a_codes, const uint8_t* a_scales,
                             const uint8_t* b_codes, const uint8_t* b_scales, int64_t m,
                             int64_t n, int64_t K, int layout, const OeEpilogue& oe, void* C,
                             int64_t ldc, int out_f32, void* scratch, size_t scratch_bytes,
                             hipStream_t stream, hipEvent_t main_done = nullptr);
// Both GEMM launchers record `main_done` (if not null) on `stream` right
// after the main kernel, before the kernels that finish its output (the
// split fixup, the outlier scatter).
adahop_status record_main_done(hipEvent_t main_done, hipStream_t stream, const char* what);

// Compute units of the current device (256 where none can be asked).
int64_t compute_units();

// ---- norm, quantizer and linear layer in MXFP8 ------------------------------
// Arguments as the public entry points', already checked; leading dimensions
// in elements (codes and scales in bytes).
adahop_status rmsnorm_launch(const void* x, int x_f32, const void* r, int r_f32, const void* gain,
                             int gain_f32, int64_t rows, int64_t cols, int64_t ldx, int64_t ldr,
                             float eps, void* h, int64_t ldh, uint16_t* y, int64_t ldy,
                             uint8_t* codes, int64_t ldc, uint8_t* scales, int64_t lds, float* rstd,
                             hipStream_t stream);
// Workgroups of the backward kernel: `partial` holds that many rows of cols
// fp32 (unused, may be null, without dgain).
int rmsnorm_backward_groups(int64_t rows, int64_t cols);
adahop_status rmsnorm_backward_launch(const void* dy, int dy_f32, const void* h, int h_f32,
                                      const void* gain, int gain_f32, const float* rstd,
                                      const void* dh, int64_t rows, int64_t cols, int64_t lddy,
                                      int64_t ldh, int64_t lddh, int64_t lddx, void* dx,
                                      float* dgain, float* partial, hipStream_t stream);
// out[c] = sum over p < parts of partial[p][c], in a fixed order.
adahop_status column_reduce_launch(const float* partial, int parts, int64_t cols, float* out,
                                   hipStream_t stream);
adahop_status mx8_quant_launch(const void* src, int f32, int64_t rows, int64_t cols, int64_t ld,
                               uint8_t* codes, int64_t ldc, uint8_t* scales, int64_t lds,
                               hipStream_t stream);
adahop_status mx8_dequant_launch(const uint8_t* codes, int64_t ldc, const uint8_t* scales, int64_t lds,
                                 int64_t rows, int64_t cols, void* dst, int f32, int64_t ldd,
                                 hipStream_t stream);
// Row groups of the epilogue's backward kernel: `partial` holds that many
// rows of n (gated: 2 n) fp32 (unused without dbias).
int64_t act_backward_groups(int64_t m, int64_t n);
adahop_status act_backward_launch(const void* dout, int d_f32, const uint16_t* z, int act, int gated,
                                  int64_t m, int64_t n, int64_t lddo, int64_t ldz, uint16_t* dz,
                                  int64_t lddz, float* dbias, float* partial, hipStream_t stream);

// The same from z, or h, kept in MXFP8 (leading dimensions in bytes); dx and dh
// are of dx_f32's type, out (bf16, or null) is act(z) [* z_up] again.
struct Mx8Matrix {
  const uint8_t* codes;
  int64_t ldc;
  const uint8_t* scales;
  int64_t lds;
};
adahop_status act_backward_mx8_launch(const void* dout, int d_f32, int64_t lddo, const Mx8Matrix& z, int act,
                                      int gated, int64_t m, int64_t n, uint16_t* dz, int64_t lddz, uint16_t* out,
                                      int64_t ldout, float* dbias, float* partial, hipStream_t stream);
adahop_status rmsnorm_backward_mx8_launch(const void* dy, int dy_f32, int64_t lddy, const Mx8Matrix& h,
                                          const void* gain, int gain_f32, const float* rstd, const void* dh,
                                          int64_t lddh, int64_t rows, int64_t cols, void* dx, int dx_f32,
                                          int64_t lddx, float* dgain, float* partial, hipStream_t stream);

struct LinearArgs {
  const uint8_t* a_codes;
  const uint8_t* a_scales;
  const uint8_t* b_codes;
  const uint8_t* b_scales;
  int64_t lda, ldas, ldb, ldbs;
  int64_t m, n, K;           // n: output columns (gated: B has 2 n rows)
  const void* bias;          // [N] or null
  int bias_f32;
  int act;                   // adahop_act
  const uint16_t* residual;  // bf16 [m][n] or null
  int64_t ldr;
  void* out;                 // bf16, or E4M3 codes with out_scales
  int64_t ldo;
  uint8_t* out_scales;       // null for a bf16 output
  int64_t ldos;
  uint16_t* z;               // bf16 [m][N] or null
  int64_t ldz;
};

// Whether the rows of a matrix, a tile's rows past its end included, lie
// within the 31-bit offsets that the tile kernel uses.
bool linear_tiles_reach(int64_t rows, int64_t ld);
adahop_status linear_tiles_launch(const LinearArgs& a, int b_fp4, int gated, const TilePlan& p, void* scratch,
                                  hipStream_t stream);
// Scaled products need scratch, exact ones none.
size_t linear_mx_scratch_bytes(int64_t m, int64_t n, int64_t K, int b_fp4, int gated, bool mx8_out);
adahop_status linear_mx_launch(const LinearArgs& a, int b_fp4, int gated, bool exact, void* scratch,
                               hipStream_t stream);

// ---- products of bf16 operands in tiles ---------------------------------------
// C[i, j] = sum_k A(i, k) B(j, k) of bf16 operands, in fp32; then, on top of
// `prev` (fp32 [m][ld_prev], or null), rounded to bf16 or stored in fp32. A lies
// along K ([m][K]) or across it ([K][m]), B across ([K][n]), or, with A across,
// in MXFP8 across ([K][n] codes, scales per 32 columns). Leading dimensions of
// operands in bytes, those of bf16 multiples of 16 and below 8 MB; 16-byte
// aligned; K of an A along it may end inside 16 bytes if zeros follow in them; n a
// multiple of 8 (codes: 32), m of an A across it likewise, or A's rows reach to the
// next multiple; an A in chunks of 64 columns has zeros from row K up to a multiple
// of 64, and 4 chunks are below 2 GB; m, n, K below 2^30, m * n below 2^46. ws:
// tile_product_bytes(...) bytes.
struct TileOperand {
  const void* p;
  int64_t ld;
  int64_t chunk;             // A: bytes from 64 columns to the next 64 (128: plain rows)
  const uint8_t* scales;
  int64_t ld_scales;
  int kind;                  // tiles::Kind
  int64_t term = 0;          // A the sum of two such matrices (B bf16): bytes from one to the other
};
struct TileOut {
  void* p;
  int64_t ld;
  int f32;
  const float* prev;
  int64_t ld_prev;
};
// a, b: the operands' kinds.
size_t tile_product_bytes(int64_t m, int64_t n, int64_t K, int a, int b);
adahop_status tile_product_launch(const TileOperand& a, const TileOperand& b, int64_t m, int64_t n, int64_t K,
                                  const TileOut& out, float* ws, hipStream_t stream);

// dW [Dout, Din] = GY^T X from X in MXFP8, checked; ws: wgrad_mx8_ws_bytes bytes.
size_t wgrad_mx8_ws_bytes(int64_t T, int64_t Din, int64_t Dout);
adahop_status wgrad_mx8_launch(const uint16_t* gy, int64_t ldgy, const Mx8Matrix& x, int64_t T, int64_t Din,
                               int64_t Dout, void* out, int out_f32, int64_t ldo, float* ws, hipStream_t stream);

// ---- cross entropy over a vocabulary ----------------------------------------
// Arguments as the public entry points', already checked; T > 0 in xent_launch.
struct XentArgs {
  int64_t T, V, D;
  const uint16_t* h;
  int64_t ldh;
  const uint16_t* w;
  int64_t ldw;
  const void* targets;
  int wide_targets;          // int64, else int32
  float scale;
};
struct XentGrad {
  const float* lse;
  const float* dloss;
  const float* dlse;         // or null
  void* dh;                  // or null
  int64_t lddh;
  int dh_f32;
  void* dw;                  // or null
  int64_t lddw;
  int dw_f32;
  int terms;                 // bf16 numbers that hold an element of g: 1 or 2
};
size_t xent_ws_bytes(int64_t T, int64_t V);
adahop_status xent_launch(const XentArgs& a, float* loss, float* lse, void* ws, hipStream_t stream);
size_t xent_backward_ws_bytes(int64_t T, int64_t V, int64_t D, int64_t piece, int terms, bool dh, bool dw);
adahop_status xent_backward_launch(const XentArgs& a, const XentGrad& b, int64_t piece, void* ws,
                                   hipStream_t stream);

}  // namespace adahop
