// Host side of the norm, MXFP8, linear-layer and cross-entropy entry points:
// argument checks and launches. Every check runs before the first launch; nothing allocates
// device memory or synchronizes.
#include <atomic>
#include <cmath>
#include <new>
#include <string>

#include "adahop_internal.h"

namespace adahop {
namespace {

constexpr int64_t kMaxCols = 32768;                 // columns of a norm's row
constexpr int64_t kMaxRows = (int64_t{1} << 31) - 1;
constexpr int64_t kMaxDim = int64_t{1} << 30;       // sizes of a product
constexpr int64_t kMaxRowBytes = int64_t{1} << 25;  // row of its weights

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool valid_dtype(int d) { return d == ADAHOP_OUT_BF16 || d == ADAHOP_OUT_F32; }

adahop_status invalid(const char* what) { return fail(ADAHOP_ERR_INVALID, what); }
adahop_status unsupported(const char* what) { return fail(ADAHOP_ERR_UNSUPPORTED, what); }

adahop_status need_workspace(const void* ws, size_t have, size_t need, const char* who) {
  if (need == 0) return ADAHOP_OK;
  if (ws == nullptr || have < need)
    return fail(ADAHOP_ERR_WORKSPACE, std::string(who) + ": workspace of " + std::to_string(need) +
                                          " bytes needed");
  if (!aligned16(ws)) return unsupported("workspace must be 16-byte aligned");
  return ADAHOP_OK;
}

// No C++ exception (an error message that cannot be allocated) leaves a C
// entry point.
template <typename F>
adahop_status entry(F&& f) noexcept {
  try {
    set_error("");
    return f();
  } catch (...) {
    return ADAHOP_ERR_INVALID;
  }
}

#define ADAHOP_TRY(expr)                         \
  do {                                           \
    const adahop_status st_ = (expr);            \
    if (st_ != ADAHOP_OK) return st_;            \
  } while (0)

template <size_t N>
bool all_zero(const int32_t (&r)[N]) {
  for (int32_t v : r)
    if (v != 0) return false;
  return true;
}

adahop_status check_mx8(int64_t rows, int64_t cols, int64_t ld, int64_t ldc, int64_t lds, int dtype) {
  if (rows < 0 || cols < 1) return invalid("mx8: rows must be >= 0 and cols >= 1");
  if (cols % 32 != 0) return invalid("mx8: cols must be a multiple of 32");
  if (!valid_dtype(dtype)) return invalid("mx8: bad dtype");
  if (ld < cols || ldc < cols || lds < cols / 32) return invalid("mx8: leading dimension too small");
  return ADAHOP_OK;
}

adahop_status check_norm_sizes(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 1) return invalid("rmsnorm: rows must be >= 0 and cols >= 1");
  if (cols > kMaxCols) return unsupported("rmsnorm: more than 32768 columns");
  if (rows > kMaxRows) return unsupported("rmsnorm: more than 2^31 - 1 rows");
  return ADAHOP_OK;
}

adahop_status norm(const adahop_rmsnorm_args* a, hipStream_t stream) {
  if (a == nullptr) return invalid("rmsnorm: null arguments");
  ADAHOP_TRY(check_norm_sizes(a->rows, a->cols));
  if (!all_zero(a->reserved)) return invalid("rmsnorm: reserved fields must be 0");
  if (!valid_dtype(a->x_dtype) || !valid_dtype(a->gain_dtype)) return invalid("rmsnorm: bad dtype");
  if (!(a->eps >= 0.0f) || std::isinf(a->eps)) return invalid("rmsnorm: eps must be finite and >= 0");
  if (a->ld_x < a->cols) return invalid("rmsnorm: ld_x below cols");
  if (a->rows == 0) return ADAHOP_OK;
  if (a->x == nullptr || a->gain == nullptr) return invalid("rmsnorm: null x or gain");
  if (a->residual != nullptr) {
    if (!valid_dtype(a->residual_dtype)) return invalid("rmsnorm: bad residual dtype");
    if (a->h == nullptr) return invalid("rmsnorm: a residual needs h");
    if (a->ld_residual < a->cols || a->ld_h < a->cols)
      return invalid("rmsnorm: ld_residual or ld_h below cols");
  }
  if (a->y == nullptr && a->codes == nullptr) return invalid("rmsnorm: neither y nor codes");
  if (a->y != nullptr && a->ld_y < a->cols) return invalid("rmsnorm: ld_y below cols");
  if (a->codes != nullptr) {
    if (a->scales == nullptr) return invalid("rmsnorm: codes without scales");
    if (a->cols % 32 != 0) return invalid("rmsnorm: an MXFP8 output needs cols in multiples of 32");
    if (a->ld_codes < a->cols || a->ld_scales < a->cols / 32)
      return invalid("rmsnorm: ld_codes or ld_scales too small");
  }
  return rmsnorm_launch(a->x, a->x_dtype, a->residual, a->residual_dtype, a->gain, a->gain_dtype,
                        a->rows, a->cols, a->ld_x, a->ld_residual, a->eps, a->h, a->ld_h, a->y,
                        a->ld_y, a->codes, a->ld_codes, a->scales, a->ld_scales, a->rstd, stream);
}

size_t norm_back_bytes(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 1 || cols > kMaxCols) return 0;
  return (size_t)rmsnorm_backward_groups(rows, cols) * (size_t)cols * sizeof(float);
}

adahop_status norm_back(const adahop_rmsnorm_backward_args* a, void* ws, size_t ws_bytes,
                        hipStream_t stream) {
  if (a == nullptr) return invalid("rmsnorm_backward: null arguments");
  ADAHOP_TRY(check_norm_sizes(a->rows, a->cols));
  if (!all_zero(a->reserved)) return invalid("rmsnorm_backward: reserved fields must be 0");
  if (!valid_dtype(a->dy_dtype) || !valid_dtype(a->h_dtype) || !valid_dtype(a->gain_dtype))
    return invalid("rmsnorm_backward: bad dtype");
  if (a->ld_dy < a->cols || a->ld_h < a->cols || a->ld_dx < a->cols ||
      (a->dh != nullptr && a->ld_dh < a->cols))
    return invalid("rmsnorm_backward: leading dimension below cols");
  if (a->gain == nullptr) return invalid("rmsnorm_backward: null gain");
  if (a->rows > 0 && (a->dy == nullptr || a->h == nullptr || a->rstd == nullptr || a->dx == nullptr))
    return invalid("rmsnorm_backward: null dy, h, rstd or dx");
  if (a->rows == 0 && a->dgain == nullptr) return ADAHOP_OK;
  if (a->dgain != nullptr)
    ADAHOP_TRY(need_workspace(ws, ws_bytes, norm_back_bytes(a->rows, a->cols), "rmsnorm_backward"));
  return rmsnorm_backward_launch(a->dy, a->dy_dtype, a->h, a->h_dtype, a->gain, a->gain_dtype, a->rstd,
                                 a->dh, a->rows, a->cols, a->ld_dy, a->ld_h, a->ld_dh, a->ld_dx,
                                 a->dx, a->dgain, static_cast<float*>(ws), stream);
}

bool valid_product(int64_t m, int64_t N, int64_t K, int32_t gated) {
  return m >= 0 && N >= 1 && K >= 1 && K % 32 == 0 && m < kMaxDim && K < kMaxDim &&
         (gated ? N <= kMaxGatedN : N < kMaxDim);
}

// Workspace of a call whose sizes, format and products are valid.
size_t linear_bytes(const adahop_linear_args& a) {
  const int64_t n = a.gated ? a.N / 2 : a.N;
  const bool mx8_out = a.out_scales != nullptr;
  if (a.m == 0 || exact_products(a.products, mx8_out, a.m, n)) return 0;
  return linear_mx_scratch_bytes(a.m, n, a.K, a.b_format == ADAHOP_MX_E2M1, a.gated, mx8_out);
}

adahop_status linear(const adahop_linear_args* a, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (a == nullptr) return invalid("linear_mx: null arguments");
  if (a->m < 0 || a->N < 1 || a->K < 1) return invalid("linear_mx: m must be >= 0, N and K >= 1");
  if (a->K % 32 != 0) return invalid("linear_mx: K is not a multiple of 32");
  if (!valid_product(a->m, a->N, a->K, a->gated))
    return unsupported("linear_mx: m, N or K of 2^30 or more, or a gated layer's N above 2^30 - 64");
  if (!all_zero(a->reserved)) return invalid("linear_mx: reserved fields must be 0");
  if (a->b_format != ADAHOP_MX_E2M1 && a->b_format != ADAHOP_MX_E4M3)
    return invalid("linear_mx: bad b_format");
  if (a->act < ADAHOP_ACT_NONE || a->act > ADAHOP_ACT_GELU_TANH)
    return invalid("linear_mx: bad activation");
  if (a->gated != 0 && a->gated != 1) return invalid("linear_mx: gated must be 0 or 1");
  if (a->products < ADAHOP_PRODUCTS_AUTO || a->products > ADAHOP_PRODUCTS_EXACT)
    return invalid("linear_mx: bad products");
  if (a->gated && a->N % 2 != 0) return invalid("linear_mx: a gated layer needs an even N");
  const int64_t n = a->gated ? a->N / 2 : a->N;
  const bool fp4 = a->b_format == ADAHOP_MX_E2M1;
  if (a->ld_a_codes < a->K || a->ld_b_codes < (fp4 ? a->K / 2 : a->K) || a->ld_a_scales < a->K / 32 ||
      a->ld_b_scales < a->K / 32)
    return invalid("linear_mx: leading dimension of A or B too small");
  if (a->ld_out < n) return invalid("linear_mx: ld_out too small");
  if (a->m == 0) return ADAHOP_OK;
  if (!a->a_codes || !a->a_scales || !a->b_codes || !a->b_scales || !a->out)
    return invalid("linear_mx: null operand or out");
  if (a->bias != nullptr && !valid_dtype(a->bias_dtype)) return invalid("linear_mx: bad bias dtype");
  if (a->residual != nullptr && a->ld_residual < n) return invalid("linear_mx: ld_residual too small");
  if (a->z != nullptr && a->ld_z < a->N) return invalid("linear_mx: ld_z too small");
  if (a->out_scales != nullptr) {
    if (n % 32 != 0) return invalid("linear_mx: an MXFP8 output needs columns in multiples of 32");
    if (a->ld_out_scales < n / 32) return invalid("linear_mx: ld_out_scales too small");
  }
  if (!aligned16(a->a_codes) || !aligned16(a->b_codes) || a->ld_a_codes % 16 != 0 ||
      a->ld_b_codes % 16 != 0)
    return unsupported("linear_mx: codes of A and B must be 16-byte aligned, rows included");
  if (a->ld_b_codes >= kMaxRowBytes || a->ld_b_scales >= kMaxRowBytes)
    return unsupported("linear_mx: rows of B 32 MB or more apart");
  ADAHOP_TRY(need_workspace(ws, ws_bytes, linear_bytes(*a), "linear_mx"));
  const LinearArgs g = {a->a_codes, a->a_scales, a->b_codes, a->b_scales, a->ld_a_codes,
                        a->ld_a_scales, a->ld_b_codes, a->ld_b_scales, a->m, n, a->K, a->bias,
                        a->bias_dtype, a->act, a->residual, a->ld_residual, a->out, a->ld_out,
                        a->out_scales, a->ld_out_scales, a->z, a->ld_z};
  return linear_mx_launch(g, fp4, a->gated, exact_products(a->products, a->out_scales != nullptr, a->m, n), ws,
                          stream);
}

size_t act_back_bytes(int64_t m, int64_t N, int32_t gated) {
  if (m < 0 || N < 1 || m >= kMaxDim || N >= kMaxDim || (gated && N % 2 != 0)) return 0;
  return (size_t)act_backward_groups(m, gated ? N / 2 : N) * (size_t)N * sizeof(float);
}

// ---- gradients from MXFP8 -------------------------------------------------------
constexpr int64_t kMaxTiled = int64_t{1} << 46;     // rows * columns of a product: 2^30 tiles
constexpr int64_t kMaxTileRow = int64_t{1} << 23;   // bytes from an operand's row to the next

// m * n, both at most 2^30.
bool tiles_fit(int64_t m, int64_t n) { return m * n < kMaxTiled; }

adahop_status act_back_mx8(const adahop_act_backward_mx8_args* a, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (a == nullptr) return invalid("act_backward_mx8: null arguments");
  if (a->m < 0 || a->N < 1) return invalid("act_backward_mx8: m must be >= 0 and N >= 1");
  if (a->m >= kMaxDim || a->N >= kMaxDim) return unsupported("act_backward_mx8: m or N of 2^30 or more");
  if (!all_zero(a->reserved)) return invalid("act_backward_mx8: reserved fields must be 0");
  if (a->act < ADAHOP_ACT_NONE || a->act > ADAHOP_ACT_GELU_TANH)
    return invalid("act_backward_mx8: bad activation");
  if (a->gated != 0 && a->gated != 1) return invalid("act_backward_mx8: gated must be 0 or 1");
  if (a->N % 32 != 0) return invalid("act_backward_mx8: N is not a multiple of 32");
  if (!valid_dtype(a->dout_dtype)) return invalid("act_backward_mx8: bad dtype");
  const int64_t n = a->gated ? a->N / 2 : a->N;
  if (a->ld_dout < n || a->ld_z_codes < a->N || a->ld_z_scales < a->N / 32 || a->ld_dz < a->N ||
      (a->out != nullptr && a->ld_out < n))
    return invalid("act_backward_mx8: leading dimension too small");
  if (a->m > 0 && (!a->dout || !a->z_codes || !a->z_scales || !a->dz))
    return invalid("act_backward_mx8: null dout, z or dz");
  if (a->dbias != nullptr)
    ADAHOP_TRY(need_workspace(ws, ws_bytes, act_back_bytes(a->m, a->N, a->gated), "act_backward_mx8"));
  const Mx8Matrix z = {a->z_codes, a->ld_z_codes, a->z_scales, a->ld_z_scales};
  return act_backward_mx8_launch(a->dout, a->dout_dtype, a->ld_dout, z, a->act, a->gated, a->m, n, a->dz, a->ld_dz,
                                 a->out, a->ld_out, a->dbias, static_cast<float*>(ws), stream);
}

adahop_status norm_back_mx8(const adahop_rmsnorm_backward_mx8_args* a, void* ws, size_t ws_bytes,
                            hipStream_t stream) {
  if (a == nullptr) return invalid("rmsnorm_backward_mx8: null arguments");
  ADAHOP_TRY(check_norm_sizes(a->rows, a->cols));
  if (!all_zero(a->reserved)) return invalid("rmsnorm_backward_mx8: reserved fields must be 0");
  if (a->cols % 32 != 0) return invalid("rmsnorm_backward_mx8: cols is not a multiple of 32");
  if (!valid_dtype(a->dy_dtype) || !valid_dtype(a->dx_dtype) || !valid_dtype(a->gain_dtype))
    return invalid("rmsnorm_backward_mx8: bad dtype");
  if (a->ld_dy < a->cols || a->ld_h_codes < a->cols || a->ld_h_scales < a->cols / 32 || a->ld_dx < a->cols ||
      (a->dh != nullptr && a->ld_dh < a->cols))
    return invalid("rmsnorm_backward_mx8: leading dimension too small");
  if (a->gain == nullptr) return invalid("rmsnorm_backward_mx8: null gain");
  if (a->rows > 0 && (!a->dy || !a->h_codes || !a->h_scales || !a->rstd || !a->dx))
    return invalid("rmsnorm_backward_mx8: null dy, h, rstd or dx");
  if (a->rows == 0 && a->dgain == nullptr) return ADAHOP_OK;
  if (a->dgain != nullptr)
    ADAHOP_TRY(need_workspace(ws, ws_bytes, norm_back_bytes(a->rows, a->cols), "rmsnorm_backward_mx8"));
  const Mx8Matrix h = {a->h_codes, a->ld_h_codes, a->h_scales, a->ld_h_scales};
  return rmsnorm_backward_mx8_launch(a->dy, a->dy_dtype, a->ld_dy, h, a->gain, a->gain_dtype, a->rstd, a->dh,
                                     a->ld_dh, a->rows, a->cols, a->dx, a->dx_dtype, a->ld_dx, a->dgain,
                                     static_cast<float*>(ws), stream);
}

bool wgrad_mx8_fits(int64_t T, int64_t Din, int64_t Dout) {
  return T < kMaxDim && Din < kMaxDim && Dout < kMaxDim && tiles_fit(Din, Dout);
}
size_t wgrad_mx8_bytes(int64_t T, int64_t Din, int64_t Dout) {
  if (T < 0 || Din < 1 || Dout < 1 || !wgrad_mx8_fits(T, Din, Dout)) return 0;
  return wgrad_mx8_ws_bytes(T, Din, Dout);
}

adahop_status wgrad_mx8(const adahop_gemm_wgrad_mx8_args* a, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (a == nullptr) return invalid("gemm_wgrad_mx8: null arguments");
  if (a->T < 0 || a->Din < 1 || a->Dout < 1) return invalid("gemm_wgrad_mx8: T must be >= 0, Din and Dout >= 1");
  if (!wgrad_mx8_fits(a->T, a->Din, a->Dout))
    return unsupported("gemm_wgrad_mx8: T, Din or Dout of 2^30 or more, or Din * Dout of 2^46 or more");
  if (!all_zero(a->reserved)) return invalid("gemm_wgrad_mx8: reserved fields must be 0");
  if (a->Din % 32 != 0) return invalid("gemm_wgrad_mx8: Din is not a multiple of 32");
  if (!valid_dtype(a->out_dtype)) return invalid("gemm_wgrad_mx8: bad dtype");
  if (a->ld_gy < a->Dout || a->ld_x_codes < a->Din || a->ld_x_scales < a->Din / 32 || a->ld_out < a->Din)
    return invalid("gemm_wgrad_mx8: leading dimension too small");
  if (!a->out || (a->T > 0 && (!a->gy || !a->x_codes || !a->x_scales)))
    return invalid("gemm_wgrad_mx8: null GY, codes, scales or out");
  if (a->Dout % 8 != 0 || a->ld_gy % 8 != 0 || a->ld_x_codes % 16 != 0 || !aligned16(a->gy) || !aligned16(a->x_codes))
    return unsupported("gemm_wgrad_mx8: rows of GY and codes must be 16-byte aligned, Dout a multiple of 8");
  if (2 * a->ld_gy >= kMaxTileRow || a->ld_x_codes >= kMaxTileRow || a->ld_x_scales >= kMaxTileRow)
    return unsupported("gemm_wgrad_mx8: rows 8 MB or more apart");
  ADAHOP_TRY(need_workspace(ws, ws_bytes, wgrad_mx8_bytes(a->T, a->Din, a->Dout), "gemm_wgrad_mx8"));
  return wgrad_mx8_launch(a->gy, a->ld_gy, {a->x_codes, a->ld_x_codes, a->x_scales, a->ld_x_scales}, a->T, a->Din,
                          a->Dout, a->out, a->out_dtype, a->ld_out, static_cast<float*>(ws), stream);
}

// ---- cross entropy ------------------------------------------------------------
constexpr int64_t kMaxBackRows = int64_t{1} << 22;  // 4 chunks of g below 2 GB

// What both calls ask of their common arguments.
template <typename Args>
adahop_status check_xent(const Args& a) {
  if (a.rows < 0 || a.vocab < 1 || a.dim < 1) return invalid("xent: rows must be >= 0, vocab and dim >= 1");
  if (a.rows >= kMaxDim || a.vocab >= kMaxDim) return unsupported("xent: rows or vocab of 2^30 or more");
  if (!tiles_fit(a.rows, a.vocab)) return unsupported("xent: rows * vocab of 2^46 or more");
  if (!all_zero(a.reserved)) return invalid("xent: reserved fields must be 0");
  if (a.target_dtype != ADAHOP_INDEX_I32 && a.target_dtype != ADAHOP_INDEX_I64)
    return invalid("xent: bad target_dtype");
  if (!std::isfinite(a.scale)) return invalid("xent: scale must be finite");
  if (a.ld_h < a.dim || a.ld_w < a.dim) return invalid("xent: ld_h or ld_w below dim");
  if (a.dim % 8 != 0 || a.ld_h % 8 != 0 || a.ld_w % 8 != 0 || !aligned16(a.h) || !aligned16(a.w))
    return unsupported("xent: rows of h and w must be 16-byte aligned, dim a multiple of 8");
  if (2 * a.ld_h >= kMaxTileRow || 2 * a.ld_w >= kMaxTileRow) return unsupported("xent: rows 8 MB or more apart");
  if (a.rows > 0 && (!a.h || !a.w || !a.targets)) return invalid("xent: null h, w or targets");
  return ADAHOP_OK;
}

template <typename Args>
XentArgs xent_args(const Args& a) {
  return {a.rows, a.vocab, a.dim, a.h, a.ld_h, a.w, a.ld_w, a.targets, a.target_dtype == ADAHOP_INDEX_I64, a.scale};
}

size_t xent_bytes(int64_t rows, int64_t vocab) {
  if (rows < 1 || vocab < 1 || rows >= kMaxDim || vocab >= kMaxDim || !tiles_fit(rows, vocab)) return 0;
  return xent_ws_bytes(rows, vocab);
}

adahop_status xent(const adahop_xent_args* a, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (a == nullptr) return invalid("xent: null arguments");
  ADAHOP_TRY(check_xent(*a));
  if (a->rows == 0) return ADAHOP_OK;
  if (!a->loss || !a->lse) return invalid("xent: null loss or lse");
  ADAHOP_TRY(need_workspace(ws, ws_bytes, xent_bytes(a->rows, a->vocab), "xent"));
  return xent_launch(xent_args(*a), a->loss, a->lse, ws, stream);
}

adahop_status check_xent_back(const adahop_xent_backward_args& a) {
  ADAHOP_TRY(check_xent(a));
  if (a.rows > 0 && !a.dh && !a.dw) return invalid("xent_backward: neither dh nor dw");
  if (a.rows >= kMaxBackRows) return unsupported("xent_backward: rows of 2^22 or more");
  if ((a.dh && (a.ld_dh < a.dim || !valid_dtype(a.dh_dtype))) ||
      (a.dw && (a.ld_dw < a.dim || !valid_dtype(a.dw_dtype))))
    return invalid("xent_backward: leading dimension of dh or dw below dim, or a bad dtype");
  if (a.piece < 0) return invalid("xent_backward: piece must be >= 0");
  if (a.g != ADAHOP_XENT_G_SPLIT && a.g != ADAHOP_XENT_G_BF16) return invalid("xent_backward: bad g");
  if (a.rows > 0 && (!a.lse || !a.dloss)) return invalid("xent_backward: null lse or dloss");
  return ADAHOP_OK;
}

int terms_of(const adahop_xent_backward_args& a) { return a.g == ADAHOP_XENT_G_SPLIT ? 2 : 1; }

size_t xent_back_bytes(const adahop_xent_backward_args& a) {
  return xent_backward_ws_bytes(a.rows, a.vocab, a.dim, a.piece, terms_of(a), a.dh != nullptr, a.dw != nullptr);
}

adahop_status xent_back(const adahop_xent_backward_args* a, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (a == nullptr) return invalid("xent_backward: null arguments");
  ADAHOP_TRY(check_xent_back(*a));
  ADAHOP_TRY(need_workspace(ws, ws_bytes, xent_back_bytes(*a), "xent_backward"));
  const XentGrad g = {a->lse, a->dloss, a->dlse, a->dh, a->ld_dh, a->dh_dtype, a->dw, a->ld_dw, a->dw_dtype,
                      terms_of(*a)};
  return xent_backward_launch(xent_args(*a), g, a->piece, ws, stream);
}

}  // namespace

int64_t compute_units() {
  static std::atomic<int> known[64];
  int dev = 0, v = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) {
    (void)hipGetLastError();
    return 256;
  }
  if ((v = known[dev].load(std::memory_order_relaxed)) > 0) return v;
  if (hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || v < 1) {
    (void)hipGetLastError();
    v = 256;
  }
  known[dev].store(v, std::memory_order_relaxed);
  return v;
}

}  // namespace adahop

using namespace adahop;

extern "C" {

adahop_status adahop_mx8_quant(const void* src, adahop_out_dtype dtype, int64_t rows, int64_t cols,
                               int64_t ld, uint8_t* codes, int64_t ld_codes, uint8_t* scales,
                               int64_t ld_scales, void* stream) {
  return entry([&]() -> adahop_status {
    ADAHOP_TRY(check_mx8(rows, cols, ld, ld_codes, ld_scales, dtype));
    if (rows > 0 && (!src || !codes || !scales)) return invalid("mx8_quant: null pointer");
    return mx8_quant_launch(src, dtype, rows, cols, ld, codes, ld_codes, scales, ld_scales,
                            static_cast<hipStream_t>(stream));
  });
}

adahop_status adahop_mx8_dequant(const uint8_t* codes, int64_t ld_codes, const uint8_t* scales,
                                 int64_t ld_scales, int64_t rows, int64_t cols, void* dst,
                                 adahop_out_dtype dtype, int64_t ld, void* stream) {
  return entry([&]() -> adahop_status {
    ADAHOP_TRY(check_mx8(rows, cols, ld, ld_codes, ld_scales, dtype));
    if (rows > 0 && (!dst || !codes || !scales)) return invalid("mx8_dequant: null pointer");
    return mx8_dequant_launch(codes, ld_codes, scales, ld_scales, rows, cols, dst, dtype, ld,
                              static_cast<hipStream_t>(stream));
  });
}

adahop_status adahop_rmsnorm(const adahop_rmsnorm_args* args, void* stream) {
  return entry([&] { return norm(args, static_cast<hipStream_t>(stream)); });
}

size_t adahop_rmsnorm_backward_workspace_size(int64_t rows, int64_t cols) {
  return norm_back_bytes(rows, cols);
}

adahop_status adahop_rmsnorm_backward(const adahop_rmsnorm_backward_args* args, void* ws,
                                      size_t ws_bytes, void* stream) {
  return entry([&] { return norm_back(args, ws, ws_bytes, static_cast<hipStream_t>(stream)); });
}

size_t adahop_linear_mx_workspace_size(int64_t m, int64_t N, int64_t K, adahop_mx_format b_format,
                                       int32_t gated) {
  if (!valid_product(m, N, K, gated) || (gated && N % 2 != 0)) return 0;
  // Of the two types of output, the one that needs more.
  const int64_t n = gated ? N / 2 : N;
  const size_t bf16 = linear_mx_scratch_bytes(m, n, K, b_format == ADAHOP_MX_E2M1, gated, false);
  const size_t mx8 = linear_mx_scratch_bytes(m, n, K, b_format == ADAHOP_MX_E2M1, gated, true);
  return bf16 > mx8 ? bf16 : mx8;
}

size_t adahop_linear_mx_args_workspace_size(const adahop_linear_args* args) {
  if (args == nullptr || !valid_product(args->m, args->N, args->K, args->gated)) return 0;
  if (args->gated && args->N % 2 != 0) return 0;
  return linear_bytes(*args);
}

adahop_status adahop_linear_mx(const adahop_linear_args* args, void* ws, size_t ws_bytes,
                               void* stream) {
  return entry([&] { return linear(args, ws, ws_bytes, static_cast<hipStream_t>(stream)); });
}

size_t adahop_act_backward_workspace_size(int64_t m, int64_t N, int32_t gated) {
  return act_back_bytes(m, N, gated);
}

adahop_status adahop_act_backward(const void* dout, adahop_out_dtype dout_dtype, int64_t ld_dout,
                                  const uint16_t* z, int64_t ld_z, int64_t m, int64_t N, adahop_act act,
                                  int32_t gated, uint16_t* dz, int64_t ld_dz, float* dbias, void* ws,
                                  size_t ws_bytes, void* stream) {
  return entry([&]() -> adahop_status {
    if (m < 0 || N < 1) return invalid("act_backward: m must be >= 0 and N >= 1");
    if (m >= kMaxDim || N >= kMaxDim) return unsupported("act_backward: m or N of 2^30 or more");
    if (act < ADAHOP_ACT_NONE || act > ADAHOP_ACT_GELU_TANH) return invalid("act_backward: bad activation");
    if (gated != 0 && gated != 1) return invalid("act_backward: gated must be 0 or 1");
    if (gated && N % 2 != 0) return invalid("act_backward: a gated layer needs an even N");
    if (!valid_dtype(dout_dtype)) return invalid("act_backward: bad dtype");
    const int64_t n = gated ? N / 2 : N;
    if (ld_dout < n || ld_z < N || ld_dz < N) return invalid("act_backward: leading dimension too small");
    if (m > 0 && (!dout || !z || !dz)) return invalid("act_backward: null dout, z or dz");
    if (dbias != nullptr)
      ADAHOP_TRY(need_workspace(ws, ws_bytes, act_back_bytes(m, N, gated), "act_backward"));
    return act_backward_launch(dout, dout_dtype, z, act, gated, m, n, ld_dout, ld_z, dz, ld_dz, dbias,
                               static_cast<float*>(ws), static_cast<hipStream_t>(stream));
  });
}

adahop_status adahop_act_backward_mx8(const adahop_act_backward_mx8_args* args, void* ws, size_t ws_bytes,
                                      void* stream) {
  return entry([&] { return act_back_mx8(args, ws, ws_bytes, static_cast<hipStream_t>(stream)); });
}

adahop_status adahop_rmsnorm_backward_mx8(const adahop_rmsnorm_backward_mx8_args* args, void* ws, size_t ws_bytes,
                                          void* stream) {
  return entry([&] { return norm_back_mx8(args, ws, ws_bytes, static_cast<hipStream_t>(stream)); });
}

size_t adahop_gemm_wgrad_mx8_workspace_size(int64_t T, int64_t Din, int64_t Dout) {
  return wgrad_mx8_bytes(T, Din, Dout);
}

adahop_status adahop_gemm_wgrad_mx8(const adahop_gemm_wgrad_mx8_args* args, void* ws, size_t ws_bytes,
                                    void* stream) {
  return entry([&] { return wgrad_mx8(args, ws, ws_bytes, static_cast<hipStream_t>(stream)); });
}

size_t adahop_xent_workspace_size(int64_t rows, int64_t vocab) { return xent_bytes(rows, vocab); }

adahop_status adahop_xent(const adahop_xent_args* args, void* ws, size_t ws_bytes, void* stream) {
  return entry([&] { return xent(args, ws, ws_bytes, static_cast<hipStream_t>(stream)); });
}

size_t adahop_xent_backward_args_workspace_size(const adahop_xent_backward_args* args) {
  size_t bytes = 0;
  const adahop_status st = entry([&]() -> adahop_status {
    if (args == nullptr) return ADAHOP_ERR_INVALID;
    ADAHOP_TRY(check_xent_back(*args));
    bytes = xent_back_bytes(*args);
    return ADAHOP_OK;
  });
  set_error("");
  return st == ADAHOP_OK ? bytes : 0;
}

adahop_status adahop_xent_backward(const adahop_xent_backward_args* args, void* ws, size_t ws_bytes,
                                   void* stream) {
  return entry([&] { return xent_back(args, ws, ws_bytes, static_cast<hipStream_t>(stream)); });
}

}  // extern "C"
