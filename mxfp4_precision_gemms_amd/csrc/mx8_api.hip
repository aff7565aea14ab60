// Host side of the norm, MXFP8 and linear-layer entry points: argument checks
// and launches. Every check runs before the first launch; nothing allocates
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

}  // extern "C"
