// RMS norm with the residual's addition and an MXFP8 output, its backward
// pass, and the MXFP8 quantizer / dequantizer (gfx950).
//
//   h = x + r (rounded to the stream's type), s = 1 / sqrt(mean(h^2) + eps),
//   y = h * s * gain, stored as MXFP8 and / or bf16.
// All are bound by HBM: every operand is read once and every result written
// once, with a row's values held in registers between the sum of squares and
// the scaling. Sums run in fp32 along fixed trees: results do not change from
// run to run.
#include "adahop_internal.h"
#include "launch_shapes.h"
#include "mx8_common.h"

namespace adahop {
namespace {

using namespace mx8;

struct NormArgs {
  const void* x;
  const void* r;
  const void* gain;
  int gain_f32;
  int64_t rows, cols;
  int64_t ldx, ldr, ldh, ldy, ldc, lds;
  float eps;
  void* h;
  uint16_t* y;
  uint8_t* codes;
  uint8_t* scales;
  float* rstd;
};

// Sum over a workgroup of Waves waves, in every thread (one barrier).
template <int Waves>
__device__ __forceinline__ float group_sum(float v, float* red) {
  v = wave_sum(v);
  if constexpr (Waves > 1) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < Waves; ++w) v += red[w];
  }
  return v;
}

__device__ __forceinline__ void load_gain(const void* gain, int f32, int64_t c, int64_t cols,
                                          float (&g)[8]) {
  if (f32)
    load_group<true>(static_cast<const float*>(gain), c, cols, g);
  else
    load_group<false>(static_cast<const uint16_t*>(gain), c, cols, g);
}

// XF32: x in fp32; Res: 0 none, 1 bf16, 2 fp32 residual stream. A row is
// spread over Waves waves, each thread holding NV groups of 8 columns; with
// Waves == 1 a workgroup takes 4 rows, one a wave, and needs no barrier.
// 32768 x 4096 in bf16 with residual: 155 .. 172 us, 5.5 .. 6.1 TB/s.
template <bool XF32, int Res, int Waves, int NV>
__global__ void __launch_bounds__(Waves == 1 ? 256 : 64 * Waves)
    rmsnorm_kernel(NormArgs a) {
  constexpr bool RF32 = Res == 2;
  using TX = typename Elem<XF32>::type;
  using TR = typename Elem<RF32>::type;
  constexpr int T = Waves == 1 ? 64 : 64 * Waves;
  __shared__ float red[Waves];
  const int64_t row = Waves == 1 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
  if (Waves == 1 && row >= a.rows) return;
  const int t = Waves == 1 ? threadIdx.x & 63 : threadIdx.x;
  const TX* x = static_cast<const TX*>(a.x) + row * a.ldx;
  float v[NV][8];
#pragma unroll
  for (int k = 0; k < NV; ++k) load_group<XF32>(x, 8 * (int64_t)(t + k * T), a.cols, v[k]);
  if constexpr (Res != 0) {
    const TR* r = static_cast<const TR*>(a.r) + row * a.ldr;
    float q[NV][8];
#pragma unroll
    for (int k = 0; k < NV; ++k) load_group<RF32>(r, 8 * (int64_t)(t + k * T), a.cols, q[k]);
    TR* h = static_cast<TR*>(a.h) + row * a.ldh;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      // The norm takes h as the stream holds it (rounded to its type), so
      // that the backward pass, which reads h, differentiates what was run.
#pragma unroll
      for (int i = 0; i < 8; ++i) v[k][i] = Elem<RF32>::rounded(v[k][i] + q[k][i]);
      store_group<RF32>(h, 8 * (int64_t)(t + k * T), a.cols, v[k]);
    }
  }
  float s = 0.0f;
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) s = __builtin_fmaf(v[k][i], v[k][i], s);
  s = group_sum<Waves>(s, red);
  const float rstd = 1.0f / sqrtf(s / (float)a.cols + a.eps);
  if (a.rstd != nullptr && t == 0) a.rstd[row] = rstd;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int64_t c = 8 * (int64_t)(t + k * T);
    float g[8];
    load_gain(a.gain, a.gain_f32, c, a.cols, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[k][i] = v[k][i] * rstd * g[i];
    if (a.y != nullptr) store_group<false>(a.y + row * a.ldy, c, a.cols, v[k]);
    if (a.codes != nullptr && c < a.cols)
      mx8_store_quad(v[k], a.codes + row * a.ldc + c, a.scales + row * a.lds + c / 32);
  }
}

// ---- backward ---------------------------------------------------------------
struct NormBackArgs {
  const void* dy;
  const void* h;
  const void* gain;
  int gain_f32;
  const float* rstd;
  const void* dh;
  int64_t rows, cols;
  int64_t lddy, ldh, lddh, lddx;
  void* dx;
  float* partial;     // [workgroups][cols], or null without dgain
};

// With n = h * s and u = gain * dy:  dx = dh + s * (u - n * mean(u * n)),
// and a workgroup's part of dgain = sum over its rows of dy * n, which stays
// in registers over all rows that the workgroup takes (every gridDim.x-th
// group of rows) and goes out once. Bound by HBM: 8 columns a thread, so that
// 16 waves a compute unit fit, each with its next row's loads in flight
// (16384 x 2048 in bf16 with dh: 45 .. 48 us, 5.6 .. 5.9 TB/s; a wave a row
// without loads ahead 76).
// Once: every row starts at a cache line.
template <bool DyF32, bool HF32, bool Once, int Waves, int NV>
__global__ void __launch_bounds__(Waves == 1 ? 256 : 64 * Waves)
    rmsnorm_backward_kernel(NormBackArgs a) {
  using TD = typename Elem<DyF32>::type;
  using TH = typename Elem<HF32>::type;
  constexpr int T = 64 * Waves;
  constexpr int RowsPer = Waves == 1 ? 4 : 1;
  __shared__ float red[2][Waves];
  __shared__ float part[Waves == 1 ? 3 * 64 * 8 : 1];
  const int wave = threadIdx.x >> 6;
  const int t = Waves == 1 ? threadIdx.x & 63 : threadIdx.x;
  struct Row {
    Raw8<DyF32> dy[NV];
    Raw8<HF32> h[NV], dh[NV];
    float s;
  };
  const int64_t step = (int64_t)gridDim.x * RowsPer;
  auto load = [&](Row& r, int64_t row) {
    const TD* dy = static_cast<const TD*>(a.dy) + row * a.lddy;
    const TH* h = static_cast<const TH*>(a.h) + row * a.ldh;
    r.s = a.rstd[row];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int64_t c = 8 * (int64_t)(t + k * T);
      r.dy[k].template load<Once>(dy, c, a.cols);
      r.h[k].template load<Once>(h, c, a.cols);
      if (a.dh != nullptr) r.dh[k].template load<Once>(static_cast<const TH*>(a.dh) + row * a.lddh, c, a.cols);
    }
  };
  // More than 8 columns a thread leave no registers for a row ahead, nor for
  // the gain.
  constexpr bool Ahead = NV == 1;
  float acc[NV][8], g[8];
  if constexpr (Ahead) load_gain(a.gain, a.gain_f32, 8 * (int64_t)t, a.cols, g);
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[k][i] = 0.0f;
  int turn = 0;
  int64_t row = (int64_t)blockIdx.x * RowsPer + (Waves == 1 ? wave : 0);
  Row now, next;
  if (Ahead && row < a.rows) load(now, row);
  for (; row < a.rows; row += step, turn ^= 1) {
    if constexpr (Ahead) {
      if (row + step < a.rows) load(next, row + step);
    } else {
      load(now, row);
    }
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float u[8], n[8];
      const int64_t at = 8 * (int64_t)(t + k * T);
      now.dy[k].get(u, at, a.cols);
      now.h[k].get(n, at, a.cols);
      if constexpr (!Ahead) load_gain(a.gain, a.gain_f32, 8 * (int64_t)(t + k * T), a.cols, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        n[i] *= now.s;
        acc[k][i] = __builtin_fmaf(u[i], n[i], acc[k][i]);
        u[i] *= g[i];
        sum = __builtin_fmaf(u[i], n[i], sum);
      }
    }
    // Two sets of partial sums in turn: a wave that is a row ahead writes
    // the other set, and is held at that row's barrier until all have read.
    const float c = group_sum<Waves>(sum, red[turn]) / (float)a.cols;
    TH* dx = static_cast<TH*>(a.dx) + row * a.lddx;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float u[8], n[8], e[8];
      const int64_t at = 8 * (int64_t)(t + k * T);
      now.dy[k].get(u, at, a.cols);
      now.h[k].get(n, at, a.cols);
      if constexpr (!Ahead) load_gain(a.gain, a.gain_f32, 8 * (int64_t)(t + k * T), a.cols, g);
      if (a.dh != nullptr) {
        now.dh[k].get(e, at, a.cols);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] += now.s * (u[i] * g[i] - n[i] * now.s * c);
      store_group<HF32>(dx, 8 * (int64_t)(t + k * T), a.cols, e);
    }
    if constexpr (Ahead) now = next;
  }
  if (a.partial == nullptr) return;
  float* out = a.partial + (int64_t)blockIdx.x * a.cols;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int64_t c = 8 * (int64_t)(t + k * T);
    if constexpr (Waves == 1) {
      // The four waves' parts of the same columns, added in wave order.
      __syncthreads();
      if (wave > 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) part[(wave - 1) * 512 + i * 64 + t] = acc[k][i];
      }
      __syncthreads();
      if (wave == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          acc[k][i] = ((acc[k][i] + part[i * 64 + t]) + part[512 + i * 64 + t]) + part[1024 + i * 64 + t];
      }
    }
    if (Waves > 1 || wave == 0) store_group<true>(out, c, a.cols, acc[k]);
  }
}

// out[c] = sum over p of partial[p][c], rows of partial `ld` apart: a workgroup
// takes 16 columns, its 64 groups of 16 lanes every 64th part; their sums are
// added in pairs, in a fixed tree. (4.9 us for 1024 x 2048, most of it latency.)
__global__ void __launch_bounds__(kReduceBlock) column_reduce_kernel(const float* __restrict__ partial,
                                                                     int parts, int64_t cols, int64_t ld,
                                                                     float* __restrict__ out) {
  __shared__ float red[64][17];
  const int lane = threadIdx.x & 15, group = threadIdx.x >> 4;
  const int64_t c = (int64_t)blockIdx.x * 16 + lane;
  float s = 0.0f;
  if (c < cols) {
#pragma unroll 8
    for (int p = group; p < parts; p += 64) s += partial[(int64_t)p * ld + c];
  }
  red[group][lane] = s;
#pragma unroll
  for (int half = 32; half >= 1; half /= 2) {
    __syncthreads();
    if (group < half) red[group][lane] += red[group + half][lane];
  }
  if (group == 0 && c < cols) out[c] = red[0][lane];
}

// ---- quantizer and dequantizer ----------------------------------------------
struct Mx8Args {
  const void* src;
  int64_t ld;
  int64_t rows, cols;      // cols a multiple of 32
  uint8_t* codes;
  uint8_t* scales;
  int64_t ldc, lds;
  void* dst;               // dequantizer's output
  int64_t ldd;
};

// Group of 8 elements `i` of the matrix: its row and first column.
__device__ __forceinline__ void group_at(int64_t i, int64_t rows, int64_t cols, int64_t* r, int64_t* c) {
  if (rows == 1) {
    *r = 0;
    *c = 8 * i;
  } else if (rows * (cols / 8) < (1LL << 31)) {
    const uint32_t per = (uint32_t)(cols / 8), q = (uint32_t)i / per;
    *r = q;
    *c = 8 * (int64_t)((uint32_t)i - q * per);
  } else {
    *r = i / (cols / 8);
    *c = 8 * (i - *r * (cols / 8));
  }
}

template <bool F32>
__global__ void __launch_bounds__(256) mx8_quant_kernel(Mx8Args a) {
  using TS = typename Elem<F32>::type;
  const int64_t n = a.rows * (a.cols / 8);
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    int64_t r, c;
    group_at(i, a.rows, a.cols, &r, &c);
    float v[8];
    Elem<F32>::load8(static_cast<const TS*>(a.src) + r * a.ld + c, v);
    mx8_store_quad(v, a.codes + r * a.ldc + c, a.scales + r * a.lds + c / 32);
  }
}

template <bool F32>
__global__ void __launch_bounds__(256) mx8_dequant_kernel(Mx8Args a) {
  using TD = typename Elem<F32>::type;
  const int64_t n = a.rows * (a.cols / 8);
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    int64_t r, c;
    group_at(i, a.rows, a.cols, &r, &c);
    u32x2 w;
    __builtin_memcpy(&w, a.codes + r * a.ldc + c, 8);
    const float s = mx8_scale(a.scales[r * a.lds + c / 32]);
    float v[8];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[j], false);
      const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[j], true);
      v[4 * j] = lo[0] * s;
      v[4 * j + 1] = lo[1] * s;
      v[4 * j + 2] = hi[0] * s;
      v[4 * j + 3] = hi[1] * s;
    }
    Elem<F32>::store8(static_cast<TD*>(a.dst) + r * a.ldd + c, v);
  }
}

int flat_grid(int64_t groups) {
  const int64_t wg = (groups + 255) / 256;
  return (int)(wg < 1 ? 1 : wg < 16384 ? wg : 16384);
}

template <bool XF32, int Res>
adahop_status norm_dispatch(const NormArgs& a, hipStream_t stream) {
  const NormShape shape = norm_shape(a.cols);
  const dim3 grid((unsigned)norm_grid(a.rows, shape.waves)), block((unsigned)norm_block(shape.waves));
#define ADAHOP_NORM(WAVES, NV) rmsnorm_kernel<XF32, Res, WAVES, NV><<<grid, block, 0, stream>>>(a)
  if (shape.waves == 1) {
    if (shape.groups == 1) ADAHOP_NORM(1, 1);
    else if (shape.groups == 2) ADAHOP_NORM(1, 2);
    else ADAHOP_NORM(1, 4);
  } else if (shape.waves == 4) {
    if (shape.groups == 2) ADAHOP_NORM(4, 2);
    else ADAHOP_NORM(4, 4);
  } else {
    if (shape.groups == 2) ADAHOP_NORM(16, 2);
    else ADAHOP_NORM(16, 4);
  }
#undef ADAHOP_NORM
  return check_launch("rmsnorm");
}

// Waves that share a row: 8 columns a lane, up to 16 waves.
int norm_back_waves(int64_t cols) {
  int w = 1;
  while (w < 16 && 512 * w < cols) w *= 2;
  return w;
}

template <bool DyF32, bool HF32, bool Once>
adahop_status norm_back_dispatch(const NormBackArgs& a, int grid, hipStream_t stream) {
  const int64_t c = a.cols;
#define ADAHOP_NORM_BACK(WAVES, NV)                                                              \
  rmsnorm_backward_kernel<DyF32, HF32, Once, WAVES, NV>                                                \
      <<<dim3((unsigned)grid), dim3(WAVES == 1 ? 256 : 64 * WAVES), 0, stream>>>(a)
  switch (norm_back_waves(c)) {
    case 1: ADAHOP_NORM_BACK(1, 1); break;
    case 2: ADAHOP_NORM_BACK(2, 1); break;
    case 4: ADAHOP_NORM_BACK(4, 1); break;
    case 8: ADAHOP_NORM_BACK(8, 1); break;
    default:
      if (c <= 8192) ADAHOP_NORM_BACK(16, 1);
      else if (c <= 16384) ADAHOP_NORM_BACK(16, 2);
      else ADAHOP_NORM_BACK(16, 4);
  }
#undef ADAHOP_NORM_BACK
  return check_launch("rmsnorm_backward");
}

}  // namespace

adahop_status rmsnorm_launch(const void* x, int x_f32, const void* r, int r_f32, const void* gain,
                             int gain_f32, int64_t rows, int64_t cols, int64_t ldx, int64_t ldr,
                             float eps, void* h, int64_t ldh, uint16_t* y, int64_t ldy,
                             uint8_t* codes, int64_t ldc, uint8_t* scales, int64_t lds, float* rstd,
                             hipStream_t stream) {
  constexpr int64_t kRows = kNormLaunchRows;
  for (int64_t at = 0; at < rows; at += kRows) {
    auto bytes = [at](const void* p, int64_t ld, int64_t size) {
      return p == nullptr ? nullptr : const_cast<char*>(static_cast<const char*>(p)) + at * ld * size;
    };
    const NormArgs a = {bytes(x, ldx, x_f32 ? 4 : 2), bytes(r, ldr, r_f32 ? 4 : 2), gain, gain_f32,
                        rows - at < kRows ? rows - at : kRows, cols, ldx, ldr, ldh, ldy, ldc, lds, eps,
                        bytes(h, ldh, r_f32 ? 4 : 2), reinterpret_cast<uint16_t*>(bytes(y, ldy, 2)),
                        reinterpret_cast<uint8_t*>(bytes(codes, ldc, 1)),
                        reinterpret_cast<uint8_t*>(bytes(scales, lds, 1)),
                        reinterpret_cast<float*>(bytes(rstd, 1, 4))};
    adahop_status st;
    if (r == nullptr) st = x_f32 ? norm_dispatch<true, 0>(a, stream) : norm_dispatch<false, 0>(a, stream);
    else if (x_f32) st = r_f32 ? norm_dispatch<true, 2>(a, stream) : norm_dispatch<true, 1>(a, stream);
    else st = r_f32 ? norm_dispatch<false, 2>(a, stream) : norm_dispatch<false, 1>(a, stream);
    if (st != ADAHOP_OK) return st;
  }
  return ADAHOP_OK;
}

int rmsnorm_backward_groups(int64_t rows, int64_t cols) {
  // 4096 waves, 16 a compute unit; each workgroup leaves one row of partial
  // sums (8 MB in all up to 8192 columns, 32 MB at 32768).
  const int waves = norm_back_waves(cols);
  const int64_t need = waves == 1 ? (rows + 3) / 4 : rows, most = waves == 1 ? 1024 : 4096 / waves;
  return (int)(need < 1 ? 1 : need < most ? need : most);
}

adahop_status rmsnorm_backward_launch(const void* dy, int dy_f32, const void* h, int h_f32,
                                      const void* gain, int gain_f32, const float* rstd,
                                      const void* dh, int64_t rows, int64_t cols, int64_t lddy,
                                      int64_t ldh, int64_t lddh, int64_t lddx, void* dx,
                                      float* dgain, float* partial, hipStream_t stream) {
  const int grid = rmsnorm_backward_groups(rows, cols);
  const bool once = line_aligned(dy, lddy, dy_f32) && line_aligned(h, ldh, h_f32) &&
                    (dh == nullptr || line_aligned(dh, lddh, h_f32));
  const NormBackArgs a = {dy, h, gain, gain_f32, rstd, dh, rows, cols, lddy, ldh, lddh, lddx, dx,
                          dgain != nullptr ? partial : nullptr};
  adahop_status st;
#define ADAHOP_NORM_TYPES(ONCE)                                                                        \
  (dy_f32 ? (h_f32 ? norm_back_dispatch<true, true, ONCE>(a, grid, stream)                             \
                   : norm_back_dispatch<true, false, ONCE>(a, grid, stream))                           \
          : (h_f32 ? norm_back_dispatch<false, true, ONCE>(a, grid, stream)                            \
                   : norm_back_dispatch<false, false, ONCE>(a, grid, stream)))
  st = once ? ADAHOP_NORM_TYPES(true) : ADAHOP_NORM_TYPES(false);
#undef ADAHOP_NORM_TYPES
  if (st != ADAHOP_OK || dgain == nullptr) return st;
  return column_reduce_launch(partial, grid, cols, dgain, stream);
}

adahop_status column_reduce_launch(const float* partial, int parts, int64_t cols, float* out,
                                   hipStream_t stream) {
  for (int64_t c = 0; c < cols; c += kReduceLaunchCols) {
    const int64_t n = cols - c < kReduceLaunchCols ? cols - c : kReduceLaunchCols;
    column_reduce_kernel<<<dim3((unsigned)reduce_grid(n)), dim3(kReduceBlock), 0, stream>>>(partial + c, parts, n,
                                                                                          cols, out + c);
    const adahop_status st = check_launch("column_reduce");
    if (st != ADAHOP_OK) return st;
  }
  return ADAHOP_OK;
}

adahop_status mx8_quant_launch(const void* src, int f32, int64_t rows, int64_t cols, int64_t ld,
                               uint8_t* codes, int64_t ldc, uint8_t* scales, int64_t lds,
                               hipStream_t stream) {
  if (rows == 0) return ADAHOP_OK;
  if (ld == cols && ldc == cols && lds == cols / 32) { cols *= rows; rows = 1; }
  const Mx8Args a = {src, ld, rows, cols, codes, scales, ldc, lds, nullptr, 0};
  const dim3 grid((unsigned)flat_grid(rows * (cols / 8)));
  if (f32) mx8_quant_kernel<true><<<grid, dim3(256), 0, stream>>>(a);
  else mx8_quant_kernel<false><<<grid, dim3(256), 0, stream>>>(a);
  return check_launch("mx8_quant");
}

adahop_status mx8_dequant_launch(const uint8_t* codes, int64_t ldc, const uint8_t* scales, int64_t lds,
                                 int64_t rows, int64_t cols, void* dst, int f32, int64_t ldd,
                                 hipStream_t stream) {
  if (rows == 0) return ADAHOP_OK;
  if (ldd == cols && ldc == cols && lds == cols / 32) { cols *= rows; rows = 1; }
  const Mx8Args a = {nullptr, 0, rows, cols, const_cast<uint8_t*>(codes), const_cast<uint8_t*>(scales),
                     ldc, lds, dst, ldd};
  const dim3 grid((unsigned)flat_grid(rows * (cols / 8)));
  if (f32) mx8_dequant_kernel<true><<<grid, dim3(256), 0, stream>>>(a);
  else mx8_dequant_kernel<false><<<grid, dim3(256), 0, stream>>>(a);
  return check_launch("mx8_dequant");
}

}  // namespace adahop
