// Linear layer on microscaled operands with its epilogue (gfx950):
//   z = A B^T + bias;  out = act(z) [gated: act(z_gate) * z_up] + residual,
// A MXFP8 [m][K], B MXFP8 or MXFP4 [N][K] (N = n, or 2 n gate and up rows),
// out bf16 or MXFP8, z optionally kept in bf16 for the backward pass.
//
// Matrix cores: v_mfma_scale_f32_16x16x128_f8f6f4, E4M3 by E4M3 or by E2M1,
// one E8M0 byte per lane and 32-element block. Lane l supplies row l % 16 and,
// of the instruction's 128 elements (g = l / 16): E2M1, 32 g .. 32 g + 31; E4M3,
// 16 g .. +15 in its first 16 bytes and 64 + 16 g .. +15 in the others. Its scale
// byte is that of elements 32 g .. 32 g + 31 for both. Checked on the device
// against exact products.
// Accuracy: within each group of 8 products of E4M3 codes the instruction
// truncates what lies under 2^-13 of the largest's power of two, then adds the
// groups in fp32. Measured against exact products: 1.5e-5 of the result (root
// mean square), 5e-5 where 1 % of A's columns are 30 times the rest, at any K.
// bf16 products of the same values are exact up to the fp32 sums, at half the
// rate; an output in bf16 or E4M3 is off by 1.7e-3 or 2.6e-2 by its own
// rounding, so large products take the faster one unless the caller asks for
// exact ones, and no fp32 output is offered. exact_products has the rule.
// The sums over K, the bias, the activation and the residual are in fp32;
// one rounding to the output.
#include "adahop_internal.h"
#include "linear_epilogue.h"

namespace adahop {
namespace {

using namespace mx8;

typedef int v8i __attribute__((ext_vector_type(8)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

// ---- few rows ---------------------------------------------------------------
// A workgroup computes 16 MT rows by 16 NB columns of the output (gated: 16 NB
// gate and as many up rows of B). Its WV waves each take every WV-th run of
// 128 T elements along K straight from memory into registers, the next run's
// loads issued before a run's products; their sums meet in LDS, added in wave
// order. B is read once, by the workgroup that owns its rows: bound by HBM,
// and by what a compute unit loads of A and B (about 28 GB/s): 1 x 4096 x
// 14336, E2M1 weights 10.6 us (2.9 TB/s; 9.4 from the last-level cache), E4M3
// 15.7 us (3.9 TB/s).
template <bool FP4, int MT, int NF, int T>
struct Run {
  v4i a[MT][T][2];
  v4i b[NF][T][FP4 ? 1 : 2];
  uint32_t sa[MT][T], sb[NF][T];
};

constexpr int kBufferFlags = 0x00020000;   // raw buffer descriptor word 3
constexpr int kPastEnd = 0x7FFFFFF0;       // an offset past the end of every buffer here

// Exact: the products on bf16 matrix cores, in which both formats' scaled
// values are exact (near the ends of E8M0's range without their scales), instead
// of the scaled ones, so that an MXFP8 output, where one code rounded the other
// way shows, is that of exact sums. A lane's 32 elements of 128 are one block,
// 32 g .. + 31, of both operands. (1 x 2048 x 4096, E2M1: 6.8 us, scaled 6.0, in
// bf16 5.1; 1 x 14336 x 4096: 11.8, 11.1 and 10.8; 1.6 % of it, on average, looks
// for far scales.)
template <bool FP4, bool Gated, bool Exact, int MT, int NB, int WV, int T>
__global__ void __launch_bounds__(64 * WV, 1) linear_few_kernel(LinearArgs a) {
#ifdef __HIP_DEVICE_COMPILE__                        // the host pass needs the launch stub alone
  constexpr int NF = Gated ? 2 * NB : NB;   // 16-row blocks of B
  constexpr int Cols = 16 * NF, Pitch = Cols + 4, KR = 128 * T;
  // Elements from one lane group's piece of a row to the next, and from a
  // lane's first piece of 16 to its second.
  constexpr int Lane = Exact ? 32 : 16, Half = Exact ? 16 : 64;
  __shared__ float red[WV][MT * 16][Pitch];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * NB), m0 = (int64_t)blockIdx.y * (16 * MT);
  const int K = (int)a.K, Kb = FP4 ? K / 2 : K;
  // A's rows may lie far apart: a pointer each; rows past the end repeat the
  // last one (what they give is not stored). B's 16 NB rows of a part are a
  // buffer, past whose end loads return 0.
  const uint8_t* ac[MT];
  const uint8_t* as[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    int64_t r = m0 + 16 * i + r16;
    r = r < a.m ? r : a.m - 1;
    ac[i] = a.a_codes + r * a.lda + Lane * g;
    as[i] = a.a_scales + r * a.ldas;
  }
  const int rows_b = (int)(a.n - n0 < 16 * NB ? a.n - n0 : 16 * NB);
  auto part = [&](const uint8_t* p, int64_t ld, int bytes, int up) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p + (n0 + up * a.n) * ld), 0,
                                             (int)((rows_b - 1) * ld) + bytes, kBufferFlags);
  };
  const __amdgpu_buffer_rsrc_t bc0 = part(a.b_codes, a.ldb, Kb, 0), bs0 = part(a.b_scales, a.ldbs, K / 32, 0);
  const __amdgpu_buffer_rsrc_t bc1 = part(a.b_codes, a.ldb, Kb, Gated), bs1 = part(a.b_scales, a.ldbs, K / 32, Gated);
  int oc[NB], os[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    oc[j] = (16 * j + r16) * (int)a.ldb + (FP4 ? 16 : Lane) * g;
    os[j] = (16 * j + r16) * (int)a.ldbs;
  }
  v4f acc[MT][NF];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NF; ++j) acc[i][j] = v4f{0, 0, 0, 0};

  using R = Run<FP4, MT, NF, T>;
  auto load = [&](R& r, int k0) {
    const v4i zero = {0, 0, 0, 0};
    const bool full = k0 + KR <= K;
#pragma unroll
    for (int j = 0; j < NF; ++j)
#pragma unroll
      for (int t = 0; t < T; ++t)
#pragma unroll
        for (int h = 0; h < (FP4 ? 1 : 2); ++h) {
          // What lies past the end of K is 0 * 2^0, for both operands.
          const int k = k0 + 128 * t + (FP4 ? 32 * g : Half * h + Lane * g);
          const int off = full || k < K ? oc[j % NB] : kPastEnd;
          const int at = FP4 ? (k0 + 128 * t) / 2 : k0 + 128 * t + Half * h;
          r.b[j][t][h] = __builtin_bit_cast(
              v4i, __builtin_amdgcn_raw_buffer_load_b128(j < NB ? bc0 : bc1, off + (full ? at : k < K ? at : 0), 0, 0));
        }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int t = 0; t < T; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int at = k0 + 128 * t + Half * h;
          r.a[i][t][h] = full || at + Lane * g < K ? *reinterpret_cast<const v4i*>(ac[i] + at) : zero;
        }
    if (full) {
#pragma unroll
      for (int j = 0; j < NF; ++j) {
        uint32_t w[T];
        const __amdgpu_buffer_rsrc_t b = j < NB ? bs0 : bs1;
        if constexpr (T == 4) {
          const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(b, os[j % NB] + k0 / 32, 0, 0);
          __builtin_memcpy(w, &v, 16);
        } else if constexpr (T == 2) {
          const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(b, os[j % NB] + k0 / 32, 0, 0);
          __builtin_memcpy(w, &v, 8);
        } else {
          w[0] = __builtin_amdgcn_raw_buffer_load_b32(b, os[j % NB] + k0 / 32, 0, 0);
        }
#pragma unroll
        for (int t = 0; t < T; ++t) r.sb[j][t] = w[t];
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) __builtin_memcpy(r.sa[i], as[i] + k0 / 32, 4 * T);
    } else {
#pragma unroll
      for (int t = 0; t < T; ++t) {
        const int k = k0 + 128 * t + 32 * g;
#pragma unroll
        for (int j = 0; j < NF; ++j)
          r.sb[j][t] = ((uint32_t)__builtin_amdgcn_raw_buffer_load_b8(j < NB ? bs0 : bs1,
                                                                      k < K ? os[j % NB] + k / 32 : kPastEnd, 0, 0) |
                        (k < K ? 0u : 127u))
                       << (8 * g);
#pragma unroll
        for (int i = 0; i < MT; ++i) r.sa[i][t] = (k < K ? (uint32_t)as[i][k / 32] : 127u) << (8 * g);
      }
    }
  };
  // A lane's 32 elements as bf16, for four instructions.
  struct Eight {
    v8bf v[4];
  };
  auto widen8 = [](const v4i& lo, const v4i& hi, uint32_t byte) {
    const float s = mx8_scale(byte);
    Eight e;
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const int x = q < 2 ? lo[2 * q + w] : hi[2 * (q - 2) + w];
        const auto a0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, s, false);
        const auto a1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, s, true);
        e.v[q][4 * w] = a0[0];
        e.v[q][4 * w + 1] = a0[1];
        e.v[q][4 * w + 2] = a1[0];
        e.v[q][4 * w + 3] = a1[1];
      }
    return e;
  };
  auto widen4 = [](const v4i& c, uint32_t byte) {
    const float s = mx8_scale(byte);
    Eight e;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t x = (uint32_t)c[q];
      const auto a0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, s, 0);
      const auto a1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, s, 1);
      const auto a2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, s, 2);
      const auto a3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, s, 3);
      e.v[q] = v8bf{a0[0], a0[1], a1[0], a1[1], a2[0], a2[1], a3[0], a3[1]};
    }
    return e;
  };
  // Scales for which bf16 holds every value of a block: a code's last bit is
  // 2^-9 (E2M1: 2^-1), bf16's least normal number 2^-126, and 448 * 2^119 (6 *
  // 2^125) the largest below 2^128. Byte 255 makes NaNs, and in a block of zeros,
  // past B's rows too, any scale will do.
  auto low = [](bool fp4) { return fp4 ? 2u : 10u; };
  auto high = [](bool fp4) { return fp4 ? 252u : 246u; };
  auto outside = [&](uint32_t byte, bool fp4) { return byte != 255u && (byte < low(fp4) || byte > high(fp4)); };
  auto nonzero = [](const v4i& c, bool fp4) {
    return ((c[0] | c[1] | c[2] | c[3]) & (fp4 ? 0x77777777 : 0x7F7F7F7F)) != 0;
  };
  auto byte_of = [&](uint32_t word) { return (word >> (8 * g)) & 255u; };
  // Whether a lane of the wave has such a block in a run.
  auto far = [&](const R& r) {
    uint32_t low_a = 255, high_a = 0, low_b = 255, high_b = 0;
#pragma unroll
    for (int t = 0; t < T; ++t) {
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const uint32_t v = byte_of(r.sa[i][t]);
        low_a = v < low_a ? v : low_a;
        high_a = v > high_a ? v : high_a;
      }
#pragma unroll
      for (int j = 0; j < NF; ++j) {
        const uint32_t v = byte_of(r.sb[j][t]);
        low_b = v < low_b ? v : low_b;
        high_b = v > high_b ? v : high_b;
      }
    }
    if (!__any(low_a < low(false) || high_a > high(false) || low_b < low(FP4) || high_b > high(FP4))) return false;
    bool any = false;
#pragma unroll
    for (int t = 0; t < T; ++t) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
        any |= outside(byte_of(r.sa[i][t]), false) &&
               (nonzero(r.a[i][t][0], false) || nonzero(r.a[i][t][1], false));
#pragma unroll
      for (int j = 0; j < NF; ++j)
        any |= outside(byte_of(r.sb[j][t]), FP4) &&
               (nonzero(r.b[j][t][0], FP4) || nonzero(r.b[j][t][FP4 ? 0 : 1], FP4));
    }
    return __any(any) != 0;
  };
  // Such a run is left out, and taken in a second pass over K (in the first, its
  // code costs the others registers: up to 26 spilled) block by block: the
  // codes' products, without scales, and the sum times both scales, whose product
  // may be ordinary where each is not.
  auto far_products = [&](const R& r) {
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll 1
      for (int block = 0; block < 4; ++block) {
        const v4i zero = {0, 0, 0, 0};
        const bool mine = g == block;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const Eight wa = widen8(mine ? r.a[i][t][0] : zero, mine ? r.a[i][t][1] : zero, 127u);
          const int row = __shfl((int)byte_of(r.sa[i][t]), 16 * block + r16);
#pragma unroll
          for (int j = 0; j < NF; ++j) {
            const v4i lo = mine ? r.b[j][t][0] : zero, hi = mine ? r.b[j][t][FP4 ? 0 : 1] : zero;
            const Eight wb = FP4 ? widen4(lo, 127u) : widen8(lo, hi, 127u);
            v4f sum = {0, 0, 0, 0};
#pragma unroll
            for (int q = 0; q < 4; ++q)
              sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb.v[q], wa.v[q], sum, 0, 0, 0);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int col = __shfl((int)byte_of(r.sb[j][t]), 16 * block + 4 * g + e);
              const float v = __builtin_amdgcn_ldexpf(sum[e], row + col - 254);
              acc[i][j][e] += row == 255 || col == 255 ? __builtin_nanf("") : v;
            }
          }
        }
      }
  };
  [[maybe_unused]] bool again = false;
  auto products = [&](const R& r) {
    if constexpr (Exact) {
      if (far(r)) {
        again = true;
        return;
      }
    }
#pragma unroll
    for (int t = 0; t < T; ++t) {
      if constexpr (Exact) {
        Eight wa[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i)
          wa[i] = widen8(r.a[i][t][0], r.a[i][t][1], byte_of(r.sa[i][t]));
#pragma unroll
        for (int j = 0; j < NF; ++j) {
          const uint32_t byte = byte_of(r.sb[j][t]);
          const Eight wb = FP4 ? widen4(r.b[j][t][0], byte) : widen8(r.b[j][t][0], r.b[j][t][FP4 ? 0 : 1], byte);
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q)
              acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb.v[q], wa[i].v[q], acc[i][j], 0, 0, 0);
        }
      } else {
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const v4i al = r.a[i][t][0], ah = r.a[i][t][1];
          const v8i fa = {al[0], al[1], al[2], al[3], ah[0], ah[1], ah[2], ah[3]};
#pragma unroll
          for (int j = 0; j < NF; ++j) {
            const v4i lo = r.b[j][t][0], hi = FP4 ? v4i{0, 0, 0, 0} : r.b[j][t][FP4 ? 0 : 1];
            // B first: lane l then holds row l % 16 and columns 4 (l / 16) .. +3.
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]}, fa, acc[i][j], FP4 ? 4 : 0, 0, 0,
                (int)(r.sb[j][t] >> (8 * g)), 0, (int)(r.sa[i][t] >> (8 * g)));
          }
        }
      }
    }
  };
  const int runs = (K + KR - 1) / KR;
  R x, y;
  int i = wave;
  if (i < runs) load(x, KR * i);
  while (i < runs) {
    if (i + WV < runs) load(y, KR * (i + WV));
    products(x);
    i += WV;
    if (i >= runs) break;
    if (i + WV < runs) load(x, KR * (i + WV));
    products(y);
    i += WV;
  }
  if constexpr (Exact) {
    if (again) {
#pragma unroll 1
      for (i = wave; i < runs; i += WV) {
        load(x, KR * i);
        if (far(x)) far_products(x);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NF; ++j)
      *reinterpret_cast<v4f*>(&red[wave][16 * i + r16][16 * j + 4 * g]) = acc[i][j];
  __syncthreads();
  // Every thread adds the waves' sums of some elements, into the first
  // wave's place; then 2 NB lanes a row finish it, 8 columns each.
  for (int e = threadIdx.x; e < MT * 16 * Cols; e += 64 * WV) {
    const int row = e / Cols, col = e % Cols;
    float s = red[0][row][col];
#pragma unroll
    for (int w = 1; w < WV; ++w) s += red[w][row][col];
    red[0][row][col] = s;
  }
  __syncthreads();
  for (int u = threadIdx.x; u < MT * 16 * 2 * NB; u += 64 * WV) {
    const int row = u / (2 * NB), col = 8 * (u % (2 * NB));
    float z[8], up[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      z[i] = red[0][row][col + i];
      up[i] = Gated ? red[0][row][16 * NB + col + i] : 0.0f;
    }
    if (m0 + row < a.m && n0 + col < a.n) epilogue8<Gated>(a, m0 + row, n0 + col, z, up);
  }
#endif
}

template <bool FP4, bool Gated, bool Exact, int MT, int NB, int WV, int T>
void few_start(const LinearArgs& a, hipStream_t stream) {
  linear_few_kernel<FP4, Gated, Exact, MT, NB, WV, T>
      <<<dim3((unsigned)((a.n + 16 * NB - 1) / (16 * NB)), (unsigned)((a.m + 16 * MT - 1) / (16 * MT))),
         dim3(64 * WV), 0, stream>>>(a);
}

// 32 columns a workgroup: 8 waves by few_narrow too (1 x 2048 x 4096, E2M1,
// exact: 6.6 us, with 4 waves 7.7; 1 x 14336 x 4096: 13.3, with 4 waves 11.7);
// gated, whose registers do not last for 8, 4.
template <bool FP4, bool Gated, bool Exact>
adahop_status few_wide(const LinearArgs& a, hipStream_t stream) {
  if constexpr (!Gated) {
    if (few_narrow(a.n)) {
      if (a.m <= 16) few_start<FP4, Gated, Exact, 1, 2, 8, FP4 ? 4 : 2>(a, stream);
      else few_start<FP4, Gated, Exact, 2, 2, 8, 2>(a, stream);
      return check_launch("linear_mx");
    }
  }
  if (a.m <= 16) few_start<FP4, Gated, Exact, 1, 2, 4, 2>(a, stream);
  else few_start<FP4, Gated, Exact, 2, 2, 4, 2>(a, stream);
  return check_launch("linear_mx");
}

template <bool FP4, bool Gated>
adahop_status few_dispatch(const LinearArgs& a, bool exact, hipStream_t stream) {
  if (exact) return few_wide<FP4, Gated, true>(a, stream);
  if (a.out_scales != nullptr || !few_narrow(a.n)) return few_wide<FP4, Gated, false>(a, stream);
  if (a.m <= 16) few_start<FP4, Gated, false, 1, 1, 8, 2>(a, stream);
  else few_start<FP4, Gated, false, 2, 1, 8, 2>(a, stream);
  return check_launch("linear_mx");
}

// Rows r0 .. r0 + rows - 1 and output columns c0 .. c0 + cols - 1 (a multiple
// of 32, and all of them for a gated layer).
LinearArgs part_of(const LinearArgs& a, int64_t r0, int64_t rows, int64_t c0, int64_t cols) {
  LinearArgs p = a;
  p.m = rows;
  p.n = cols;
  p.a_codes += r0 * a.lda;
  p.a_scales += r0 * a.ldas;
  p.b_codes += c0 * a.ldb;
  p.b_scales += c0 * a.ldbs;
  if (a.bias) p.bias = static_cast<const char*>(a.bias) + c0 * (a.bias_f32 ? 4 : 2);
  if (a.residual) p.residual += r0 * a.ldr + c0;
  p.out = static_cast<char*>(a.out) + (r0 * a.ldo + c0) * (a.out_scales ? 1 : 2);
  if (a.out_scales) p.out_scales += r0 * a.ldos + c0 / 32;
  if (a.z) p.z += r0 * a.ldz + c0;
  return p;
}

// In launches whose grid fits: its second dimension (blocks of 16 or 32 rows)
// and, in its first, the threads.
adahop_status few_launch(const LinearArgs& a, int b_fp4, int gated, bool exact, hipStream_t stream) {
  constexpr int64_t kRows = int64_t{1} << 20;
  const int64_t cols = gated ? a.n : kFewLaunchCols;
  for (int64_t r = 0; r < a.m; r += kRows)
    for (int64_t c = 0; c < a.n; c += cols) {
      const LinearArgs p = part_of(a, r, a.m - r < kRows ? a.m - r : kRows, c, a.n - c < cols ? a.n - c : cols);
      adahop_status st;
      if (b_fp4) st = gated ? few_dispatch<true, true>(p, exact, stream) : few_dispatch<true, false>(p, exact, stream);
      else st = gated ? few_dispatch<false, true>(p, exact, stream) : few_dispatch<false, false>(p, exact, stream);
      if (st != ADAHOP_OK) return st;
    }
  return ADAHOP_OK;
}

}  // namespace

size_t linear_mx_scratch_bytes(int64_t m, int64_t n, int64_t K, int b_fp4, int gated, bool mx8_out) {
  const int64_t cus = compute_units();
  const TilePlan p = linear_tile_plan(m, n, K, b_fp4, gated, cus);
  return take_few(m, p, n, K, b_fp4, gated, mx8_out, cus) ? 0 : p.scale_bytes + p.part_bytes;
}

adahop_status linear_mx_launch(const LinearArgs& a, int b_fp4, int gated, bool exact, void* scratch,
                               hipStream_t stream) {
  if (a.m == 0) return ADAHOP_OK;
  if (exact) return few_launch(a, b_fp4, gated, true, stream);
  const int64_t cus = compute_units();
  const TilePlan plan = linear_tile_plan(a.m, a.n, a.K, b_fp4, gated, cus);
  if (take_few(a.m, plan, a.n, a.K, b_fp4, gated, a.out_scales != nullptr, cus))
    return few_launch(a, b_fp4, gated, false, stream);
  if (linear_tiles_reach(a.m, a.lda) && linear_tiles_reach(a.n, a.ldb))
    return linear_tiles_launch(a, b_fp4, gated, plan, scratch, stream);
  // Operands of 2 GB and more: in pieces that the tile kernel's offsets
  // reach. Rows 4 MB apart and gated weights of 2 GB a part go by the
  // streaming kernel.
  auto most = [](int64_t rows, int64_t ld) {
    if (linear_tiles_reach(rows, ld)) return rows;
    const int64_t c = ((int64_t{1} << 31) / ld - 1024) / 512 * 512;
    return c > 0 && linear_tiles_reach(c, ld) ? c : int64_t{0};
  };
  const int64_t rows = most(a.m, a.lda), cols = most(a.n, a.ldb);
  if (rows == 0 || cols == 0 || (gated && cols < a.n)) return few_launch(a, b_fp4, gated, false, stream);
  for (int64_t r = 0; r < a.m; r += rows)
    for (int64_t c = 0; c < a.n; c += cols) {
      const LinearArgs p = part_of(a, r, a.m - r < rows ? a.m - r : rows, c, a.n - c < cols ? a.n - c : cols);
      TilePlan t = plan;                     // its scratch fits every piece
      t.parts = 1;
      const adahop_status st = linear_tiles_launch(p, b_fp4, gated, t, scratch, stream);
      if (st != ADAHOP_OK) return st;
    }
  return ADAHOP_OK;
}

}  // namespace adahop
