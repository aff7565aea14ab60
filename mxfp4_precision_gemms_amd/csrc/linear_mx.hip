// Linear layer on microscaled operands with its epilogue (gfx950):
//   z = A B^T + bias;  out = act(z) [gated: act(z_gate) * z_up] + residual,
// A MXFP8 [m][K], B MXFP8 or MXFP4 [N][K] (N = n, or 2 n gate and up rows),
// out bf16 or MXFP8, z optionally kept in bf16 for the backward pass.
//
// Matrix cores: v_mfma_scale_f32_{16x16x128,32x32x64}_f8f6f4, E4M3 by E4M3 or
// by E2M1, one E8M0 byte per lane and 32-element block. Lane l supplies row
// l % R (R = 16 or 32) and, of the instruction's K = 2048 / R elements: E2M1,
// 32 g .. 32 g + 31 (g = l / R); E4M3, 16 g .. +15 in its first 16 bytes and
// K / 2 + 16 g .. +15 in the others. Its scale byte is that of elements
// 32 g .. 32 g + 31 for both. Checked on the device against exact products.
// Accuracy: within each group of 8 products of E4M3 codes the instruction
// truncates what lies under 2^-13 of the largest's power of two, then adds the
// groups in fp32. Measured against exact products: 1.5e-5 of the result (root
// mean square), 5e-5 where 1 % of A's columns are 30 times the rest, at any K.
// bf16 products of the same values would be exact up to the fp32 sums, at half
// the rate; an output in bf16 or E4M3 is off by 1.7e-3 or 2.6e-2 by its own
// rounding, so the faster product is taken, and no fp32 output is offered.
// The sums over K, the bias, the activation and the residual are in fp32;
// one rounding to the output.
#include "adahop_internal.h"
#include "mx8_common.h"

namespace adahop {
namespace {

using namespace mx8;

typedef int v8i __attribute__((ext_vector_type(8)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float act_runtime(int act, float z) {
  switch (act) {
    case kActRelu: return act_value<kActRelu>(z);
    case kActSilu: return act_value<kActSilu>(z);
    case kActGelu: return act_value<kActGelu>(z);
    case kActGeluTanh: return act_value<kActGeluTanh>(z);
    default: return z;
  }
}

__device__ __forceinline__ void add_bias(const LinearArgs& a, int64_t c, int64_t end, float (&z)[8]) {
  float b[8];
  if (a.bias_f32)
    load_group<true>(static_cast<const float*>(a.bias), c, end, b);
  else
    load_group<false>(static_cast<const uint16_t*>(a.bias), c, end, b);
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] += b[i];
}

// Epilogue of columns c .. c + 7 (c a multiple of 8, below n) of row r: z
// (and, gated, up) hold the products. For an MXFP8 output (n a multiple of
// 32) the four lanes of a quad hold the four groups of one block.
template <bool Gated>
__device__ __forceinline__ void epilogue8(const LinearArgs& a, int64_t r, int64_t c, float (&z)[8],
                                          float (&up)[8]) {
  if (a.bias != nullptr) {
    add_bias(a, c, a.n, z);
    if constexpr (Gated) add_bias(a, a.n + c, 2 * a.n, up);
  }
  if (a.z != nullptr) {
    store_group<false>(a.z + r * a.ldz, c, a.n, z);
    if constexpr (Gated) store_group<false>(a.z + r * a.ldz + a.n, c, a.n, up);
  }
  float o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    o[i] = act_runtime(a.act, z[i]);
    if constexpr (Gated) o[i] *= up[i];
  }
  if (a.residual != nullptr) {
    float e[8];
    load_group<false>(a.residual + r * a.ldr, c, a.n, e);
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] += e[i];
  }
  if (a.out_scales != nullptr)
    mx8_store_quad(o, static_cast<uint8_t*>(a.out) + r * a.ldo + c, a.out_scales + r * a.ldos + c / 32);
  else
    store_group<false>(static_cast<uint16_t*>(a.out) + r * a.ldo, c, a.n, o);
}

// ---- few rows ---------------------------------------------------------------
// A workgroup computes 16 MT rows by 32 columns of the output (gated: 32 gate
// and 32 up rows of B), its 8 waves each taking every 8th run of 512 along K
// straight from memory into registers; their sums meet in LDS and one wave
// per 16 rows finishes. B is read once, by the workgroup that owns its rows.
constexpr int kFewWaves = 8;

template <bool FP4, bool Gated, int MT>
__global__ void __launch_bounds__(64 * kFewWaves) linear_few_kernel(LinearArgs a) {
  constexpr int NB = Gated ? 4 : 2;         // 16-row blocks of B
  constexpr int Pitch = NB * 16 + 4;
  __shared__ float red[kFewWaves][MT * 16][Pitch];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r16 = lane & 15, g = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 32, m0 = (int64_t)blockIdx.y * (16 * MT);
  const uint8_t* ac[MT];
  const uint8_t* as[MT];
  const uint8_t* bc[NB];
  const uint8_t* bs[NB];
  // Rows past the end repeat the last one: what they give is not stored.
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    int64_t r = m0 + 16 * i + r16;
    r = r < a.m ? r : a.m - 1;
    ac[i] = a.a_codes + r * a.lda;
    as[i] = a.a_scales + r * a.ldas;
  }
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    int64_t c = n0 + 16 * (j & 1) + r16;
    c = (c < a.n ? c : a.n - 1) + (j >= 2 ? a.n : 0);
    bc[j] = a.b_codes + c * a.ldb;
    bs[j] = a.b_scales + c * a.ldbs;
  }
  v4f acc[MT][NB];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = v4f{0, 0, 0, 0};

  const v4i zero = {0, 0, 0, 0};
  for (int64_t k0 = 512 * (int64_t)wave; k0 < a.K; k0 += 512 * kFewWaves) {
    const bool full = k0 + 512 <= a.K;
    uint32_t sa[MT][4], sb[NB][4];
    auto scales = [&](const uint8_t* row, uint32_t (&s)[4]) {
      if (full) {
        u32x4 w;
        __builtin_memcpy(&w, row + k0 / 32, 16);
#pragma unroll
        for (int t = 0; t < 4; ++t) s[t] = w[t] >> (8 * g);
      } else {
#pragma unroll
        for (int t = 0; t < 4; ++t) s[t] = k0 + 128 * t + 32 * g < a.K ? row[k0 / 32 + 4 * t + g] : 127u;
      }
    };
    // 16 bytes of a row's codes, 0 past the end of K (k: first element).
    auto piece = [&](const uint8_t* row, int64_t k, int64_t byte) {
      return full || k < a.K ? *reinterpret_cast<const v4i*>(row + byte) : zero;
    };
#pragma unroll
    for (int i = 0; i < MT; ++i) scales(as[i], sa[i]);
#pragma unroll
    for (int j = 0; j < NB; ++j) scales(bs[j], sb[j]);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int64_t k = k0 + 128 * t;
      v8i fa[MT], fb[NB];
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const v4i lo = piece(ac[i], k + 16 * g, k + 16 * g);
        const v4i hi = piece(ac[i], k + 64 + 16 * g, k + 64 + 16 * g);
        fa[i] = v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      }
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        if constexpr (FP4) {
          const v4i lo = piece(bc[j], k + 32 * g, k / 2 + 16 * g);
          fb[j] = v8i{lo[0], lo[1], lo[2], lo[3], 0, 0, 0, 0};
        } else {
          const v4i lo = piece(bc[j], k + 16 * g, k + 16 * g);
          const v4i hi = piece(bc[j], k + 64 + 16 * g, k + 64 + 16 * g);
          fb[j] = v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        }
      }
      // B first: lane l then holds row l % 16 and columns 4 (l / 16) .. +3.
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              fb[j], fa[i], acc[i][j], FP4 ? 4 : 0, 0, 0, (int)sb[j][t], 0, (int)sa[i][t]);
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
      *reinterpret_cast<v4f*>(&red[wave][16 * i + r16][16 * j + 4 * g]) = acc[i][j];
  __syncthreads();
  // Thread t of the first MT waves: row t / 4 of the tile, columns 8 (t % 4).
  if (threadIdx.x >= 64 * MT) return;
  const int row = threadIdx.x >> 2, col = 8 * (threadIdx.x & 3);
  float z[8], up[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] = up[i] = 0.0f;
#pragma unroll
  for (int w = 0; w < kFewWaves; ++w)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      z[i] += red[w][row][col + i];
      if constexpr (Gated) up[i] += red[w][row][32 + col + i];
    }
  if (m0 + row < a.m && n0 + col < a.n) epilogue8<Gated>(a, m0 + row, n0 + col, z, up);
}

template <bool FP4, bool Gated>
adahop_status few_dispatch(const LinearArgs& a, hipStream_t stream) {
  const unsigned gx = (unsigned)((a.n + 31) / 32);
#define ADAHOP_FEW(MT)                                                                       \
  linear_few_kernel<FP4, Gated, MT>                                                          \
      <<<dim3(gx, (unsigned)((a.m + 16 * MT - 1) / (16 * MT))), dim3(64 * kFewWaves), 0, stream>>>(a)
  if (a.m <= 16) ADAHOP_FEW(1);
  else ADAHOP_FEW(2);
#undef ADAHOP_FEW
  return check_launch("linear_mx");
}

}  // namespace

size_t linear_mx_scratch_bytes(int64_t, int64_t, int64_t, int, int) { return 0; }

adahop_status linear_mx_launch(const LinearArgs& a, int b_fp4, int gated, void*, size_t,
                               hipStream_t stream) {
  if (a.m == 0) return ADAHOP_OK;
  if (b_fp4) return gated ? few_dispatch<true, true>(a, stream) : few_dispatch<true, false>(a, stream);
  return gated ? few_dispatch<false, true>(a, stream) : few_dispatch<false, false>(a, stream);
}

}  // namespace adahop
