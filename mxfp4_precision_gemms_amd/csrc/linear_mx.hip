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
#include "linear_epilogue.h"

namespace adahop {
namespace {

using namespace mx8;

typedef int v8i __attribute__((ext_vector_type(8)));
typedef int v4i __attribute__((ext_vector_type(4)));

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

// Up to kFewRows rows the weights are streamed once past all of them.
constexpr int64_t kFewRows = 32;

adahop_status few_launch(const LinearArgs& a, int b_fp4, int gated, hipStream_t stream) {
  if (b_fp4) return gated ? few_dispatch<true, true>(a, stream) : few_dispatch<true, false>(a, stream);
  return gated ? few_dispatch<false, true>(a, stream) : few_dispatch<false, false>(a, stream);
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

}  // namespace

size_t linear_mx_scratch_bytes(int64_t m, int64_t n, int64_t K, int b_fp4, int gated) {
  if (m <= kFewRows) return 0;
  const TilePlan p = linear_tile_plan(m, n, K, b_fp4, gated);
  return p.scale_bytes + p.part_bytes;
}

adahop_status linear_mx_launch(const LinearArgs& a, int b_fp4, int gated, void* scratch, size_t,
                               hipStream_t stream) {
  if (a.m == 0) return ADAHOP_OK;
  if (a.m <= kFewRows) return few_launch(a, b_fp4, gated, stream);
  if (linear_tiles_reach(a.m, a.lda) && linear_tiles_reach(a.n, a.ldb))
    return linear_tiles_launch(a, b_fp4, gated, linear_tile_plan(a.m, a.n, a.K, b_fp4, gated), scratch, stream);
  // Operands of 2 GB and more: in pieces that the tile kernel's offsets
  // reach. Rows 4 MB apart and gated weights of 2 GB a part go by the
  // streaming kernel, in launches that fit its grid.
  auto most = [](int64_t rows, int64_t ld) {
    if (linear_tiles_reach(rows, ld)) return rows;
    int64_t c = ((int64_t{1} << 31) / ld - 1024) / 512 * 512;
    return c > 0 && linear_tiles_reach(c, ld) ? c : int64_t{0};
  };
  const int64_t rows = most(a.m, a.lda), cols = most(a.n, a.ldb);
  const bool tiles = rows > 0 && cols > 0 && (!gated || cols == a.n);
  const int64_t dr = tiles ? rows : int64_t{1} << 20, dc = tiles ? cols : a.n;
  for (int64_t r = 0; r < a.m; r += dr)
    for (int64_t c = 0; c < a.n; c += dc) {
      const LinearArgs p = part_of(a, r, a.m - r < dr ? a.m - r : dr, c, a.n - c < dc ? a.n - c : dc);
      adahop_status st;
      if (tiles) {
        TilePlan t = linear_tile_plan(p.m, p.n, p.K, b_fp4, gated);
        t.parts = 1;
        st = linear_tiles_launch(p, b_fp4, gated, t, scratch, stream);
      } else {
        st = few_launch(p, b_fp4, gated, stream);
      }
      if (st != ADAHOP_OK) return st;
    }
  return ADAHOP_OK;
}

}  // namespace adahop
