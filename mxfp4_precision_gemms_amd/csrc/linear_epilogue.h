// Epilogue of the linear layer's kernels: from fp32 products to
//   z = product + bias;  out = act(z) [gated: act(z_gate) * z_up] + residual,
// z kept in bf16 if asked for, out rounded once, to bf16 or MXFP8. gfx950 only.
#pragma once

#include "adahop_internal.h"
#include "mx8_common.h"

namespace adahop {
namespace mx8 {

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

__device__ __forceinline__ void load_bias(const LinearArgs& a, int64_t c, int64_t end, float (&b)[8]) {
  if (a.bias_f32)
    load_group<true>(static_cast<const float*>(a.bias), c, end, b);
  else
    load_group<false>(static_cast<const uint16_t*>(a.bias), c, end, b);
}

// Columns c .. c + 7 (c a multiple of 8, below n) of row r: z (and, gated, up)
// hold the products. For an MXFP8 output (n a multiple of 32) the four lanes
// of a quad hold the four groups of one block.
template <bool Gated>
__device__ __forceinline__ void epilogue8(const LinearArgs& a, int64_t r, int64_t c, float (&z)[8],
                                          float (&up)[8]) {
  if (a.bias != nullptr) {
    float b[8];
    load_bias(a, c, a.n, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] += b[i];
    if constexpr (Gated) {
      load_bias(a, a.n + c, a.n + a.n, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) up[i] += b[i];
    }
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

// ---- a wave's accumulators ----------------------------------------------------
// acc[i][j]: lane l holds, of row 16 i + l % 16 of the wave's rows, four
// elements of each of four blocks: with g = l / 16, the 16 columns c + 4 j + e
// (c the lane's first column), or, gated, the 8 gate columns c + 4 j + e
// (j < 2) and the 8 up columns of the same indexes (j >= 2).
// One block row at a time, with the activation's switch (uniform over the
// grid) inside: the other rows' accumulators are all that stays live.
template <int Act, bool Gated>
__device__ __forceinline__ void row_act(v4f (&acc)[4]) {
#pragma unroll
  for (int j = 0; j < (Gated ? 2 : 4); ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float v = act_value<Act>(acc[j][e]);
      acc[j][e] = Gated ? v * acc[j + 2 * Gated][e] : v;
    }
}

template <bool Gated>
__device__ __forceinline__ void row_epilogue(const LinearArgs& a, v4f (&acc)[4], int64_t r, int64_t c) {
  constexpr int H = Gated ? 1 : 2;          // groups of 8 output columns a lane holds
  // Half h of the lane's accumulators starts at column c + 8 h, or, gated,
  // at gate (h = 0) or up (h = 1) column c.
  if (a.bias != nullptr) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float b[8];
      load_bias(a, Gated ? c + h * a.n : c + 8 * h, Gated ? a.n + h * a.n : a.n, b);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[2 * h + e / 4][e % 4] += b[e];
    }
  }
  auto group = [&](int h, float (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = acc[2 * h + e / 4][e % 4];
  };
  if (a.z != nullptr && r < a.m) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float v[8];
      group(h, v);
      store_group<false>(a.z + r * a.ldz + (Gated ? h * a.n : 0), Gated ? c : c + 8 * h, a.n, v);
    }
  }
  switch (a.act) {
    case kActRelu: row_act<kActRelu, Gated>(acc); break;
    case kActSilu: row_act<kActSilu, Gated>(acc); break;
    case kActGelu: row_act<kActGelu, Gated>(acc); break;
    case kActGeluTanh: row_act<kActGeluTanh, Gated>(acc); break;
    default:
      if constexpr (Gated) row_act<kActNone, Gated>(acc);
  }
  float o[H][8];
#pragma unroll
  for (int h = 0; h < H; ++h) group(h, o[h]);
  if (a.residual != nullptr && r < a.m) {
#pragma unroll
    for (int h = 0; h < H; ++h) {
      float e[8];
      load_group<false>(a.residual + r * a.ldr, c + 8 * h, a.n, e);
#pragma unroll
      for (int k = 0; k < 8; ++k) o[h][k] += e[k];
    }
  }
  if (a.out_scales != nullptr) {
    // A block of 32 columns: two lanes' 16 (lanes l and l ^ 16) or, gated,
    // four lanes' 8.
    uint32_t top = 0;
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t b = abs_bits(o[h][k]);
        top = top > b ? top : b;
      }
    uint32_t other = (uint32_t)__shfl_xor((int)top, 16);
    top = top > other ? top : other;
    if constexpr (Gated) {
      other = (uint32_t)__shfl_xor((int)top, 32);
      top = top > other ? top : other;
    }
    const uint32_t byte = mx8_scale_byte(top);
    const bool nan = byte == 255u;
    const float inv = mx8_inverse(nan ? 127u : byte);
    if (r < a.m && c < a.n) {
      uint8_t* to = static_cast<uint8_t*>(a.out) + r * a.ldo + c;
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const u32x2 w = {mx8_pack4(o[h], inv, nan), mx8_pack4(o[h] + 4, inv, nan)};
        __builtin_memcpy(to + 8 * h, &w, 8);
      }
      if (c % 32 == 0) a.out_scales[r * a.ldos + c / 32] = (uint8_t)byte;
    }
  } else if (r < a.m) {
#pragma unroll
    for (int h = 0; h < H; ++h)
      store_group<false>(static_cast<uint16_t*>(a.out) + r * a.ldo, c + 8 * h, a.n, o[h]);
  }
}

template <bool Gated, int FM>
__device__ __forceinline__ void wave_epilogue(const LinearArgs& a, v4f (&acc)[FM][4], int64_t row0,
                                              int64_t c) {
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    row_epilogue<Gated>(a, acc[i], row0 + 16 * i, c);
    __builtin_amdgcn_sched_barrier(0);
  }
}

}  // namespace mx8
}  // namespace adahop
