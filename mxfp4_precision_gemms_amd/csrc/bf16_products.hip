// Products of bf16 operands stored as they come, in bf16 or fp32 (gfx950): the
// two of the cross entropy's gradient, and a linear layer's weight gradient from
// its MXFP8 input. The kernel stands in bf16_tiles.h. Bound by the matrix cores
// under the power limit where there are tiles enough.
#include "bf16_tiles.h"

namespace adahop {
namespace {

using namespace tiles;
using mx8::f32x2_to_bf16x2;

// A product as it stands: to bf16 or fp32, on top of `prev` if given. n is a
// multiple of 8, so 4 columns are inside or outside together.
struct StoreEpi {
  void* out;
  int64_t ld;
  int f32;
  const float* prev;         // [m][ld_prev], or null
  int64_t ld_prev;
  template <bool Wide>
  __device__ __forceinline__ void store(v4f (&acc)[8][4], const Spot& at, int64_t m, int64_t n) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t r = at.row0 + 16 * i;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int step = (Wide ? 4 : 16) * j;
        if (at.to != nullptr) {
          *reinterpret_cast<v4f*>(at.to + (at.lrow + 16 * i) * kTile + at.lcol + step) = acc[i][j];
          continue;
        }
        const int64_t c = at.col0 + step;
        if (r >= m || c >= n) continue;
        v4f v = acc[i][j];
        if (prev != nullptr) {
          v4f p;
          __builtin_memcpy(&p, prev + r * ld_prev + c, 16);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] += p[e];
        }
        if (f32) {
          __builtin_memcpy(static_cast<float*>(out) + r * ld + c, &v, 16);
        } else {
          const mx8::u32x2 w = {f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3])};
          __builtin_memcpy(static_cast<uint16_t*>(out) + r * ld + c, &w, 8);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
};

// Adds the parts of the split tiles in order and stores them. Workgroup b takes
// rows 16 (b % 16) .. +15 of split tile b / 16.
__global__ void __launch_bounds__(256) tile_join_kernel(TileArgs t, StoreEpi epi) {
  const int tile = blockIdx.x >> 4, band = blockIdx.x & 15;
  int tm, tn;
  tile_at(t.full + tile, t.tiles_m, t.tiles_n, &tm, &tn);
  const int lc = 4 * (threadIdx.x & 63);
  const int64_t c = (int64_t)tn * kTile + lc;
  const float* first = t.split_ws + (int64_t)tile * t.parts * (kTile * kTile);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int lr = 16 * band + (threadIdx.x >> 6) + 4 * i;
    const int64_t r = (int64_t)tm * kTile + lr;
    if (r >= t.m || c >= t.n) continue;
    v4f v = *reinterpret_cast<const v4f*>(first + lr * kTile + lc);
    for (int p = 1; p < t.parts; ++p) {
      const v4f b = *reinterpret_cast<const v4f*>(first + (int64_t)p * (kTile * kTile) + lr * kTile + lc);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += b[e];
    }
    if (epi.prev != nullptr) {
      v4f b;
      __builtin_memcpy(&b, epi.prev + r * epi.ld_prev + c, 16);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += b[e];
    }
    if (epi.f32) {
      __builtin_memcpy(static_cast<float*>(epi.out) + r * epi.ld + c, &v, 16);
    } else {
      const mx8::u32x2 w = {f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3])};
      __builtin_memcpy(static_cast<uint16_t*>(epi.out) + r * epi.ld + c, &w, 8);
    }
  }
}

// The last round of tiles split along K where it leaves half of the compute
// units or more without one (a part: at least 4 pairs of stages).
struct Split {
  int64_t full, split;
  int parts;
};
Split split_of(int64_t m, int64_t n, int64_t K) {
  const int64_t all = tiles_of(m) * tiles_of(n), cus = compute_units(), rem = all % cus;
  int64_t parts = rem > 0 ? cus / rem : 1;
  if (parts > units_of(K) / 4) parts = units_of(K) / 4;
  if (parts > 32) parts = 32;
  if (parts < 2) return {all, 0, 1};
  return {all - rem, rem, (int)parts};
}
}  // namespace

size_t tile_product_bytes(int64_t m, int64_t n, int64_t K) {
  const Split s = split_of(m, n, K);
  return s.split ? (size_t)s.split * s.parts * kTile * kTile * sizeof(float) : 0;
}

adahop_status tile_product_launch(const TileOperand& a, const TileOperand& b, int64_t m, int64_t n, int64_t K,
                                  const TileOut& out, float* ws, hipStream_t stream) {
  TileArgs t = tile_args({static_cast<const uint8_t*>(a.p), a.ld, a.scales, a.ld_scales},
                         {static_cast<const uint8_t*>(b.p), b.ld, b.scales, b.ld_scales}, m, n, K);
  const Split s = split_of(m, n, K);
  t.full = (int)s.full;
  t.split = (int)s.split;
  t.parts = s.parts;
  t.split_ws = ws;
  // Codes are loaded three stages ahead, which has to stay within the next tile.
  if (b.kind == kCodes && t.units < 2) t.units = 2;
  const StoreEpi epi = {out.p, out.ld, out.f32, out.prev, out.ld_prev};
  const dim3 grid = tile_grid(t), block(kThreads);
  if (b.kind == kCodes) bf16_tile_kernel<kAcross, kCodes, StoreEpi><<<grid, block, 0, stream>>>(t, epi);
  else if (a.kind == kAcross) bf16_tile_kernel<kAcross, kAcross, StoreEpi><<<grid, block, 0, stream>>>(t, epi);
  else bf16_tile_kernel<kAlong, kAcross, StoreEpi><<<grid, block, 0, stream>>>(t, epi);
  adahop_status st = check_launch("tile product");
  if (st != ADAHOP_OK || t.split == 0) return st;
  tile_join_kernel<<<dim3((unsigned)(16 * t.split)), dim3(256), 0, stream>>>(t, epi);
  return check_launch("tile product join");
}

adahop_status wgrad_mx8_launch(const uint16_t* gy, int64_t ldgy, const Mx8Matrix& x, int64_t T, int64_t Din,
                               int64_t Dout, void* out, int out_f32, int64_t ldo, float* ws, hipStream_t stream) {
  return tile_product_launch({gy, 2 * ldgy, nullptr, 0, kAcross}, {x.codes, x.ldc, x.scales, x.lds, kCodes}, Dout, Din,
                             T, {out, ldo, out_f32, nullptr, 0}, ws, stream);
}

}  // namespace adahop
