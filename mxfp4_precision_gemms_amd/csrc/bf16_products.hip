// Products of bf16 operands stored as they come, in bf16 or fp32 (gfx950): the
// two of the cross entropy's gradient, and a linear layer's weight gradient from
// its MXFP8 input. The kernel stands in bf16_tiles.h. Bound by the matrix cores
// under the power limit where there are tiles enough: 8192 x 4096 x 65536 (dh) 2.88
// ms, 65536 x 4096 x 8192 (dw) 2.94, 4096 x 14336 x 32768 from codes 2.79 .. 2.95.
#include "bf16_tiles.h"

namespace adahop {
namespace {

using namespace tiles;
using mx8::f32x2_to_bf16x2;

// Exchanges the odd groups of 16 (32) lanes of a with the even ones of b.
[[maybe_unused]] __device__ __forceinline__ void swap16(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}
[[maybe_unused]] __device__ __forceinline__ void swap32(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}

// A product as it stands: to bf16 or fp32, on top of `prev` if given. n is a
// multiple of 8, so 8 columns are inside or outside together. bf16 goes out in 32
// bytes a lane: the four lanes of a row exchange their blocks' columns first
// (rows written 8 bytes a lane: 32000 x 2048 from one row in 46 us instead of 39).
struct StoreEpi {
  void* out;
  int64_t ld;
  int f32;
  const float* prev;         // [m][ld_prev], or null
  int64_t ld_prev;
  __device__ __forceinline__ v4f with_prev(v4f v, int64_t r, int64_t c) const {
    v4f p;
    __builtin_memcpy(&p, prev + r * ld_prev + c, 16);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += p[e];
    return v;
  }
  __device__ __forceinline__ void put(v4f v, int64_t r, int64_t c) const {
    if (prev != nullptr) v = with_prev(v, r, c);
    if (f32) {
      __builtin_memcpy(static_cast<float*>(out) + r * ld + c, &v, 16);
    } else {
      const mx8::u32x2 w = {f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3])};
      __builtin_memcpy(static_cast<uint16_t*>(out) + r * ld + c, &w, 8);
    }
  }
  template <bool Wide, int FM>
  __device__ __forceinline__ void store(v4f (&acc)[FM][4], const Spot& at, int64_t m, int64_t n) const {
    static_assert(!Wide, "");
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int64_t r = at.row0 + at.step * i;
      if (at.to == nullptr && !f32) {
        uint32_t w[4][2];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v4f v = acc[i][j];
          if (prev != nullptr && r < m && at.col0 + 16 * j < n) v = with_prev(v, r, at.col0 + 16 * j);
          w[j][0] = f32x2_to_bf16x2(v[0], v[1]);
          w[j][1] = f32x2_to_bf16x2(v[2], v[3]);
        }
        // From columns 16 j + 4 g of block j to columns 16 g + 4 j.
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          swap16(w[0][h], w[1][h]);
          swap16(w[2][h], w[3][h]);
          swap32(w[0][h], w[2][h]);
          swap32(w[1][h], w[3][h]);
        }
        const int64_t c = at.col0 + 12 * ((threadIdx.x >> 4) & 3);
        uint16_t* to = static_cast<uint16_t*>(out) + r * ld + c;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const mx8::u32x4 v = {w[2 * h][0], w[2 * h][1], w[2 * h + 1][0], w[2 * h + 1][1]};
          if (r < m && c + 8 * h < n) __builtin_memcpy(to + 8 * h, &v, 16);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int64_t c = at.col0 + 16 * j;
          if (r >= m || c >= n) continue;
          if (at.to != nullptr) *reinterpret_cast<v4f*>(at.to + (at.lrow + at.step * i) * at.bn + at.lcol + 16 * j) = acc[i][j];
          else put(acc[i][j], r, c);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
};

// Adds the parts of the split tiles in order and stores them, 4 columns a thread
// (1024 elements a workgroup). Eight parts' loads are in flight at a time.
__global__ void __launch_bounds__(256) tile_join_kernel(TileArgs t, StoreEpi epi) {
  const int size = t.bm * t.bn, per = size / 1024;
  const int tile = blockIdx.x / per, at = 1024 * (blockIdx.x - tile * per) + 4 * threadIdx.x;
  int tm, tn;
  tile_at(t.full + tile, t.tiles_m, t.tiles_n, &tm, &tn);
  const int lr = at / t.bn, lc = at - lr * t.bn;
  const int64_t r = (int64_t)tm * t.bm + lr, c = (int64_t)tn * t.bn + lc;
  if (r >= t.m || c >= t.n) return;
  const float* first = t.split_ws + (int64_t)tile * t.parts * size + at;
  v4f v = *reinterpret_cast<const v4f*>(first);
  for (int p = 1; p < t.parts; p += 8) {
    v4f b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      b[i] = *reinterpret_cast<const v4f*>(first + (int64_t)(p + i < t.parts ? p + i : p) * size);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (p + i < t.parts) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += b[i][e];
      }
  }
  epi.put(v, r, c);
}

ProductPlan plan_of(int64_t m, int64_t n, int64_t K, int a, int b) {
  return product_plan(m, n, K, (Kind)a, (Kind)b, true, compute_units());
}
}  // namespace

size_t tile_product_bytes(int64_t m, int64_t n, int64_t K, int a, int b) {
  const ProductPlan p = plan_of(m, n, K, a, b);
  return (size_t)p.split * p.parts * tile_rows(p.tile) * tile_cols(p.tile) * sizeof(float) * (p.split ? 1 : 0);
}

adahop_status tile_product_launch(const TileOperand& a, const TileOperand& b, int64_t m, int64_t n, int64_t K,
                                  const TileOut& out, float* ws, hipStream_t stream) {
  const ProductPlan plan = plan_of(m, n, K, a.kind, b.kind);
  TileArgs t = tile_args(plan, {static_cast<const uint8_t*>(a.p), a.ld, a.chunk, a.scales, a.ld_scales, a.term},
                         {static_cast<const uint8_t*>(b.p), b.ld, b.chunk, b.scales, b.ld_scales}, m, n, K);
  t.split_ws = ws;
  const StoreEpi epi = {out.p, out.ld, out.f32, out.prev, out.ld_prev};
  if (b.kind == kCodes) tile_launch<kAcross, kCodes>(plan, t, epi, stream);
  else if (a.kind == kAcross && a.term != 0) tile_launch<kAcross, kAcross, 2>(plan, t, epi, stream);
  else if (a.kind == kAcross) tile_launch<kAcross, kAcross>(plan, t, epi, stream);
  else if (a.term != 0) tile_launch<kAlong, kAcross, 2>(plan, t, epi, stream);
  else tile_launch<kAlong, kAcross>(plan, t, epi, stream);
  adahop_status st = check_launch("tile product");
  if (st != ADAHOP_OK || t.split == 0) return st;
  tile_join_kernel<<<dim3((unsigned)(t.split * (t.bm * t.bn / 1024))), dim3(256), 0, stream>>>(t, epi);
  return check_launch("tile product join");
}

size_t wgrad_mx8_ws_bytes(int64_t T, int64_t Din, int64_t Dout) {
  return tile_product_bytes(Dout, Din, T, kAcross, kCodes);
}

adahop_status wgrad_mx8_launch(const uint16_t* gy, int64_t ldgy, const Mx8Matrix& x, int64_t T, int64_t Din,
                               int64_t Dout, void* out, int out_f32, int64_t ldo, float* ws, hipStream_t stream) {
  return tile_product_launch({gy, 2 * ldgy, 128, nullptr, 0, kAcross}, {x.codes, x.ldc, 0, x.scales, x.lds, kCodes}, Dout, Din,
                             T, {out, ldo, out_f32, nullptr, 0}, ws, stream);
}

}  // namespace adahop
