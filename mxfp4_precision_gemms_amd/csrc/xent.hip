// Softmax cross entropy over a vocabulary, from hidden states h [T, D] and output
// weights w [V, D] in bf16, without the logits; and its gradient (gfx950).
//
//   z = scale h w^T,  lse_t = log sum_v exp z_tv,  loss_t = lse_t - z_t,y(t)
//   g_tv = scale ((dloss_t + dlse_t) exp(z_tv - lse_t) - dloss_t [v = y(t)])
//   dh = g w,  dw = g^T h
//
// Forward: one product in tiles (bf16_tiles.h) whose epilogue leaves,
// for each row and 64 columns, their maximum and the sum of their exponentials
// under it, and the target's logit; a second kernel joins them in a fixed order.
// Backward: the vocabulary in pieces; for each the logits again, whose epilogue
// writes g of the piece, and the two products of g. Only bf16 runs on the bf16
// matrix cores, so g is held as the sum of two bf16 numbers, the nearest and the
// nearest to what that leaves: off by at most 2^-16 of each element. The caller
// may take the first alone (at most 2^-8; no sum is formed in it), which saves two
// fifths of the operations: bf16 outputs, whose own rounding is 1.7e-3 in the root
// mean square, are then 2.3e-3 .. 2.6e-3 off. Everything else is fp32. dh is
// added up over the pieces in fp32 and rounded once.
//
// Bound by the matrix cores: 2 T V D operations forward, 10 T V D backward (6 with
// one number). Measured: 8192 x 131072 x 4096 (T, V, D) forward 6.0 .. 6.1 ms,
// 1440 .. 1470 TFLOP/s, backward 30.8 .. 31.0 ms, 1420 .. 1430 (one number 17.9 ..
// 18.4, 1440 .. 1480); 1531 x 50021 x 2048 in 245 and 1310 us (781 .. 797). One row
// by the weights' bytes: 1 x 131072 x 4096 in 177 us, 6.1 TB/s.
#include "bf16_tiles.h"

namespace adahop {
namespace {

using namespace tiles;
using mx8::f32x2_to_bf16x2;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMinusInf = -__builtin_inff();

// exp(x - max) with max replaced by 0 where it is no number to subtract, so
// that a row of -inf sums to 0 and one with +inf to +inf.
__device__ __forceinline__ float shift_of(float max) {
  return __builtin_fabsf(max) < __builtin_inff() ? max : 0.0f;
}
__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(kLog2e * x); }

// A wave's block rows in the tile; past the last row, that one.
struct Rows {
  int64_t first;             // the tile's
  int lrow, step, last;
  __device__ __forceinline__ Rows(const Spot& at, int64_t m) : first(at.row0 - at.lrow), lrow(at.lrow), step(at.step) {
    const int64_t rows = m - first;
    last = rows < 256 ? (int)rows - 1 : 255;
  }
  template <typename T>
  __device__ __forceinline__ T of(const T* p, int i) const {
    const int r = lrow + step * i;
    return (p + first)[(unsigned)(r < last ? r : last)];
  }
};
struct Targets {
  const void* p;
  int wide;                  // int64, else int32
  __device__ __forceinline__ int64_t at(int64_t row) const {
    return wide ? static_cast<const int64_t*>(p)[row] : (int64_t)static_cast<const int32_t*>(p)[row];
  }
  // Those of a wave's block rows.
  template <int FM>
  __device__ __forceinline__ void at(const Rows& rows, int64_t (&t)[FM]) const {
    if (wide) {
#pragma unroll
      for (int i = 0; i < FM; ++i) t[i] = rows.of(static_cast<const int64_t*>(p), i);
    } else {
#pragma unroll
      for (int i = 0; i < FM; ++i) t[i] = rows.of(static_cast<const int32_t*>(p), i);
    }
  }
};

// A row's value from those of its four lanes, 16 lanes apart.
template <typename F>
__device__ __forceinline__ float of_row(float x, F&& f) {
#ifdef __HIP_DEVICE_COMPILE__
  const uint32_t v = __builtin_bit_cast(uint32_t, x);
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  const uint32_t u = __builtin_bit_cast(uint32_t, f(__builtin_bit_cast(float, (uint32_t)a[0]), __builtin_bit_cast(float, (uint32_t)a[1])));
  const auto b = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  x = f(__builtin_bit_cast(float, (uint32_t)b[0]), __builtin_bit_cast(float, (uint32_t)b[1]));
#endif
  return x;
}

// ---- epilogues ----------------------------------------------------------------
// What they need of their rows is loaded for all of them before the first is
// stored: loads and stores are waited for in their order, so a row's loads between
// two rows' stores would wait for the first's (gradient of 8192 x 32000 x 1024, g
// in one number: 1290 us, so 1258).
//
// The logits' maximum and sum over the wave's 64 columns of each row, and the
// target's logit.
struct StatsEpi {
  float scale;
  Targets y;
  float2* part;              // [64 columns][T]
  float* said;               // [T]: the target's logit
  template <bool Wide, int FM>
  __device__ __forceinline__ void store(v4f (&acc)[FM][4], const Spot& at, int64_t m, int64_t n) const {
    static_assert(Wide, "");
    float2* to = part + at.group * m;
    const int inside = n - at.col0 < 16 ? (int)(n - at.col0) : 16;
    const Rows rows(at, m);
    int64_t t[FM];             // first used after the sums
    y.at(rows, t);
    __builtin_amdgcn_sched_barrier(0);
    // Step by step for all block rows, so that the exchanges between lanes have
    // others beside them (row by row, through LDS, 8192 x 32000 x 1024 took 435 us;
    // so 412).
    float top[FM], sum[FM];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][e / 4][e % 4] *= scale;
    if (inside < 16) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (e >= inside) acc[i][e / 4][e % 4] = kMinusInf;
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      top[i] = kMinusInf;
#pragma unroll
      for (int e = 0; e < 16; ++e) top[i] = __builtin_fmaxf(top[i], acc[i][e / 4][e % 4]);
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) top[i] = of_row(top[i], [](float a, float b) { return __builtin_fmaxf(a, b); });
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const float by = shift_of(top[i]);
      sum[i] = 0.0f;
#pragma unroll
      for (int e = 0; e < 16; ++e) sum[i] += exp_of(acc[i][e / 4][e % 4] - by);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) sum[i] = of_row(sum[i], [](float a, float b) { return a + b; });
    // All targets are here: one that no lane used would otherwise be waited for, with
    // the next stages' loads, where its register is taken again.
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 15));
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int64_t r = at.row0 + at.step * i;
      if (r < m) {
        if ((threadIdx.x & 48) == 0) to[r] = float2{top[i], sum[i]};
        const int64_t d = t[i] - at.col0;
        if (d >= 0 && d < inside) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (d == e) said[r] = acc[i][e / 4][e % 4];
        }
      }
    }
  }
};

// The gradient of a piece's logits, columns v0 .. of the vocabulary, 64 columns of
// all rows together: a stage of either product then reads whole stretches of
// memory (from whole rows dh of 8192 x 65536 x 4096 took 2904 us, so 2861; of
// 1531 x 50021 x 2048 269 and 264). A tile's columns past the piece's end are
// written as zeros. all and the target's place of each row are held, its share is
// read again by the lane that needs it: its registers would be spilled.
// Terms: 2, g's nearest bf16 and, `term` elements on, that of what it leaves.
template <int Terms>
struct GradEpi {
  float scale;
  Targets y;
  const float* lse;
  const float* dloss;
  const float* dlse;         // or null
  int64_t v0, vocab;
  uint16_t* g;               // [64 columns][padded][64]
  int64_t term;
  int64_t padded;            // T rounded up to a multiple of 64; rows from T on are zeros
  // What the bf16 of these bits leaves of v (exact); nothing where it is no number.
  static __device__ __forceinline__ float left(float v, uint32_t bits) {
    const float near = __builtin_bit_cast(float, bits);
    return __builtin_fabsf(near) < __builtin_inff() ? v - near : 0.0f;
  }
  template <bool Wide, int FM>
  __device__ __forceinline__ void store(v4f (&acc)[FM][4], const Spot& at, int64_t m, int64_t n) const {
    static_assert(Wide, "");
    const int inside = n - at.col0 < 16 ? (int)(n - at.col0) : 16;
    const Rows rows(at, m);
    int place[FM];             // the target's, in the lane's columns
    float less[FM], all[FM];
    {
      int64_t t[FM];
      y.at(rows, t);
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        less[i] = rows.of(lse, i);
        all[i] = rows.of(dloss, i);
      }
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        if (t[i] < 0 || t[i] >= vocab) all[i] = 0.0f;
        const int64_t d = t[i] - v0 - at.col0;
        place[i] = d >= 0 && d < inside ? (int)d : -1;
      }
      if (dlse != nullptr) {
#pragma unroll
        for (int i = 0; i < FM; ++i) all[i] += rows.of(dlse, i);
      }
#pragma unroll
      for (int i = 0; i < FM; ++i) all[i] *= scale;
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int64_t r = at.row0 + at.step * i;
      float own = 0.0f;
      if (r < m && place[i] >= 0) own = scale * dloss[r];
      uint16_t* to = g + (at.group * padded + r) * 64 + at.col0 % 64;
#pragma unroll
      for (int e0 = 0; e0 < 16; e0 += 8) {
        mx8::u32x4 w[Terms] = {};
        if (r < m) {
          float v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            v[e] = all[i] * exp_of(__builtin_fmaf(acc[i][(e0 + e) / 4][e % 4], scale, -less[i]));
            if (e0 + e >= inside) v[e] = 0.0f;
            if (place[i] == e0 + e) v[e] -= own;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            w[0][e] = f32x2_to_bf16x2(v[2 * e], v[2 * e + 1]);
            if constexpr (Terms == 2)
              w[1][e] = f32x2_to_bf16x2(left(v[2 * e], w[0][e] << 16), left(v[2 * e + 1], w[0][e] & 0xFFFF0000u));
          }
        }
        if (r < padded) {
#pragma unroll
          for (int s = 0; s < Terms; ++s) *reinterpret_cast<mx8::u32x4*>(to + s * term + e0) = w[s];
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
};

// ---- joining ------------------------------------------------------------------
// lse and loss of a row from its parts' maxima and sums: 256 / Rows lanes a row,
// lane l taking parts l, l + lanes, ...; then the lanes in pairs.
struct FinishArgs {
  const float2* part;
  const float* said;
  Targets y;
  int64_t rows, vocab;
  int64_t parts;
  float* loss;
  float* lse;
};
__device__ __forceinline__ float2 join(float2 a, float2 b) {
  const float top = __builtin_fmaxf(a.x, b.x), by = shift_of(top);
  // A part of -inf alone holds a sum of 0 (or a NaN): no shift applies to it.
  auto shifted = [&](float2 p) { return p.x == kMinusInf ? p.y : p.y * exp_of(shift_of(p.x) - by); };
  return float2{top, shifted(a) + shifted(b)};
}
template <int Rows>
__global__ void __launch_bounds__(256) xent_finish_kernel(FinishArgs a) {
  constexpr int Lanes = 256 / Rows;
  __shared__ float2 red[Lanes][Rows + 1];
  const int row = threadIdx.x % Rows, lane = threadIdx.x / Rows;
  for (int64_t base = (int64_t)blockIdx.x * Rows; base < a.rows; base += (int64_t)gridDim.x * Rows) {
    const int64_t r = base + row;
    float2 s = {kMinusInf, 0.0f};
    if (r < a.rows) {
#pragma unroll 8
      for (int64_t p = lane; p < a.parts; p += Lanes) s = join(s, a.part[p * a.rows + r]);
    }
    red[lane][row] = s;
#pragma unroll
    for (int half = Lanes / 2; half >= 1; half /= 2) {
      __syncthreads();
      if (lane < half) red[lane][row] = join(red[lane][row], red[lane + half][row]);
    }
    if (lane == 0 && r < a.rows) {
      s = red[0][row];
      const float lse = shift_of(s.x) + logf(s.y);
      const int64_t t = a.y.at(r);
      a.lse[r] = lse;
      a.loss[r] = t >= 0 && t < a.vocab ? lse - a.said[r] : 0.0f;
    }
    __syncthreads();
  }
}

// ---- host ---------------------------------------------------------------------
Operand along(const uint16_t* p, int64_t ld) { return {reinterpret_cast<const uint8_t*>(p), 2 * ld, 128, nullptr, 0}; }
// Groups of 64 columns that leave a maximum and a sum for a row.
int64_t groups_of(int64_t V) { return whole_tiles(V) / 64; }
TileOperand operand(const uint16_t* p, int64_t ld, Kind kind) { return {p, 2 * ld, 128, nullptr, 0, kind}; }

}  // namespace

size_t xent_ws_bytes(int64_t T, int64_t V) {
  return align_up(sizeof(float2) * (size_t)groups_of(V) * (size_t)T, kAlign) + sizeof(float) * (size_t)T;
}

adahop_status xent_launch(const XentArgs& a, float* loss, float* lse, void* ws, hipStream_t stream) {
  const Targets y = {a.targets, a.wide_targets};
  float2* part = static_cast<float2*>(ws);
  float* said = reinterpret_cast<float*>(static_cast<char*>(ws) +
                                         align_up(sizeof(float2) * (size_t)groups_of(a.V) * (size_t)a.T, kAlign));
  const ProductPlan plan = product_plan(a.T, a.V, a.D, kAlong, kAlong, false, compute_units());
  const TileArgs t = tile_args(plan, along(a.h, a.ldh), along(a.w, a.ldw), a.T, a.V, a.D);
  tile_launch<kAlong, kAlong>(plan, t, StatsEpi{a.scale, y, part, said}, stream);
  const adahop_status st = check_launch("xent");
  if (st != ADAHOP_OK) return st;
  const FinishArgs f = {part, said, y, a.T, a.V, (int64_t)t.tiles_n * (t.bn / 64), loss, lse};
  // Few rows: more lanes a row (1 row of 500 parts: 7 us with 16 lanes, 4 with 128).
  auto groups = [&](int rows) {
    const int64_t n = (a.T + rows - 1) / rows;
    return dim3((unsigned)(n < 1 << 20 ? n : 1 << 20));
  };
  if (a.T <= 512) xent_finish_kernel<2><<<groups(2), dim3(256), 0, stream>>>(f);
  else xent_finish_kernel<16><<<groups(16), dim3(256), 0, stream>>>(f);
  return check_launch("xent_finish");
}

// ---- backward -------------------------------------------------------------------
namespace {
struct BackLayout {
  XentPieces p;
  size_t off_sum, off_split, bytes;
};
BackLayout back_layout(int64_t T, int64_t V, int64_t D, int64_t piece, int terms, bool dh, bool dw) {
  BackLayout l{};
  l.p = xent_pieces(T, V, piece, terms);
  size_t at = align_up(2 * (size_t)terms * (size_t)padded_rows(T) * (size_t)l.p.size, kAlign);
  l.off_sum = at;
  if (dh && l.p.count > 1) at += align_up(4 * (size_t)T * (size_t)D, kAlign);
  l.off_split = at;
  const int64_t last = V - (l.p.count - 1) * l.p.size;
  size_t split = 0;
  for (const int64_t n : {l.p.size < V ? l.p.size : V, last}) {
    const size_t s = dh ? tile_product_bytes(T, D, n, kAlong, kAcross) : 0, u = dw ? tile_product_bytes(n, D, T, kAcross, kAcross) : 0;
    split = split > s ? split : s;
    split = split > u ? split : u;
  }
  l.bytes = at + split;
  return l;
}

}  // namespace

size_t xent_backward_ws_bytes(int64_t T, int64_t V, int64_t D, int64_t piece, int terms, bool dh, bool dw) {
  return T == 0 ? 0 : back_layout(T, V, D, piece, terms, dh, dw).bytes;
}

adahop_status xent_backward_launch(const XentArgs& a, const XentGrad& b, int64_t piece, void* ws,
                                   hipStream_t stream) {
  if (a.T == 0) {
    if (b.dw == nullptr) return ADAHOP_OK;
    // A product over no rows: zeros.
    const TileOut to = {b.dw, b.lddw, b.dw_f32, nullptr, 0};
    return tile_product_launch(operand(nullptr, 8, kAcross), operand(nullptr, 8, kAcross), a.V, a.D, 0, to, nullptr,
                               stream);
  }
  const BackLayout l = back_layout(a.T, a.V, a.D, piece, b.terms, b.dh != nullptr, b.dw != nullptr);
  uint16_t* g = static_cast<uint16_t*>(ws);
  float* sum = reinterpret_cast<float*>(static_cast<char*>(ws) + l.off_sum);
  float* split = reinterpret_cast<float*>(static_cast<char*>(ws) + l.off_split);
  const Targets y = {a.targets, a.wide_targets};
  const int64_t padded = padded_rows(a.T), term = padded * l.p.size;
  auto part = [&](Kind kind) { return TileOperand{g, 128, 128 * padded, nullptr, 0, kind, b.terms == 2 ? 2 * term : 0}; };
  for (int64_t q = 0; q < l.p.count; ++q) {
    const int64_t v0 = q * l.p.size, n = a.V - v0 < l.p.size ? a.V - v0 : l.p.size;
    const uint16_t* w = a.w + v0 * a.ldw;
    const ProductPlan plan = product_plan(a.T, n, a.D, kAlong, kAlong, false, compute_units());
    const TileArgs t = tile_args(plan, along(a.h, a.ldh), along(w, a.ldw), a.T, n, a.D);
    auto logits = [&](auto epi) { tile_launch<kAlong, kAlong>(plan, t, epi, stream); };
    if (b.terms == 2) logits(GradEpi<2>{a.scale, y, b.lse, b.dloss, b.dlse, v0, a.V, g, term, padded});
    else logits(GradEpi<1>{a.scale, y, b.lse, b.dloss, b.dlse, v0, a.V, g, term, padded});
    adahop_status st = check_launch("xent_backward logits");
    if (st != ADAHOP_OK) return st;
    if (b.dh != nullptr) {
      const bool last = q + 1 == l.p.count;
      const TileOut to = {last ? b.dh : sum, last ? b.lddh : a.D, last ? b.dh_f32 : 1, q > 0 ? sum : nullptr, a.D};
      st = tile_product_launch(part(kAlong), operand(w, a.ldw, kAcross), a.T, a.D, n, to, split,
                               stream);
      if (st != ADAHOP_OK) return st;
    }
    if (b.dw != nullptr) {
      const TileOut to = {static_cast<char*>(b.dw) + (b.dw_f32 ? 4 : 2) * v0 * b.lddw, b.lddw, b.dw_f32, nullptr, 0};
      st = tile_product_launch(part(kAcross), operand(a.h, a.ldh, kAcross), n, a.D, a.T, to, split,
                               stream);
      if (st != ADAHOP_OK) return st;
    }
  }
  return ADAHOP_OK;
}

}  // namespace adahop
