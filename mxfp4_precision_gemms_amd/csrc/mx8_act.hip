// Backward pass of the linear layer's epilogue (gfx950): from the gradient of
// act(z) [* z_up] (+ residual) to the gradient of z, and the bias's.
//
//   plain:  dz = dout * act'(z)
//   gated:  z = [gate | up];  dgate = dout * up * act'(gate),  dup = dout * act(gate)
//   dbias = sum of dz over the rows
// Bound by HBM (one read of dout and z, one write of dz; about 20 fp32
// operations an element): gated 16384 x 14336 445 .. 449 us, 5.2 TB/s; bias +
// GELU 2050 x 8191 27 us, 3.7 TB/s. The bias gradient stays in registers over the rows
// that a workgroup takes, so it costs no second pass over dz; the workgroups'
// partial sums are added in a fixed order by column_reduce_kernel.
#include "adahop_internal.h"
#include "mx8_common.h"

namespace adahop {
namespace {

using namespace mx8;

struct ActBackArgs {
  const void* dout;
  const uint16_t* z;
  uint16_t* dz;
  int64_t m, n;
  int64_t lddo, ldz, lddz;
  int64_t rows_per;      // rows of a workgroup
  float* partial;        // [gridDim.y][n or 2 n], or null
};

// 32 groups of 8 columns by 8 row lanes.
template <int Act, bool Gated, bool DF32>
__global__ void __launch_bounds__(256) act_backward_kernel(ActBackArgs a) {
  using TD = typename Elem<DF32>::type;
  constexpr int P = Gated ? 2 : 1;
  __shared__ float red[P][8][8][32];
  const int cg = threadIdx.x & 31, rl = threadIdx.x >> 5;
  const int64_t c = ((int64_t)blockIdx.x * 32 + cg) * 8;
  float acc[P][8];
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[p][i] = 0.0f;
  const int64_t r0 = (int64_t)blockIdx.y * a.rows_per;
  const int64_t r1 = r0 + a.rows_per < a.m ? r0 + a.rows_per : a.m;
  if (c < a.n) {
    // A row's loads are in flight while the one before is computed.
    struct Row {
      Raw8<DF32> g;
      Raw8<false> z[P];
    };
    auto load = [&](Row& x, int64_t r) {
      x.g.template load<false>(static_cast<const TD*>(a.dout) + r * a.lddo, c, a.n);
#pragma unroll
      for (int p = 0; p < P; ++p) x.z[p].template load<false>(a.z + r * a.ldz + p * a.n, c, a.n);
    };
    Row now, next;
    if (r0 + rl < r1) load(now, r0 + rl);
    for (int64_t r = r0 + rl; r < r1; r += 8) {
      if (r + 8 < r1) load(next, r + 8);
      float g[8], z[P][8], d[P][8];
      now.g.get(g, c, a.n);
#pragma unroll
      for (int p = 0; p < P; ++p) now.z[p].get(z[p], c, a.n);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float value, slope;
        act_both<Act>(z[0][i], &value, &slope);
        if constexpr (Gated) {
          d[0][i] = g[i] * slope * z[1][i];
          d[1][i] = g[i] * value;
          acc[1][i] += d[1][i];
        } else {
          d[0][i] = g[i] * slope;
        }
        acc[0][i] += d[0][i];
      }
#pragma unroll
      for (int p = 0; p < P; ++p) store_group<false>(a.dz + r * a.lddz + p * a.n, c, a.n, d[p]);
      now = next;
    }
  }
  if (a.partial == nullptr) return;
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int i = 0; i < 8; ++i) red[p][rl][i][cg] = acc[p][i];
  __syncthreads();
  // Thread t adds column t of the workgroup's 256 over the row lanes.
  const int i = threadIdx.x & 7, g = threadIdx.x >> 3;
  const int64_t col = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (col < a.n) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      float s = 0.0f;
#pragma unroll
      for (int l = 0; l < 8; ++l) s += red[p][l][i][g];
      a.partial[(int64_t)blockIdx.y * (P * a.n) + p * a.n + col] = s;
    }
  }
}

// Rows a workgroup takes: at least 64 (the partial sums then cost under 2 %
// of the traffic), more where that would leave over 4096 workgroups.
int64_t rows_per_group(int64_t m, int64_t n) {
  const int64_t across = (n + 255) / 256;
  const int64_t down = 4096 / across > 1 ? 4096 / across : 1;
  const int64_t per = (m + down - 1) / down;
  return per < 64 ? 64 : (per + 7) / 8 * 8;
}

template <int Act, bool Gated>
adahop_status act_dispatch(const ActBackArgs& a, dim3 grid, int d_f32, hipStream_t stream) {
  if (d_f32) act_backward_kernel<Act, Gated, true><<<grid, dim3(256), 0, stream>>>(a);
  else act_backward_kernel<Act, Gated, false><<<grid, dim3(256), 0, stream>>>(a);
  return check_launch("act_backward");
}

}  // namespace

int64_t act_backward_groups(int64_t m, int64_t n) {
  const int64_t per = rows_per_group(m, n);
  return m < 1 ? 1 : (m + per - 1) / per;
}

adahop_status act_backward_launch(const void* dout, int d_f32, const uint16_t* z, int act, int gated,
                                  int64_t m, int64_t n, int64_t lddo, int64_t ldz, uint16_t* dz,
                                  int64_t lddz, float* dbias, float* partial, hipStream_t stream) {
  if (m == 0 && dbias == nullptr) return ADAHOP_OK;
  const int64_t groups = act_backward_groups(m, n);
  const ActBackArgs a = {dout, z, dz, m, n, lddo, ldz, lddz, rows_per_group(m, n),
                         dbias != nullptr ? partial : nullptr};
  const dim3 grid((unsigned)((n + 255) / 256), (unsigned)groups);
  adahop_status st = ADAHOP_ERR_INVALID;
#define ADAHOP_ACT(A)                                                                     \
  case A:                                                                                 \
    st = gated ? act_dispatch<A, true>(a, grid, d_f32, stream)                            \
               : act_dispatch<A, false>(a, grid, d_f32, stream);                          \
    break
  switch (act) {
    ADAHOP_ACT(kActNone);
    ADAHOP_ACT(kActRelu);
    ADAHOP_ACT(kActSilu);
    ADAHOP_ACT(kActGelu);
    ADAHOP_ACT(kActGeluTanh);
  }
#undef ADAHOP_ACT
  if (st != ADAHOP_OK || dbias == nullptr) return st;
  return column_reduce_launch(partial, (int)groups, gated ? 2 * n : n, dbias, stream);
}

}  // namespace adahop
