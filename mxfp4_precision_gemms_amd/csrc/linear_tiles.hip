// Linear layer on microscaled operands, many rows: output tiles fed through LDS
// (gfx950). The mathematics, the matrix instruction's operand layout and its
// accuracy stand in linear_mx.hip.
//
// A workgroup of WM x WN waves computes 16 FM WM rows by 64 WN rows of B
// (gated: 32 WN gate and 32 WN up rows), a wave 16 FM by 64 as FM x 4 blocks
// of v_mfma_scale_f32_16x16x128. K advances 128 elements a stage through NS
// LDS slots that global->LDS loads fill up to NS stages ahead.
//
// LDS rows of 128 bytes (E4M3) or 64 (E2M1) keep their 16-byte chunks XORed
// with row bits, so that the 16 rows which one quarter of a wave reads at one
// chunk lie in 16 different 16-byte columns of the 256 bytes of banks: A's
// are consecutive; B's are permuted so that a lane's four blocks hold 16
// consecutive columns of the output (gated: 8 gate and the same 8 up columns),
// which makes the epilogue's loads and stores 16 bytes wide. Row r of block j
// (r = 4 q + s) is B row 16 q + 4 j + s of the wave's 64, gated 32 (j / 2) +
// 8 q + 4 (j % 2) + s; its chunk c is stored at c ^ (2 q + s / 2) (E2M1:
// c ^ q).
//
// Measured: 32768 x 4096 x 14336, E4M3 weights: 1.38 .. 1.50 ms, 2.6 .. 2.8
// PFLOP/s; the matrix cores busy 69 % of the time at a clock that the power
// limit holds at 1.72 GHz. 4096 x 14336 gated x 4096, E2M1 weights: 341 .. 379
// us, 2.5 .. 2.8 PFLOP/s, busy 66 % at 1.97 GHz. Few tiles: what a compute unit
// loads (30 .. 50 GB/s) binds, so K is split until all have work.
#include <type_traits>
#include <utility>

#include "linear_epilogue.h"

namespace adahop {
namespace {

using namespace mx8;

typedef int v8i __attribute__((ext_vector_type(8)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;

template <typename F, int... Is>
__device__ __forceinline__ void for_each_impl(F&& f, std::integer_sequence<int, Is...>) {
  (f(std::integral_constant<int, Is>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void for_each(F&& f) {
  for_each_impl(f, std::make_integer_sequence<int, N>{});
}
template <int V>
using Int = std::integral_constant<int, V>;

// s_waitcnt immediate: vmcnt bits [3:0] and [15:14], expcnt [6:4] (7: no
// wait), lgkmcnt [11:8].
constexpr int waitcnt_imm(int vm, int lgkm) {
  return (vm & 15) | ((vm >> 4) << 14) | (7 << 4) | ((lgkm & 15) << 8);
}
constexpr int kBufferFlags = 0x00020000;   // raw buffer descriptor word 3
// An offset past the end of every buffer here (extents stay below 2^31 - 16,
// a tile's included): such a load returns 0 without touching memory.
constexpr int kPastEnd = 0x7FFFFFF0;
constexpr int kGroupM = 4;                 // tile rows that run together on one XCD (8: 351 us instead of 339
                                           // on 4096 x 14336 gated x 4096)

struct TileArgs {
  const uint8_t* sa;         // scales: row strides, and from one stage
  const uint8_t* sb;         // (Stay) or 4 stages to the next, in bytes
  int sa_row, sa_step, sb_row, sb_step;
  int sa_bytes, sb_bytes;
  int a_bytes, b_bytes;      // extents of A and B (gated: of one part)
  int tiles_m, tiles_n;
  int nk;                    // stages of K
  int parts;                 // K parts of a tile (1: the epilogue runs here)
  float* partial;            // [part][tile][wave][FM][4][64] v4f
};

// Logical position of workgroup `bid` of `count`: the hardware deals
// workgroups round-robin to the 8 XCDs; each gets a contiguous band.
__device__ __forceinline__ int xcd_band(int bid, int count) {
  return count % 8 == 0 ? (bid & 7) * (count / 8) + (bid >> 3) : bid;
}
// Tile of a logical position: groups of kGroupM tile rows, column by column,
// so that the tiles an XCD runs at once share rows of both operands in its L2.
__device__ __forceinline__ void tile_at(int pos, int tiles_m, int tiles_n, int* tm, int* tn) {
  const int per_group = kGroupM * tiles_n;
  const int group = pos / per_group, first = group * kGroupM;
  const int gm = tiles_m - first < kGroupM ? tiles_m - first : kGroupM;
  const int in = pos - group * per_group;
  *tm = first + in % gm;
  *tn = in / gm;
}

// Scale words of a slot: A's rows (64 at least, so that one load of a wave
// holds rows of one operand), then B's, in loads of 64 by Waves waves.
constexpr int scale_rows_a(int BM) { return BM < 64 ? 64 : BM; }
constexpr int scale_loads(int BM, int BN, int Waves) {
  return ((scale_rows_a(BM) + BN) / 64 + Waves - 1) / Waves;
}

// Loads of a wave in a stage: every fourth takes the scales too.
constexpr int loads_at(int stage, int loads, int scales) { return loads + ((stage & 3) == 0 ? scales : 0); }

template <bool FP4, int BM, int BN>
struct CodeSlot {
  uint8_t a[BM * 128];
  uint8_t b[BN * (FP4 ? 64 : 128)];
};
// Stay: the halves of each wave's A rows and B with the stage's scale words
// are freed, and filled, at different times of a stage.
struct HalfSlot {
  uint8_t a[128 * 128];
};
template <bool FP4>
struct WordSlot {
  uint32_t sc[512];                          // A's 4 groups of 64 words, then B's
  uint8_t b[256 * (FP4 ? 64 : 128)];
};

template <bool FP4, bool Gated, int WM, int WN, int FM, int NS>
__global__ void __launch_bounds__(64 * WM * WN, 1) linear_tile_kernel(LinearArgs a, TileArgs t) {
#ifdef __HIP_DEVICE_COMPILE__                        // the host pass needs the launch stub alone
  constexpr int Waves = WM * WN, BM = 16 * FM * WM, BN = 64 * WN;
  constexpr int Bb = FP4 ? 64 : 128;                   // bytes of a B row and stage
  constexpr int Ra = 8 * Waves, Rb = (FP4 ? 16 : 8) * Waves;   // rows a load of every wave fills
  constexpr int LA = BM / Ra, LB = BN / Rb, LS = scale_loads(BM, BN, Waves);
  constexpr int Sb = scale_rows_a(BM);                 // row of B's first scales
  // Two slots: workgroups stay, and load the next tile's first stages during a
  // tile's last ones and its epilogue; a tile takes an even number of stages
  // (one of zeros follows an odd number), so that each begins in slot 0. Four
  // slots: one tile a workgroup.
  constexpr bool Stay = NS == 2;
  static_assert(Stay ? WM == 2 && WN == 4 && FM == 8 : NS == 4, "");
  // Scales. Stay: ordered beforehand by stage and 64 rows, so that a word holds
  // one block of the four rows that a lane's fragments take; each fragment
  // names its byte. Else 16 bytes a row every 4 stages, where possible from
  // the operand as it is, held as one byte a stage. (A word a row and stage
  // costs as many requests as the codes: 391 us instead of 344 for 4096 x
  // 14336 gated x 4096, 88 instead of 64 for 64 x 4096 x 14336.)
  constexpr int Unit = Stay ? 2 : 4;
  constexpr int Codes = LA + LB;                       // loads of a wave and stage
  static_assert(BM % Ra == 0 && BN % Rb == 0 && NS * Codes + LS < 64, "");
  using S = CodeSlot<FP4, BM, BN>;
  // One LDS object for each part that is filled at once: alias analysis then
  // sees that loads into one do not touch another, and adds no wait before
  // the reads.
  __shared__ __attribute__((aligned(1024))) v4i scales[Stay ? 1 : 64 * Waves * LS];
  __shared__ __attribute__((aligned(1024))) S s0;
  __shared__ __attribute__((aligned(1024))) S s1;
  __shared__ __attribute__((aligned(1024))) S s2;
  __shared__ __attribute__((aligned(1024))) S s3;
  __shared__ __attribute__((aligned(1024))) HalfSlot f0, f1, r0, r1;   // Stay: first and last rows of A
  __shared__ __attribute__((aligned(1024))) WordSlot<FP4> w0, w1;
  auto slot = [&](auto I) -> S& {
    if constexpr (I == 0) return s0;
    else if constexpr (I == 1) return s1;
    else if constexpr (I == 2) return s2;
    else return s3;
  };
  auto half = [&](auto I, auto H) -> HalfSlot& {
    if constexpr (I == 0 && H == 0) return f0;
    else if constexpr (I == 0) return r0;
    else if constexpr (H == 0) return f1;
    else return r1;
  };
  auto words = [&](auto I) -> WordSlot<FP4>& {
    if constexpr (I == 0) return w0;
    else return w1;
  };

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int r16 = lane & 15, g = lane >> 4;
  const int items = t.tiles_m * t.tiles_n * t.parts;

  // The stages and what they call are always inlined: a call would pass the
  // accumulators through memory.

  // ---- loader: this wave's share of each stage, NS stages ahead -------------
  const __amdgpu_buffer_rsrc_t rb_a = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(a.a_codes), 0, t.a_bytes, kBufferFlags);
  // Gated: load j of this wave fills gate (part 0) or up (part 1) rows; the
  // rows of a load lie in one 32-row half of a 64-row slice.
  auto part_of = [&](int j) { return Gated ? ((Rb * j + (Rb / Waves) * wave) >> 5) & 1 : 0; };
  const __amdgpu_buffer_rsrc_t rb_b0 = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(a.b_codes + (Rb >= 64 ? part_of(0) * a.n * a.ldb : 0)), 0, t.b_bytes, kBufferFlags);
  const __amdgpu_buffer_rsrc_t rb_b1 = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(a.b_codes + (Gated && Rb < 64 ? a.n * a.ldb : 0)), 0, t.b_bytes, kBufferFlags);
  const int ra = 8 * wave + (lane >> 3);                     // A row of load 0; + Ra j
  const int ca = (lane & 7) ^ ((ra >> 1) & 7);               // logical chunk of load 0
  const int rb = (FP4 ? 16 : 8) * wave + (lane >> (FP4 ? 2 : 3));
  // XOR key of B row r: q and s as in the fragments' row order. Rb is a power
  // of two, so the key of row rb + Rb j is that of rb XOR that of Rb j.
  auto key_b = [](int r) constexpr {
    const int q = (r >> (Gated ? 3 : 4)) & 3;
    return FP4 ? q : 2 * q + ((r >> 1) & 1);
  };
  const int cb = (lane & (FP4 ? 3 : 7)) ^ key_b(rb);
  static_assert(Ra % 16 == 0, "A's key is the same for every load");
  // A load's address is this lane's offset within a tile (below), plus the
  // tile's and the load's rows, scalar. A 64-row slice of B holds, gated, 32
  // gate and 32 up rows of 32 columns.
  const uint32_t oa = (uint32_t)ra * (uint32_t)a.lda;
  const uint32_t ob = (uint32_t)(Gated ? (rb >> 6) * 32 + (rb & 31) : rb) * (uint32_t)a.ldb;
  // Scale words: load q of this wave holds rows 64 (wave + Waves q) + lane of
  // the slot's.
  bool s_is_a[LS], s_none[LS];
  uint32_t os[LS];
  __amdgpu_buffer_rsrc_t rb_s[LS];
#pragma unroll
  for (int q = 0; q < LS; ++q) {
    const int first = 64 * (wave + Waves * q);
    s_is_a[q] = first < Sb;
    const int r = first + lane - (s_is_a[q] ? 0 : Sb);
    s_none[q] = r >= (s_is_a[q] ? BM : BN);
    const int row = Gated && !s_is_a[q] ? (r >> 6) * 32 + (r & 31) + ((r >> 5) & 1) * (int)a.n : r;
    os[q] = Stay ? 4u * r : (uint32_t)row * (uint32_t)(s_is_a[q] ? t.sa_row : t.sb_row);
    rb_s[q] = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(s_is_a[q] ? t.sa : t.sb), 0,
                                                s_is_a[q] ? t.sa_bytes : t.sb_bytes, kBufferFlags);
  }

  auto item_at = [&](int round) {
    const int G = gridDim.x, base = round * G;
    if (base >= items) return -1;
    const int cnt = items - base < G ? items - base : G;
    return (int)blockIdx.x < cnt ? base + xcd_band(blockIdx.x, cnt) : -1;
  };
  auto locate = [&](int item, int* tm, int* tn, int* k0, int* k1) {
    const int tile = item / t.parts, part = item - tile * t.parts;
    int m_, n_;
    tile_at(tile, t.tiles_m, t.tiles_n, &m_, &n_);
    *tm = __builtin_amdgcn_readfirstlane(m_);
    *tn = __builtin_amdgcn_readfirstlane(n_);
    const int64_t units = (t.nk + Unit - 1) / Unit;
    *k0 = __builtin_amdgcn_readfirstlane(Unit * (int)(units * part / t.parts));
    const int end = Unit * (int)(units * (part + 1) / t.parts);
    *k1 = __builtin_amdgcn_readfirstlane(Stay || end < t.nk ? end : t.nk);
  };
  // An item's place, all scalar.
  struct Place {
    int tm, tn, k0, k1;
    uint32_t a, b, sa, sb;
  };
  // Without an item: a stage past the end of any K.
  auto place = [&](int item) {
    Place p{0, 0, 1 << 23, 1 << 24, 0, 0, 0, 0};
    if (item < 0) return p;
    locate(item, &p.tm, &p.tn, &p.k0, &p.k1);
    p.a = (uint32_t)(p.tm * BM) * (uint32_t)a.lda;
    p.b = (uint32_t)(p.tn * (Gated ? BN / 2 : BN)) * (uint32_t)a.ldb;
    p.sa = (uint32_t)(p.tm * BM) * (uint32_t)t.sa_row;
    p.sb = (uint32_t)(p.tn * (Gated && !Stay ? BN / 2 : BN)) * (uint32_t)t.sb_row;
    return p;
  };
  // Load q of stage k of an item into slot I. Chunks past the end of K are
  // zeros, for both operands; a stage past it must not have NaN scales.
  auto issue = [&](auto I, auto Q, int k, uint32_t base_a, uint32_t base_b, uint32_t base_sa,
                   uint32_t base_sb) __attribute__((always_inline)) {
    constexpr int q = decltype(Q)::value;
    // The scalar offset stays inside the buffers (the range check may
    // subtract it from their size).
    const int kt = k < t.nk ? k : 0;
    if constexpr (q < LA) {
      const int c = ca ^ ((Ra * q / 2) & 7);
      const uint32_t v = 128 * k + 16 * c < (int)a.K ? oa + 16 * c : kPastEnd;
      lds_void* to;
      // Stay: loads 0 and 2 hold the first halves of the waves' rows.
      if constexpr (Stay) to = (lds_void*)&half(I, Int<q % 2>{}).a[1024 * (Waves * (q / 2) + wave)];
      else to = (lds_void*)&slot(I).a[1024 * (Waves * q + wave)];
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb_a, to, 16, (int)(v + (base_a + q * Ra * (uint32_t)a.lda)),
                                               128 * kt, 0, 0);
    } else if constexpr (q < Codes) {
      constexpr int j = q - LA;
      const int c = cb ^ key_b(Rb * j);
      const uint32_t v = Bb * k + 16 * c < (int)(FP4 ? a.K / 2 : a.K) ? ob + 16 * c : kPastEnd;
      // Rows of B from one load to the next: Rb, of which gated a half each
      // gate and up rows.
      constexpr int step = !Gated ? Rb * j : Rb >= 64 ? Rb * j / 2 : 32 * (Rb * j / 64) + (Rb * j) % 32;
      const __amdgpu_buffer_rsrc_t r = Gated && Rb < 64 && ((Rb * j) >> 5) % 2 == 1 ? rb_b1 : rb_b0;
      lds_void* to;
      if constexpr (Stay) to = (lds_void*)&words(I).b[1024 * (Waves * j + wave)];
      else to = (lds_void*)&slot(I).b[1024 * (Waves * j + wave)];
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, to, 16, (int)(v + (base_b + step * (uint32_t)a.ldb)), Bb * kt,
                                               0, 0);
    } else {
      // A stage's words, or, else, 16 bytes a row for stages k .. k + 3.
      constexpr int j = q - Codes;
      const uint32_t v = k < t.nk && !s_none[j] ? os[j] : kPastEnd;
      const int at = (int)(v + (s_is_a[j] ? base_sa : base_sb));
      const int step = s_is_a[j] ? t.sa_step : t.sb_step;
      if constexpr (Stay)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rb_s[j], (lds_void*)&words(I).sc[64 * (wave + Waves * j)], 4, at,
                                                 kt * step, 0, 0);
      else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rb_s[j], (lds_void*)&scales[64 * (wave + Waves * j)], 16, at,
                                                 (kt >> 2) * step, 0, 0);
    }
  };
  // Stage k of item `now`, or, past its last, of item `next`: the scalar
  // selects keep the stages free of branches.
  auto issue_at = [&](auto I, auto Q, int k, const Place& now, const Place& next) __attribute__((always_inline)) {
    const bool in = k < now.k1;
    if constexpr (!Stay) {
      issue(I, Q, in ? k : 1 << 23, now.a, now.b, now.sa, now.sb);
      return;
    }
    issue(I, Q, in ? k : k - now.k1 + next.k0, in ? now.a : next.a, in ? now.b : next.b,
          in ? now.sa : next.sa, in ? now.sb : next.sb);
  };

  // ---- fragments ------------------------------------------------------------
  const int q4 = r16 >> 2, sub = r16 & 3;
  const int fa_row = 16 * FM * wm + r16;
  const int fa_lo = (Stay ? 64 * wm + r16 : fa_row) * 128 + 16 * (g ^ ((r16 >> 1) & 7));
  const int fb_row = 64 * wn + (Gated ? 8 : 16) * q4 + sub;
  const int fb_lo = fb_row * Bb + 16 * (FP4 ? g ^ q4 : g ^ (2 * q4 + (sub >> 1)));
  auto b_step = [](int j) { return Gated ? 32 * (j >> 1) + 4 * (j & 1) : 4 * j; };

  v4f acc[FM][4];
  v8i fa[4], fb[4];
  int sa[FM], sb[4];                         // Stay: sa[0], sa[1] and sb[0] alone
  [[maybe_unused]] v4i raw[FM + 4];
  auto read_a = [&](auto I, auto B, auto J) __attribute__((always_inline)) {
    constexpr int b = decltype(B)::value, i = decltype(J)::value;
    const uint8_t* p;
    if constexpr (Stay) p = half(I, Int<i / 4>{}).a + 2048 * (i % 4);
    else p = slot(I).a + 2048 * i;
    const v4i lo = *reinterpret_cast<const v4i*>(p + fa_lo);
    const v4i hi = *reinterpret_cast<const v4i*>(p + (fa_lo ^ 64));
    fa[b] = v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  };
  auto read_b = [&](auto I, auto J) __attribute__((always_inline)) {
    constexpr int j = decltype(J)::value;
    const uint8_t* p;
    if constexpr (Stay) p = words(I).b + Bb * b_step(j);
    else p = slot(I).b + Bb * b_step(j);
    const v4i lo = *reinterpret_cast<const v4i*>(p + fb_lo);
    if constexpr (FP4) {
      fb[j] = v8i{lo[0], lo[1], lo[2], lo[3], 0, 0, 0, 0};
    } else {
      const v4i hi = *reinterpret_cast<const v4i*>(p + (fb_lo ^ 64));
      fb[j] = v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    }
  };
  // Stay: byte i % 4 of sa[i / 4] is that of block row i, byte j of sb[0] that
  // of block j.
  auto read_words = [&](auto I) __attribute__((always_inline)) {
    const uint32_t* p = words(I).sc + lane;
    sa[0] = (int)p[128 * wm];
    sa[1] = (int)p[128 * wm + 64];
    sb[0] = (int)p[256 + 64 * wn];
  };
  // Else 4 stages' scales: 16 bytes a row (block g of stage t in byte 4 t + g),
  // of which byte t of a lane's register is stage t's.
  auto read_scales = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < FM; ++i) raw[i] = scales[fa_row + 16 * i];
#pragma unroll
    for (int j = 0; j < 4; ++j) raw[FM + j] = scales[Sb + fb_row + b_step(j)];
  };
  const uint32_t pick = g | (4 + g) << 8;
  auto pack_scales = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < FM + 4; ++i) {
      const uint32_t lo = __builtin_amdgcn_perm((uint32_t)raw[i][1], (uint32_t)raw[i][0], pick);
      const uint32_t hi = __builtin_amdgcn_perm((uint32_t)raw[i][3], (uint32_t)raw[i][2], pick);
      (i < FM ? sa[i < FM ? i : 0] : sb[i < FM ? 0 : i - FM]) = (int)__builtin_amdgcn_perm(hi, lo, 0x05040100u);
    }
  };
  auto mma = [&](auto I, auto R, auto B, auto J) __attribute__((always_inline)) {
    constexpr int i = decltype(R)::value, b = decltype(B)::value, j = decltype(J)::value;
    constexpr int ta = Stay ? i % 4 : decltype(I)::value, tb = Stay ? j : decltype(I)::value;
    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
        fb[j], fa[b], acc[i][j], FP4 ? 4 : 0, 0, tb, sb[Stay ? 0 : j], ta, sa[Stay ? i / 4 : i]);
  };

  // Stay. Stage k in slot I: enters with its B fragments, scales and first two
  // A fragments read; leaves with the next stage's. The slot's parts are
  // refilled with stage k + 2 as soon as all waves have read them: B after the
  // first block row (loads due one and a half stages later), the first four
  // block rows of A after the third, the last four after the sixth (at its
  // end only the next stage's first are due). Loads still in flight at each
  // wait: the 9 (E2M1: 7) of the parts issued since.
  [[maybe_unused]] auto stay_stage = [&](auto I, int k, const Place& now,
                                         const Place& next) __attribute__((always_inline)) {
    constexpr int at = decltype(I)::value;
    using Next = Int<1 - at>;
    auto row = [&](auto R) {
      constexpr int i = decltype(R)::value;
      for_each<4>([&](auto J) { mma(I, R, Int<i % 4>{}, J); });
    };
    auto load = [&](auto Q) { issue_at(I, Q, k + 2, now, next); };
    read_a(I, Int<2>{}, Int<2>{});
    row(Int<0>{});
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(Codes + LS, 0));   // B, its words and A 0 .. 2 are read
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    read_a(I, Int<3>{}, Int<3>{});
    row(Int<1>{});
    for_each<(LB + LS) / 2>([&](auto Q) { load(Int<LA + Q>{}); });
    __builtin_amdgcn_sched_barrier(0);
    read_a(I, Int<0>{}, Int<4>{});
    row(Int<2>{});
    for_each<LB + LS - (LB + LS) / 2>([&](auto Q) { load(Int<LA + (LB + LS) / 2 + Q>{}); });
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(63, 2));           // A 3 is read
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    read_a(I, Int<1>{}, Int<5>{});
    row(Int<3>{});
    load(Int<0>{});
    __builtin_amdgcn_sched_barrier(0);
    read_a(I, Int<2>{}, Int<6>{});
    row(Int<4>{});
    load(Int<2>{});
    __builtin_amdgcn_sched_barrier(0);
    read_a(I, Int<3>{}, Int<7>{});
    row(Int<5>{});
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(Codes + LS, 0));
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    read_a(Next{}, Int<0>{}, Int<0>{});
    read_a(Next{}, Int<1>{}, Int<1>{});
    for_each<4>([&](auto J) {
      mma(I, Int<6>{}, Int<2>{}, J);
      mma(I, Int<7>{}, Int<3>{}, J);
      read_b(Next{}, J);
      if constexpr (J == 1) load(Int<1>{});
      if constexpr (J == 2) load(Int<3>{});
      __builtin_amdgcn_sched_barrier(0);
    });
    read_words(Next{});
  };

  // Stage in slot I: enters with its B fragments and its first two A
  // fragments read; leaves with the next stage's. Fragment i of A sits in
  // buffer (i + Off) % 4.
  [[maybe_unused]] auto stage = [&](auto I, int k, const Place& now,
                                    const Place& next) __attribute__((always_inline)) {
    constexpr int slot_now = decltype(I)::value;
    using Next = Int<(slot_now + 1) % 4>;
    constexpr int Off = (FM * slot_now) % 4;
    for_each<FM - 2>([&](auto R) {
      constexpr int i = decltype(R)::value;
      read_a(I, Int<(i + 2 + Off) % 4>{}, Int<i + 2>{});
      for_each<4>([&](auto J) { mma(I, R, Int<(i + Off) % 4>{}, J); });
      __builtin_amdgcn_sched_barrier(0);
    });
    // All of this slot's reads are in; the next stage's loads of this wave
    // have landed when only the later stages' are in flight. The barrier
    // publishes the next stage and frees this slot.
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(loads_at(slot_now + 3, Codes, LS) + loads_at(slot_now + 2, Codes, LS), 0));
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (slot_now == 3) read_scales();
    read_a(Next{}, Int<(FM + Off) % 4>{}, Int<0>{});
    read_a(Next{}, Int<(FM + 1 + Off) % 4>{}, Int<1>{});
    for_each<4>([&](auto J) {
      constexpr int j = decltype(J)::value;
      mma(I, Int<FM - 2>{}, Int<(FM - 2 + Off) % 4>{}, J);
      mma(I, Int<FM - 1>{}, Int<(FM - 1 + Off) % 4>{}, J);
      read_b(Next{}, J);
      // The freed slot's loads (and the scales' of the next 4 stages) are
      // spread over these MFMAs.
      constexpr int n = loads_at(slot_now, Codes, LS);
      for_each<n*(j + 1) / 4 - n * j / 4>([&](auto Q) { issue_at(I, Int<n * j / 4 + Q>{}, k + 4, now, next); });
      __builtin_amdgcn_sched_barrier(0);
    });
    if constexpr (slot_now == 3) pack_scales();
  };

  int item = item_at(0);
  if (item < 0) return;
  Place now = place(item), next = place(Stay ? item_at(1) : -1);
  [[maybe_unused]] int round = 1;
  for_each<NS>([&](auto I) {
    auto load = [&](auto Q) { issue_at(I, Q, now.k0 + I, now, next); };
    if constexpr (Stay) {
      for_each<LB + LS>([&](auto Q) { load(Int<LA + Q>{}); });
      load(Int<0>{});
      load(Int<2>{});
      load(Int<1>{});
      load(Int<3>{});
    } else {
      for_each<loads_at(decltype(I)::value, Codes, LS)>(load);
    }
  });
  __builtin_amdgcn_s_waitcnt(waitcnt_imm(Stay ? 2 + Codes + LS : 3 * Codes, 15));
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  if constexpr (Stay) {
    read_words(Int<0>{});
  } else {
    read_scales();
    pack_scales();
  }
  read_a(Int<0>{}, Int<0>{}, Int<0>{});
  read_a(Int<0>{}, Int<1>{}, Int<1>{});
  for_each<4>([&](auto J) { read_b(Int<0>{}, J); });

  while (item >= 0) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = v4f{0, 0, 0, 0};
    int k = now.k0;
    if constexpr (Stay) {
      for (; k < now.k1; k += 2) {
        stay_stage(Int<0>{}, k, now, next);
        stay_stage(Int<1>{}, k + 1, now, next);
      }
    } else {
      for (; k + NS <= now.k1; k += NS)
        for_each<NS>([&](auto I) { stage(I, k + I, now, next); });
      for_each<NS - 1>([&](auto I) {
        if (k + I < now.k1) stage(I, k + I, now, next);
      });
    }
    if (t.parts > 1) {
      const int tile = item / t.parts, part = item - tile * t.parts;
      v4f* to = reinterpret_cast<v4f*>(t.partial) +
                (((int64_t)part * t.tiles_m * t.tiles_n + tile) * Waves + wave) * (FM * 4 * 64) + lane;
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) to[64 * (4 * i + j)] = acc[i][j];
    } else {
      wave_epilogue<Gated, FM>(a, acc, (int64_t)now.tm * BM + 16 * FM * wm + r16,
                               Gated ? (int64_t)now.tn * (BN / 2) + 32 * wn + 8 * g
                                     : (int64_t)now.tn * BN + 64 * wn + 16 * g);
    }
    if constexpr (!Stay) break;
    item = item_at(round);
    now = next;
    next = place(item < 0 ? -1 : item_at(++round));
  }
  // No load may be in flight into LDS when the workgroup ends.
  __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));
#endif
}

// Adds the K parts of the tiles in part order and runs the epilogue. A wave
// takes 16 rows (block row i of a tile's wave) by 64 columns.
template <bool Gated>
__global__ void __launch_bounds__(256) linear_parts_kernel(LinearArgs a, TileArgs t, int WM, int WN, int FM) {
  const int lane = threadIdx.x & 63;
  const int waves = WM * WN;
  const int64_t tiles = (int64_t)t.tiles_m * t.tiles_n;
  const int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (id >= tiles * waves * FM) return;
  const int i = (int)(id % FM), wave = (int)(id / FM % waves);
  const int64_t tile = id / FM / waves;
  int tm, tn;
  tile_at((int)tile, t.tiles_m, t.tiles_n, &tm, &tn);
  const v4f* from = reinterpret_cast<const v4f*>(t.partial) + id * (4 * 64) + lane;
  const int64_t step = tiles * waves * FM * (4 * 64);
  v4f acc[1][4];
#pragma unroll
  for (int j = 0; j < 4; ++j) acc[0][j] = v4f{0, 0, 0, 0};
  // Four parts' loads at a time; the sums in part order.
  int p = 0;
  for (; p + 4 <= t.parts; p += 4, from += 4 * step) {
    v4f v[4][4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int j = 0; j < 4; ++j) v[q][j] = from[q * step + 64 * j];
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[0][j] += v[q][j];
  }
  for (; p < t.parts; ++p, from += step)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[0][j] += from[64 * j];
  const int wm = wave / WN, wn = wave % WN, g = lane >> 4;
  wave_epilogue<Gated, 1>(a, acc, (int64_t)tm * (16 * FM * WM) + 16 * (FM * wm + i) + (lane & 15),
                          Gated ? (int64_t)tn * (32 * WN) + 32 * wn + 8 * g
                                : (int64_t)tn * (64 * WN) + 64 * wn + 16 * g);
}

// Scales in the tile kernel's order, what lies past the ends 2^0. By stage
// and 64 rows: [K / 128][groups][block g][r] words, byte i that of row 16 i + r
// of the group, or, for B (kind 1, gated 2), of the row that lane r takes of
// block i (see the top). Else (kind 3) [K / 512][rows] 16 bytes. A thread takes
// 4 rows' 16 bytes of 4 stages, of kind 3 one row's.
__device__ __forceinline__ u32x4 four_stages(const uint8_t* s, int64_t k4, int64_t Ks) {
  u32x4 w = {0, 0, 0, 0};
  if (16 * k4 + 16 <= Ks) {
    __builtin_memcpy(&w, s + 16 * k4, 16);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      w[i / 4] |= (16 * k4 + i < Ks ? (uint32_t)s[16 * k4 + i] : 127u) << (8 * (i % 4));
  }
  return w;
}
struct ScaleOrder {
  const uint8_t* from;
  int64_t ld, rows;          // rows of a part
  uint32_t* to;
  int64_t groups;            // of 64 rows (kind 3: of 16)
};
__global__ void __launch_bounds__(256) scale_order_kernel(ScaleOrder a, ScaleOrder b, int kind_a, int kind_b,
                                                          int64_t Ks, int nk) {
  const int r = threadIdx.x & 15;
  const int64_t k4 = (int64_t)blockIdx.y * 16 + (threadIdx.x >> 4);
  const bool is_a = (int64_t)blockIdx.x < a.groups;
  const ScaleOrder o = is_a ? a : b;
  const int kind = is_a ? kind_a : kind_b;
  const int64_t group = blockIdx.x - (is_a ? 0 : a.groups);
  if (4 * k4 >= nk) return;
  if (kind == 3) {
    const int64_t row = 16 * group + r;
    if (row >= o.rows) return;
    const u32x4 w = four_stages(o.from + row * o.ld, k4, Ks);
    __builtin_memcpy(o.to + 4 * (k4 * o.rows + row), &w, 16);
    return;
  }
  u32x4 w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int q = r >> 2, sub = r & 3;
    int64_t row;
    bool up = false;
    if (kind == 0) {
      row = 64 * group + 16 * i + r;
    } else if (kind == 1) {
      row = 64 * group + 16 * q + 4 * i + sub;
    } else {
      row = 32 * group + 8 * q + 4 * (i & 1) + sub;
      up = i >= 2;
    }
    w[i] = u32x4{0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu};
    if (row < o.rows) w[i] = four_stages(o.from + (row + (up ? o.rows : 0)) * o.ld, k4, Ks);
  }
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    if (4 * k4 + t >= nk) break;
    uint32_t* to = o.to + ((4 * k4 + t) * o.groups + group) * 64 + r;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const uint32_t pick = g | (4 + g) << 8;
      const uint32_t lo = __builtin_amdgcn_perm(w[1][t], w[0][t], pick);
      const uint32_t hi = __builtin_amdgcn_perm(w[3][t], w[2][t], pick);
      to[16 * g] = __builtin_amdgcn_perm(hi, lo, 0x05040100u);
    }
  }
}

constexpr int64_t kMaxExtent = (int64_t{1} << 31) - 16;

// Extent in bytes that a tile's rows of a matrix may reach past its end.
bool extent_ok(int64_t rows, int64_t ld) { return ld < kMaxExtent / 512 && (rows + 512) * ld < kMaxExtent; }

template <bool FP4, bool Gated, int WM, int WN, int FM, int NS>
adahop_status tile_launch(const LinearArgs& a, TileArgs t, hipStream_t stream) {
  constexpr int BM = 16 * FM * WM, BN = (Gated ? 32 : 64) * WN;
  t.tiles_m = (int)((a.m + BM - 1) / BM);
  t.tiles_n = (int)((a.n + BN - 1) / BN);
  const int64_t items = (int64_t)t.tiles_m * t.tiles_n * t.parts;
    // Two slots: one workgroup a compute unit stays.
  const int64_t room = compute_units();
  linear_tile_kernel<FP4, Gated, WM, WN, FM, NS>
      <<<dim3((unsigned)(NS == 2 && items > room ? room : items)), dim3(64 * WM * WN), 0, stream>>>(a, t);
  const adahop_status st = check_launch("linear_mx");
  if (st != ADAHOP_OK || t.parts == 1) return st;
  const int64_t waves = (int64_t)t.tiles_m * t.tiles_n * WM * WN * FM;
  linear_parts_kernel<Gated><<<dim3((unsigned)((waves + 3) / 4)), dim3(256), 0, stream>>>(a, t, WM, WN, FM);
  return check_launch("linear_mx");
}

template <bool FP4, bool Gated>
adahop_status shape_launch(const LinearArgs& a, const TilePlan& p, const TileArgs& t, hipStream_t stream) {
  if (p.shape == kTile256) return tile_launch<FP4, Gated, 2, 4, 8, 2>(a, t, stream);
  if (p.shape == kTile128) return tile_launch<FP4, Gated, 2, 2, 4, 4>(a, t, stream);
  if (p.shape == kTile64) return tile_launch<FP4, Gated, 2, 2, 2, 4>(a, t, stream);
  return tile_launch<FP4, Gated, 1, 2, 2, 4>(a, t, stream);
}

}  // namespace

bool linear_tiles_reach(int64_t rows, int64_t ld) { return extent_ok(rows, ld); }

adahop_status linear_tiles_launch(const LinearArgs& a, int b_fp4, int gated, const TilePlan& p, void* scratch,
                                  hipStream_t stream) {
  const int64_t parts = gated ? 2 : 1, N = parts * a.n, Ks = a.K / 32;
  TileArgs t{};
  t.nk = (int)((a.K + 127) / 128);
  t.parts = p.parts;
  t.a_bytes = (int)((a.m - 1) * a.lda + a.K);
  t.b_bytes = (int)((a.n - 1) * a.ldb + (b_fp4 ? a.K / 2 : a.K));
  const uintptr_t bits = reinterpret_cast<uintptr_t>(a.a_scales) | reinterpret_cast<uintptr_t>(a.b_scales) |
                         (uintptr_t)a.ldas | (uintptr_t)a.ldbs;
  const bool by_stage = p.shape == kTile256;
  // Four stages' scales of a row are read as they are where every row's are
  // whole and aligned.
  if (!by_stage && a.K % 512 == 0 && (bits & 15) == 0 && extent_ok(a.m, a.ldas) && extent_ok(N, a.ldbs)) {
    t.sa = a.a_scales; t.sa_row = (int)a.ldas; t.sa_step = 16;
    t.sa_bytes = (int)((a.m - 1) * a.ldas + Ks);
    t.sb = a.b_scales; t.sb_row = (int)a.ldbs; t.sb_step = 16;
    t.sb_bytes = (int)((N - 1) * a.ldbs + Ks);
  } else {
    const int64_t steps = by_stage ? t.nk : (t.nk + 3) / 4;
    uint8_t* to = static_cast<uint8_t*>(scratch);
    ScaleOrder oa{a.a_scales, a.ldas, a.m, nullptr, 0}, ob{a.b_scales, a.ldbs, by_stage ? a.n : N, nullptr, 0};
    oa.groups = by_stage ? (a.m + 63) / 64 : (a.m + 15) / 16;
    ob.groups = !by_stage ? (N + 15) / 16 : gated ? (a.n + 31) / 32 : (a.n + 63) / 64;
    // Bytes of a step: 256 a group, or 16 a row.
    const int64_t sa = by_stage ? 256 * oa.groups : 16 * a.m, sb = by_stage ? 256 * ob.groups : 16 * N;
    oa.to = reinterpret_cast<uint32_t*>(to);
    ob.to = reinterpret_cast<uint32_t*>(to + steps * sa);
    scale_order_kernel<<<dim3((unsigned)(oa.groups + ob.groups), (unsigned)((t.nk + 63) / 64)), dim3(256), 0,
                         stream>>>(oa, ob, by_stage ? 0 : 3, by_stage ? (gated ? 2 : 1) : 3, Ks, t.nk);
    const adahop_status st = check_launch("linear_mx");
    if (st != ADAHOP_OK) return st;
    t.sa = to; t.sa_row = by_stage ? 4 : 16; t.sa_step = (int)sa; t.sa_bytes = (int)(steps * sa);
    t.sb = to + steps * sa; t.sb_row = t.sa_row; t.sb_step = (int)sb; t.sb_bytes = (int)(steps * sb);
  }
  t.partial = reinterpret_cast<float*>(static_cast<char*>(scratch) + p.scale_bytes);
  if (b_fp4) return gated ? shape_launch<true, true>(a, p, t, stream) : shape_launch<true, false>(a, p, t, stream);
  return gated ? shape_launch<false, true>(a, p, t, stream) : shape_launch<false, false>(a, p, t, stream);
}

}  // namespace adahop
