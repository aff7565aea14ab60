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
constexpr int kGroupM = 8;                 // tile rows that run together on one XCD

struct TileArgs {
  const uint8_t* sa;         // scale words (4 blocks of a row): row and stage
  const uint8_t* sb;         // strides in bytes
  int sa_row, sa_stage, sb_row, sb_stage;
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

template <bool FP4, int BM, int BN>
struct Slot {
  uint32_t sc[BM + BN > 256 ? 512 : 256];   // A's scale words, then B's
  uint8_t a[BM * 128];
  uint8_t b[BN * (FP4 ? 64 : 128)];
};

template <bool FP4, bool Gated, int WM, int WN, int FM, int NS>
__global__ void __launch_bounds__(64 * WM * WN, 1) linear_tile_kernel(LinearArgs a, TileArgs t) {
  constexpr int Waves = WM * WN, BM = 16 * FM * WM, BN = 64 * WN;
  constexpr int Bb = FP4 ? 64 : 128;                   // bytes of a B row and stage
  constexpr int Ra = 8 * Waves, Rb = (FP4 ? 16 : 8) * Waves;   // rows a load of every wave fills
  constexpr int LA = BM / Ra, LB = BN / Rb;            // loads of a wave and stage
  constexpr int Loads = LA + LB + 1;                   // and one of scale words
  // Two slots: workgroups stay, and load the next tile's first stages during a
  // tile's last ones and its epilogue; a tile takes an even number of stages
  // (one of zeros follows an odd number), so that each begins in slot 0. Four
  // slots: one tile a workgroup.
  constexpr bool Stay = NS == 2;
  constexpr int Unit = Stay ? 2 : 1;
  static_assert(BM % Ra == 0 && BN % Rb == 0 && BM + BN <= 64 * Waves && NS % 2 == 0, "");
  using S = Slot<FP4, BM, BN>;
  // One LDS object a slot: alias analysis then sees that loads into one slot
  // do not touch the one being read, and adds no wait before the reads.
  __shared__ __attribute__((aligned(1024))) S s0;
  __shared__ __attribute__((aligned(1024))) S s1;
  __shared__ __attribute__((aligned(1024))) S s2;
  __shared__ __attribute__((aligned(1024))) S s3;
  auto slot = [&](auto I) -> S& {
    if constexpr (I == 0) return s0;
    else if constexpr (I == 1) return s1;
    else if constexpr (I == 2) return s2;
    else return s3;
  };

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int r16 = lane & 15, g = lane >> 4;
  const int items = t.tiles_m * t.tiles_n * t.parts;

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
  const bool sc_is_a = 64 * wave < BM;
  const __amdgpu_buffer_rsrc_t rb_s = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(sc_is_a ? t.sa : t.sb), 0, sc_is_a ? t.sa_bytes : t.sb_bytes, kBufferFlags);
  const int sc_stage = sc_is_a ? t.sa_stage : t.sb_stage;
  const int ra = 8 * wave + (lane >> 3);                     // A row of load 0; + Ra j
  const int ca = (lane & 7) ^ ((ra >> 1) & 7);               // logical chunk (the same for every j)
  const int rb = (FP4 ? 16 : 8) * wave + (lane >> (FP4 ? 2 : 3));
  // XOR key of B row r: q and s as in the fragments' row order.
  const int qb = (rb >> (Gated ? 3 : 4)) & 3;
  const int cb = FP4 ? (lane & 3) ^ qb : (lane & 7) ^ (2 * qb + ((rb >> 1) & 1));
  static_assert(Ra % 16 == 0 && Rb % 32 == 0, "A's key is the same for every load");
  // A load's address is this lane's offset within a tile (below), plus the
  // tile's and the load's rows, scalar. A 64-row slice of B holds, gated, 32
  // gate and 32 up rows of 32 columns.
  const uint32_t oa = (uint32_t)ra * (uint32_t)a.lda + 16 * ca;
  const uint32_t ob = (uint32_t)(Gated ? (rb >> 6) * 32 + (rb & 31) : rb) * (uint32_t)a.ldb;
  const int rs = 64 * wave + lane - (sc_is_a ? 0 : BM);      // row of the scale words
  const bool no_scale = !sc_is_a && rs >= BN;
  const uint32_t os = (uint32_t)(Gated && !sc_is_a ? (rs >> 6) * 32 + (rs & 31) + ((rs >> 5) & 1) * (int)a.n : rs) *
                      (uint32_t)(sc_is_a ? t.sa_row : t.sb_row);

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
    *k1 = __builtin_amdgcn_readfirstlane(Unit * (int)(units * (part + 1) / t.parts));
  };
  // An item's place, all scalar.
  struct Place {
    int tm, tn, k0, k1;
    uint32_t a, b, s;
  };
  // Without an item: a stage past the end of any K.
  auto place = [&](int item) {
    Place p{0, 0, 1 << 23, 1 << 24, 0, 0, 0};
    if (item < 0) return p;
    locate(item, &p.tm, &p.tn, &p.k0, &p.k1);
    p.a = (uint32_t)(p.tm * BM) * (uint32_t)a.lda;
    p.b = (uint32_t)(p.tn * (Gated ? BN / 2 : BN)) * (uint32_t)a.ldb;
    p.s = sc_is_a ? (uint32_t)(p.tm * BM) * (uint32_t)t.sa_row
                  : (uint32_t)(p.tn * (Gated ? BN / 2 : BN)) * (uint32_t)t.sb_row;
    return p;
  };
  // Load q of stage k of an item into slot I. Chunks past the end of K are
  // zeros, for both operands; a stage past it must not have NaN scales.
  auto issue = [&](auto I, auto Q, int k, uint32_t base_a, uint32_t base_b, uint32_t base_s) {
    constexpr int q = decltype(Q)::value;
    S& s = slot(I);
    // The scalar offset stays inside the buffers (the range check may
    // subtract it from their size).
    const int kt = k < t.nk ? k : 0;
    if constexpr (q < LA) {
      const uint32_t v = 128 * k + 16 * ca < (int)a.K ? oa : kPastEnd;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb_a, (lds_void*)&s.a[1024 * (Waves * q + wave)], 16,
                                               (int)(v + (base_a + q * Ra * (uint32_t)a.lda)), 128 * kt, 0, 0);
    } else if constexpr (q < LA + LB) {
      constexpr int j = q - LA;
      // Loads 32 rows apart alternate bit 5 of the row, which enters the key.
      const int c = !FP4 && !Gated && Rb == 32 ? cb ^ (4 * (j & 1)) : cb;
      const uint32_t v = Bb * k + 16 * c < (int)(FP4 ? a.K / 2 : a.K) ? ob + 16 * c : kPastEnd;
      // Rows of B from one load to the next: Rb, of which gated a half each
      // gate and up rows.
      constexpr int step = !Gated ? Rb * j : Rb >= 64 ? Rb * j / 2 : 32 * (Rb * j / 64) + (Rb * j) % 32;
      const __amdgpu_buffer_rsrc_t r = Gated && Rb < 64 && ((Rb * j) >> 5) % 2 == 1 ? rb_b1 : rb_b0;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)&s.b[1024 * (Waves * j + wave)], 16,
                                               (int)(v + (base_b + step * (uint32_t)a.ldb)), Bb * kt, 0, 0);
    } else {
      const uint32_t v = k < t.nk && !no_scale ? os : kPastEnd;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb_s, (lds_void*)&s.sc[64 * wave], 4, (int)(v + base_s),
                                               kt * sc_stage, 0, 0);
    }
  };
  // Stage k of item `now`, or, past its last, of item `next`: the scalar
  // selects keep the stages free of branches.
  auto issue_at = [&](auto I, auto Q, int k, const Place& now, const Place& next) {
    const bool in = k < now.k1;
    issue(I, Q, in ? k : k - now.k1 + next.k0, in ? now.a : next.a, in ? now.b : next.b, in ? now.s : next.s);
  };

  // ---- fragments ------------------------------------------------------------
  const int q4 = r16 >> 2, s4 = r16 & 3;
  const int fa_row = 16 * FM * wm + r16;
  const int fa_lo = fa_row * 128 + 16 * (g ^ ((r16 >> 1) & 7));
  const int fb_row = 64 * wn + (Gated ? 8 : 16) * q4 + s4;
  const int fb_lo = fb_row * Bb + 16 * (FP4 ? g ^ q4 : g ^ (2 * q4 + (s4 >> 1)));
  auto b_step = [](int j) { return Gated ? 32 * (j >> 1) + 4 * (j & 1) : 4 * j; };

  v4f acc[FM][4];
  v8i fa[4], fb[4];
  int sa[4], sb[4];
  auto read_a = [&](auto I, auto B, int i) {
    constexpr int b = decltype(B)::value;
    const S& s = slot(I);
    const v4i lo = *reinterpret_cast<const v4i*>(&s.a[fa_lo + 2048 * i]);
    const v4i hi = *reinterpret_cast<const v4i*>(&s.a[(fa_lo ^ 64) + 2048 * i]);
    fa[b] = v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    sa[b] = reinterpret_cast<const uint8_t*>(s.sc)[4 * (fa_row + 16 * i) + g];
  };
  auto read_b = [&](auto I, auto J) {
    constexpr int j = decltype(J)::value;
    const S& s = slot(I);
    const v4i lo = *reinterpret_cast<const v4i*>(&s.b[fb_lo + Bb * b_step(j)]);
    if constexpr (FP4) {
      fb[j] = v8i{lo[0], lo[1], lo[2], lo[3], 0, 0, 0, 0};
    } else {
      const v4i hi = *reinterpret_cast<const v4i*>(&s.b[(fb_lo ^ 64) + Bb * b_step(j)]);
      fb[j] = v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    }
    sb[j] = reinterpret_cast<const uint8_t*>(s.sc)[4 * (BM + fb_row + b_step(j)) + g];
  };
  auto mma = [&](int i, int b, int j) {
    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb[j], fa[b], acc[i][j], FP4 ? 4 : 0, 0, 0,
                                                                 sb[j], 0, sa[b]);
  };

  // Stage in slot I: enters with its B fragments and its first two A
  // fragments read; leaves with the next stage's. Fragment i of A sits in
  // buffer (i + Off) % 4.
  auto stage = [&](auto I, int k, const Place& now, const Place& next) {
    constexpr int slot_now = decltype(I)::value, slot_next = (slot_now + 1) % NS;
    constexpr int Off = (FM * slot_now) % 4;
    for_each<FM - 2>([&](auto R) {
      constexpr int i = decltype(R)::value;
      read_a(I, Int<(i + 2 + Off) % 4>{}, i + 2);
#pragma unroll
      for (int j = 0; j < 4; ++j) mma(i, (i + Off) % 4, j);
      __builtin_amdgcn_sched_barrier(0);
    });
    // All of this slot's reads are in; the next stage's loads of this wave
    // have landed when only the later stages' are in flight. The barrier
    // publishes the next stage and frees this slot.
    __builtin_amdgcn_s_waitcnt(waitcnt_imm((NS - 2) * Loads, 0));
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    read_a(Int<slot_next>{}, Int<(FM + Off) % 4>{}, 0);
    read_a(Int<slot_next>{}, Int<(FM + 1 + Off) % 4>{}, 1);
    for_each<4>([&](auto J) {
      constexpr int j = decltype(J)::value;
      mma(FM - 2, (FM - 2 + Off) % 4, J);
      mma(FM - 1, (FM - 1 + Off) % 4, J);
      read_b(Int<slot_next>{}, J);
      // The freed slot's loads are spread over these MFMAs.
      for_each<Loads*(j + 1) / 4 - Loads * j / 4>(
          [&](auto Q) { issue_at(I, Int<Loads * j / 4 + Q>{}, k + NS, now, next); });
      __builtin_amdgcn_sched_barrier(0);
    });
  };

  int item = item_at(0);
  if (item < 0) return;
  Place now = place(item), next = place(Stay ? item_at(1) : -1);
  [[maybe_unused]] int round = 1;
  for_each<NS>([&](auto I) {
    for_each<Loads>([&](auto Q) { issue_at(I, Q, now.k0 + I, now, next); });
  });
  __builtin_amdgcn_s_waitcnt(waitcnt_imm((NS - 1) * Loads, 15));
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  read_a(Int<0>{}, Int<0>{}, 0);
  read_a(Int<0>{}, Int<1>{}, 1);
  for_each<4>([&](auto J) { read_b(Int<0>{}, J); });

  while (item >= 0) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = v4f{0, 0, 0, 0};
    int k = now.k0;
    if constexpr (Stay) {
      for (; k < now.k1; k += 2) {
        stage(Int<0>{}, k, now, next);
        stage(Int<1>{}, k + 1, now, next);
      }
    } else {
      for (; k + 4 <= now.k1; k += 4) {
        stage(Int<0>{}, k, now, next);
        stage(Int<1>{}, k + 1, now, next);
        stage(Int<2>{}, k + 2, now, next);
        stage(Int<3>{}, k + 3, now, next);
      }
      if (k < now.k1) stage(Int<0>{}, k, now, next);
      if (k + 1 < now.k1) stage(Int<1>{}, k + 1, now, next);
      if (k + 2 < now.k1) stage(Int<2>{}, k + 2, now, next);
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
  v4f acc[1][4];
#pragma unroll
  for (int j = 0; j < 4; ++j) acc[0][j] = from[64 * j];
  for (int p = 1; p < t.parts; ++p) {
    from += tiles * waves * FM * (4 * 64);
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[0][j] += from[64 * j];
  }
  const int wm = wave / WN, wn = wave % WN, g = lane >> 4;
  wave_epilogue<Gated, 1>(a, acc, (int64_t)tm * (16 * FM * WM) + 16 * (FM * wm + i) + (lane & 15),
                          Gated ? (int64_t)tn * (32 * WN) + 32 * wn + 8 * g
                                : (int64_t)tn * (64 * WN) + 64 * wn + 16 * g);
}

// Scale words by stage, [K / 128 rounded up][rows], bytes past the end of K 2^0.
__global__ void __launch_bounds__(256) scale_words_kernel(const uint8_t* a, int64_t lda, int64_t rows_a,
                                                          uint32_t* to_a, const uint8_t* b, int64_t ldb,
                                                          int64_t rows_b, uint32_t* to_b, int64_t Ks,
                                                          int nk) {
  // 64 rows by 4 stages a workgroup; consecutive threads write consecutive rows.
  const int64_t r = (int64_t)blockIdx.x * 64 + (threadIdx.x & 63);
  const int kt = blockIdx.y * 4 + (threadIdx.x >> 6);
  const bool is_a = r < rows_a;
  const int64_t row = is_a ? r : r - rows_a;
  if (row >= (is_a ? rows_a : rows_b) || kt >= nk) return;
  const uint8_t* s = (is_a ? a + row * lda : b + row * ldb) + 4 * (int64_t)kt;
  uint32_t w = 0;
  if (4 * (int64_t)kt + 4 <= Ks) {
    __builtin_memcpy(&w, s, 4);
  } else {
    for (int i = 0; i < 4; ++i) w |= (4 * (int64_t)kt + i < Ks ? (uint32_t)s[i] : 127u) << (8 * i);
  }
  (is_a ? to_a + (int64_t)kt * rows_a : to_b + (int64_t)kt * rows_b)[row] = w;
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
  const size_t lds = NS * sizeof(Slot<FP4, BM, 64 * WN>);
  const int64_t room = (int64_t)device_cus() * (int64_t)(160 * 1024 / lds);
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
  return tile_launch<FP4, Gated, 2, 2, 2, 4>(a, t, stream);
}

}  // namespace

bool linear_tiles_reach(int64_t rows, int64_t ld) { return extent_ok(rows, ld); }

TilePlan linear_tile_plan(int64_t m, int64_t n, int64_t K, int b_fp4, int gated) {
  TilePlan p{};
  (void)b_fp4;
  const int64_t N = gated ? 2 * n : n;
  const int64_t nk = (K + 127) / 128;
  auto tiles = [&](int64_t bm, int64_t bn) { return ((m + bm - 1) / bm) * ((N + bn - 1) / bn); };
  p.parts = 1;
  if (tiles(256, 256) >= 192) p.shape = kTile256;
  else if (tiles(128, 128) >= 128) p.shape = kTile128;
  else p.shape = kTile64;
  p.scale_bytes = (size_t)(nk * 4 * (m + N) + 15) / 16 * 16;
  return p;
}

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
  if (a.K % 128 == 0 && (bits & 3) == 0 && extent_ok(a.m, a.ldas) &&
      extent_ok(gated ? a.n + a.n : a.n, a.ldbs)) {
    t.sa = a.a_scales; t.sa_row = (int)a.ldas; t.sa_stage = 4;
    t.sa_bytes = (int)((a.m - 1) * a.ldas + Ks);
    t.sb = a.b_scales; t.sb_row = (int)a.ldbs; t.sb_stage = 4;
    t.sb_bytes = (int)(((gated ? a.n : 0) + a.n - 1) * a.ldbs + Ks);
  } else {
    uint32_t* wa = static_cast<uint32_t*>(scratch);
    uint32_t* wb = wa + t.nk * a.m;
    scale_words_kernel<<<dim3((unsigned)((a.m + N + 63) / 64), (unsigned)((t.nk + 3) / 4)), dim3(256), 0,
                         stream>>>(a.a_scales, a.ldas, a.m, wa, a.b_scales, a.ldbs, N, wb, Ks, t.nk);
    const adahop_status st = check_launch("linear_mx");
    if (st != ADAHOP_OK) return st;
    t.sa = reinterpret_cast<const uint8_t*>(wa); t.sa_row = 4; t.sa_stage = (int)(4 * a.m);
    t.sa_bytes = (int)(4 * a.m * t.nk);
    t.sb = reinterpret_cast<const uint8_t*>(wb); t.sb_row = 4; t.sb_stage = (int)(4 * N);
    t.sb_bytes = (int)(4 * N * t.nk);
  }
  t.partial = reinterpret_cast<float*>(static_cast<char*>(scratch) + p.scale_bytes);
  if (b_fp4) return gated ? shape_launch<true, true>(a, p, t, stream) : shape_launch<true, false>(a, p, t, stream);
  return gated ? shape_launch<false, true>(a, p, t, stream) : shape_launch<false, false>(a, p, t, stream);
}

}  // namespace adahop
