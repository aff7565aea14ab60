// Products of bf16 operands in 256 x 256 tiles fed through LDS, with an
// epilogue of the caller's (gfx950): C[i, j] = sum_k A(i, k) B(j, k) in fp32.
//
// An operand lies along K ([rows][K], row-major) or across it ([K][rows]); B
// may also be MXFP8 codes and scales across K, widened to bf16 on their way into
// LDS. Any sizes; K of an operand along it in 16-byte chunks, rows of one
// across it too (the caller checks).
//
// A workgroup of 8 waves, two a SIMD, computes a tile, a wave 128 x 64 of it as
// 8 x 4 blocks of v_mfma_f32_16x16x32_bf16 (B first, so that a lane holds four
// neighbouring columns of a row). K advances 64 elements a stage through two
// LDS slots of 64 KB. A slot's parts are refilled with the stage after next as
// soon as all waves have read them: B after the first block row, A's halves
// after the fourth and the last, so that every load has more than a stage of
// time. Workgroups stay: the next tile's first stages are loaded during a tile's
// last ones and its epilogue.
//
// LDS of an operand along K: rows of 128 bytes, the 16-byte chunks XORed with
// row bits so that the 16 rows which a quarter of a wave reads at one chunk lie
// in different banks. B's rows are permuted: row r = 4 q + s of block j is B row
// 16 q + 4 j + s of the wave's 64, so a lane's four blocks hold 16 neighbouring
// columns of C.
// LDS of one across K: K-rows of 256 (a half of A) or 512 bytes (B), read with
// ds_read_b64_tr_b16: lane i of 16 receives element i of four K-rows whose 16
// elements (32 bytes) the lanes 4 t .. 4 t + 3 address. The 32-byte groups of
// K-row k are XORed with h(k) = k % 4 + 4 (k / 8 % 2): the 8 K-rows that half a
// wave reads lie in 8 different groups. A lane's block j then holds columns
// 16 j + 4 g .. +3 of the wave's 64 (g = lane / 16).
#pragma once

#include <type_traits>
#include <utility>

#include "adahop_internal.h"
#include "mx8_common.h"

namespace adahop {
namespace tiles {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v2i __attribute__((ext_vector_type(2)));
typedef short v4s16 __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) v4s16 lds_v4s16;

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
// An offset past the end of every buffer here (256 rows, each less than
// kMaxRowBytes from the next): such a load returns 0 without touching memory.
constexpr int kPastEnd = 0x7FFFFFF0;
constexpr int64_t kMaxRowBytes = int64_t{1} << 23;

constexpr int kTile = 256;                 // rows and columns of a tile
constexpr int kStageK = 64;                // K elements of a stage
constexpr int kThreads = 512;
constexpr int kGroupM = 4;                 // tile rows that run together on one XCD

// How an operand lies: along K, across it, or across it in MXFP8 (B alone).
enum Kind { kAlong = 0, kAcross = 1, kCodes = 2 };

struct Operand {
  const uint8_t* p;
  int64_t ld;                // bytes from a row to the next
  const uint8_t* scales;     // kCodes: a byte per 32 columns
  int64_t ld_scales;
};

struct TileArgs {
  Operand a, b;
  int64_t m, n, K;
  int tiles_m, tiles_n;
  int units;                 // pairs of stages of K
  // Items 0 .. full - 1 are whole tiles; those after them each one of `parts`
  // parts of K of a tile, whose sums go to split_ws ([tile][part][256][256]).
  int full, split, parts;
  float* split_ws;
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

// What an epilogue is told of the wave's accumulators: acc[i][j][e] is row
// row0 + 16 i, column col0 + (BK == kAlong ? 4 j : 16 j) + e.
struct Spot {
  int64_t row0, col0;
  int tn, wn;                // tile column, wave column
  int part;                  // < 0: a whole tile
  float* to;                 // of a part: its 256 x 256 sums
  int lrow, lcol;            // row and column in the tile
};

struct Half {
  uint8_t a[128 * 128];
};
struct Wide {
  uint8_t b[256 * 128];
};

template <Kind AK, Kind BK, typename Epi>
__global__ void __launch_bounds__(kThreads, 1) bf16_tile_kernel(TileArgs t, Epi epi) {
#ifdef __HIP_DEVICE_COMPILE__                        // the host pass needs the launch stub alone
  constexpr int Loads = 8;                           // of a wave and stage: 4 of A, 4 of B
  // One LDS object for each part that is filled at once: alias analysis then
  // sees that loads into one do not touch another, and adds no wait before
  // the reads.
  __shared__ __attribute__((aligned(1024))) Half f0, f1, r0, r1;   // first and last 64 rows of a wave
  __shared__ __attribute__((aligned(1024))) Wide w0, w1;
  auto half = [&](auto I, auto H) -> Half& {
    if constexpr (I == 0 && H == 0) return f0;
    else if constexpr (I == 0) return r0;
    else if constexpr (H == 0) return f1;
    else return r1;
  };
  auto wide = [&](auto I) -> Wide& {
    if constexpr (I == 0) return w0;
    else return w1;
  };

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int r16 = lane & 15, g = lane >> 4;
  const int items = t.full + t.split * t.parts;

  // ---- items ----------------------------------------------------------------
  auto item_at = [&](int round) {
    const int G = gridDim.x, base = round * G;
    if (base >= items) return -1;
    const int cnt = items - base < G ? items - base : G;
    return (int)blockIdx.x < cnt ? base + xcd_band(blockIdx.x, cnt) : -1;
  };
  // An item's place, all scalar. Stages k0 .. k1 - 1, an even number; a / b: the
  // tile's first byte at k = 0, a_bytes / b_bytes: bytes from there to the end
  // of the tile's rows (across K: of one K-row).
  struct Place {
    int tm, tn, k0, k1, part, split_tile;
    const uint8_t* a;
    const uint8_t* b;
    const uint8_t* scales;
    int a_bytes, b_bytes;
  };
  // Bytes of the 16-byte chunks that hold n elements.
  auto chunks = [](int64_t n) { return 2 * ((n + 7) & ~(int64_t)7); };
  auto place = [&](int item) {
    // Without an item: a stage past the end of any K.
    Place p{0, 0, 1 << 28, 1 << 28, -1, 0, t.a.p, t.b.p, t.b.scales, 0, 0};
    if (item < 0) return p;
    int tile = item, part = -1;
    if (item >= t.full) {
      const int s = item - t.full;
      p.split_tile = __builtin_amdgcn_readfirstlane(s / t.parts);
      tile = t.full + p.split_tile;
      part = s - p.split_tile * t.parts;
    }
    int m_, n_;
    tile_at(tile, t.tiles_m, t.tiles_n, &m_, &n_);
    p.tm = __builtin_amdgcn_readfirstlane(m_);
    p.tn = __builtin_amdgcn_readfirstlane(n_);
    p.part = __builtin_amdgcn_readfirstlane(part);
    p.k0 = 0;
    p.k1 = 2 * t.units;
    if (p.part >= 0) {
      p.k0 = 2 * __builtin_amdgcn_readfirstlane((int)((int64_t)t.units * p.part / t.parts));
      p.k1 = 2 * __builtin_amdgcn_readfirstlane((int)((int64_t)t.units * (p.part + 1) / t.parts));
    }
    const int64_t m0 = (int64_t)p.tm * kTile, n0 = (int64_t)p.tn * kTile;
    if constexpr (AK == kAlong) {
      const int64_t rows = t.m - m0 < kTile ? t.m - m0 : kTile;
      p.a = t.a.p + m0 * t.a.ld;
      p.a_bytes = (int)((rows - 1) * t.a.ld + chunks(t.K));
    } else {
      p.a = t.a.p + 2 * m0;
      p.a_bytes = (int)chunks(t.m - m0 < kTile ? t.m - m0 : kTile);
    }
    if constexpr (BK == kAlong) {
      const int64_t rows = t.n - n0 < kTile ? t.n - n0 : kTile;
      p.b = t.b.p + n0 * t.b.ld;
      p.b_bytes = (int)((rows - 1) * t.b.ld + chunks(t.K));
    } else if constexpr (BK == kAcross) {
      p.b = t.b.p + 2 * n0;
      p.b_bytes = (int)chunks(t.n - n0 < kTile ? t.n - n0 : kTile);
    } else {
      p.b = t.b.p + n0;
      p.scales = t.b.scales + n0 / 32;
      p.b_bytes = (int)(t.n - n0 < kTile ? t.n - n0 : kTile);   // a multiple of 32
    }
    return p;
  };

  // ---- loads: this wave's share of a stage ------------------------------------
  // The descriptor starts at stage k's first byte and ends with its last, so
  // that rows and K-rows past the ends read as 0. `left`: elements of K from
  // the stage's first.
  struct Source {
    __amdgpu_buffer_rsrc_t a, b, scales;
    int left;
  };
  auto source_of = [&](Kind kind, const uint8_t* p, int bytes, int64_t ld, int k, int left) {
    if (kind == kAlong) {
      const int64_t at = (int64_t)128 * k;
      return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p + at), 0,
                                               left > 0 ? bytes - 128 * k : 0, kBufferFlags);
    }
    const int rows = left < kStageK ? left : kStageK;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p + (int64_t)kStageK * k * ld), 0,
                                             rows > 0 ? (rows - 1) * (int)ld + bytes : 0, kBufferFlags);
  };
  // Stage k of item `now`, or, past its last, of item `next`: the scalar
  // selects keep the stages free of branches.
  auto source = [&](int k, const Place& now, const Place& next) __attribute__((always_inline)) {
    const bool in = k < now.k1;
    const int at = in ? k : k - now.k1 + next.k0;
    const int64_t rest = t.K - (int64_t)kStageK * at;
    const int left = (int)(rest < 0 ? 0 : rest < kStageK ? rest : kStageK);
    const int kk = left > 0 ? at : 0;
    Source s;
    s.left = left;
    s.a = source_of(AK, in ? now.a : next.a, in ? now.a_bytes : next.a_bytes, t.a.ld, kk, left);
    s.b = source_of(BK, in ? now.b : next.b, in ? now.b_bytes : next.b_bytes, t.b.ld, kk, left);
    if constexpr (BK == kCodes)
      s.scales = source_of(BK, in ? now.scales : next.scales, (in ? now.b_bytes : next.b_bytes) / 32, t.b.ld_scales,
                           kk, left);
    return s;
  };
  // Along K, load q of this wave fills rows 64 q + 8 wave + lane / 8 with chunks
  // XORed as they are read; across, K-rows (A) 32 (q / 2) + 4 wave + lane / 16 of
  // half q % 2, (B) 16 q + 2 wave + lane / 32.
  const int row8 = 8 * wave + (lane >> 3);
  const int ca = (lane & 7) ^ ((row8 >> 1) & 7);
  const int cb = (lane & 7) ^ (2 * ((row8 >> 4) & 3) + ((row8 >> 1) & 1));
  const int ka = 4 * wave + (lane >> 4), kb = 2 * wave + (lane >> 5);
  const int ga = ((lane & 15) >> 1) ^ ((ka & 3) + 4 * ((ka >> 3) & 1));
  const int gb0 = ((lane & 31) >> 1) ^ ((kb & 3) + 4 * ((kb >> 3) & 1));
  const int oa = AK == kAlong ? row8 * (int)t.a.ld + 16 * ca
                              : ka * (int)t.a.ld + 256 * (ga >> 2) + 32 * (ga & 3) + 16 * (lane & 1);
  // Codes: two runs of 16 of a stage a thread, K-rows 32 u + thread / 16.
  const int kc = threadIdx.x >> 4, gc = threadIdx.x & 15;
  const int ob = BK == kCodes ? kc * (int)t.b.ld + 16 * gc : BK == kAlong ? row8 * (int)t.b.ld + 16 * cb : kb * (int)t.b.ld + 32 * gb0 + 16 * (lane & 1);
  // Codes of the stage after the next but one, loaded a stage ahead of their
  // widening into the slot that the stage before them frees.
  v4i codes[2];
  uint8_t scale[2];
  const int oc = kc * 512 + 32 * (gc ^ ((kc & 3) + 4 * ((kc >> 3) & 1)));
  auto widen = [&](auto I) __attribute__((always_inline)) {
    for_each<2>([&](auto U) {
      const float by = mx8::mx8_scale(scale[U]);
      v4i w[2];
      for_each<4>([&](auto D) {
        constexpr int d = decltype(D)::value;
        const int four = codes[U][d];
        const auto lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)four, by, false);
        const auto hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)four, by, true);
        w[d / 2][2 * (d % 2)] = __builtin_bit_cast(int, lo);
        w[d / 2][2 * (d % 2) + 1] = __builtin_bit_cast(int, hi);
      });
      v4i* to = reinterpret_cast<v4i*>(wide(I).b + oc + 16384 * decltype(U)::value);
      to[0] = w[0];
      to[1] = w[1];
    });
  };
  // Across K, a row's last bytes are followed by the next row's: columns past
  // the tile's end reach only sums that are not stored.
  auto issue = [&](auto I, auto Q, const Source& s) __attribute__((always_inline)) {
    constexpr int q = decltype(Q)::value;
    if constexpr (q < 4) {
      int v;
      if constexpr (AK == kAlong) v = 8 * ca < s.left ? oa + 64 * q * (int)t.a.ld : kPastEnd;
      else v = oa + 32 * (q / 2) * (int)t.a.ld + 128 * (q % 2);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(s.a, (lds_void*)&half(I, Int<q % 2>{}).a[1024 * (8 * (q / 2) + wave)],
                                               16, v, 0, 0, 0);
    } else if constexpr (BK == kCodes) {
      constexpr int u = (q - 4) / 2;
      if constexpr (q % 2 == 0)
        codes[u] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(s.b, ob + 32 * u * (int)t.b.ld, 0, 0));
      else
        scale[u] = __builtin_amdgcn_raw_buffer_load_b8(s.scales, (kc + 32 * u) * (int)t.b.ld_scales + gc / 2, 0, 0);
    } else {
      constexpr int j = q - 4;
      int v;
      if constexpr (BK == kAlong) {
        v = 8 * cb < s.left ? ob + 64 * j * (int)t.b.ld : kPastEnd;
      } else {
        v = ob + 16 * j * (int)t.b.ld;
      }
      __builtin_amdgcn_raw_ptr_buffer_load_lds(s.b, (lds_void*)&wide(I).b[1024 * (8 * j + wave)], 16, v, 0, 0, 0);
    }
  };

  // ---- fragments --------------------------------------------------------------
  const int q4 = r16 >> 2, sub = r16 & 3;
  const int hk = q4 + 4 * (g & 1);                   // h(k) of this lane's K-rows
  const int fa = AK == kAlong ? (64 * wm + r16) * 128 + 16 * (g ^ ((r16 >> 1) & 7))
                              : (8 * g + q4) * 256 + 8 * sub;
  const int fb = BK == kAlong ? (64 * wn + 16 * q4 + sub) * 128 + 16 * (g ^ (2 * q4 + (sub >> 1)))
                              : (8 * g + q4) * 512 + 8 * sub;
  int xa[4], xb[4];                                  // across K: the groups of the blocks
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    xa[i] = fa + 32 * ((4 * wm + i) ^ hk);
    xb[i] = fb + 32 * ((4 * wn + i) ^ hk);
  }
  v4f acc[8][4];
  v4i A[4][2], B[4][2];
  auto tr = [](const uint8_t* p, int next) __attribute__((always_inline)) {
    const v2i lo = __builtin_bit_cast(v2i, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s16*)p));
    const v2i hi = __builtin_bit_cast(v2i, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s16*)(p + next)));
    return v4i{lo[0], lo[1], hi[0], hi[1]};
  };
  auto read_a = [&](auto I, auto Buf, auto R) __attribute__((always_inline)) {
    constexpr int b = decltype(Buf)::value, i = decltype(R)::value;
    const uint8_t* p = half(I, Int<i / 4>{}).a;
    if constexpr (AK == kAlong) {
      A[b][0] = *reinterpret_cast<const v4i*>(p + 2048 * (i % 4) + fa);
      A[b][1] = *reinterpret_cast<const v4i*>(p + 2048 * (i % 4) + (fa ^ 64));
    } else {
      A[b][0] = tr(p + xa[i % 4], 1024);
      A[b][1] = tr(p + xa[i % 4] + 8192, 1024);
    }
  };
  auto read_b = [&](auto I, auto J) __attribute__((always_inline)) {
    constexpr int j = decltype(J)::value;
    const uint8_t* p = wide(I).b;
    if constexpr (BK == kAlong) {
      B[j][0] = *reinterpret_cast<const v4i*>(p + 512 * j + fb);
      B[j][1] = *reinterpret_cast<const v4i*>(p + 512 * j + (fb ^ 64));
    } else {
      B[j][0] = tr(p + xb[j], 2048);
      B[j][1] = tr(p + xb[j] + 16384, 2048);
    }
  };
  auto mma = [&](auto R, auto Buf, auto S, auto J) __attribute__((always_inline)) {
    constexpr int i = decltype(R)::value, b = decltype(Buf)::value, s = decltype(S)::value, j = decltype(J)::value;
    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, B[j][s]),
                                                        __builtin_bit_cast(v8bf, A[b][s]), acc[i][j], 0, 0, 0);
  };
  auto row = [&](auto R) __attribute__((always_inline)) {
    for_each<2>([&](auto S) {
      for_each<4>([&](auto J) { mma(R, Int<decltype(R)::value % 4>{}, S, J); });
    });
  };
  constexpr int ReadsA = AK == kAlong ? 2 : 4;       // LDS reads of a block row's fragments

  // Stage k in slot I: enters with its B fragments and first two A fragments
  // read; leaves with the next stage's. Loads still in flight at the first and
  // the last wait: the 8 issued since those of the parts that are due.
  auto stage = [&](auto I, int k, const Place& now, const Place& next) __attribute__((always_inline)) {
    using Next = Int<1 - decltype(I)::value>;
    const Source s = source(k + 2, now, next);
    const Source sb = BK == kCodes ? source(k + 3, now, next) : s;
    read_a(I, Int<2>{}, Int<2>{});
    row(Int<0>{});
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(Loads, 0));         // B and A 0 .. 2 are read
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    read_a(I, Int<3>{}, Int<3>{});
    row(Int<1>{});
    if constexpr (BK == kCodes) widen(I);
    issue(I, Int<4>{}, sb);
    issue(I, Int<5>{}, sb);
    __builtin_amdgcn_sched_barrier(0);
    read_a(I, Int<0>{}, Int<4>{});
    row(Int<2>{});
    issue(I, Int<6>{}, sb);
    issue(I, Int<7>{}, sb);
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(63, ReadsA));       // A 3 is read
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    read_a(I, Int<1>{}, Int<5>{});
    row(Int<3>{});
    issue(I, Int<0>{}, s);
    __builtin_amdgcn_sched_barrier(0);
    read_a(I, Int<2>{}, Int<6>{});
    row(Int<4>{});
    issue(I, Int<2>{}, s);
    __builtin_amdgcn_sched_barrier(0);
    read_a(I, Int<3>{}, Int<7>{});
    row(Int<5>{});
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(Loads, 0));
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    read_a(Next{}, Int<0>{}, Int<0>{});
    read_a(Next{}, Int<1>{}, Int<1>{});
    for_each<4>([&](auto J) {
      mma(Int<6>{}, Int<2>{}, Int<0>{}, J);
      mma(Int<7>{}, Int<3>{}, Int<0>{}, J);
      mma(Int<6>{}, Int<2>{}, Int<1>{}, J);
      mma(Int<7>{}, Int<3>{}, Int<1>{}, J);
      read_b(Next{}, J);
      if constexpr (J == 1) issue(I, Int<1>{}, s);
      if constexpr (J == 2) issue(I, Int<3>{}, s);
      __builtin_amdgcn_sched_barrier(0);
    });
  };

  int item = item_at(0);
  if (item < 0) return;
  Place now = place(item), next = place(item_at(1));
  int round = 1;
  for_each<2>([&](auto I) {
    const Source s = source(now.k0 + I, now, next);
    for_each<4>([&](auto Q) { issue(I, Int<4 + Q>{}, s); });
    if constexpr (BK == kCodes) widen(I);
    issue(I, Int<0>{}, s);
    issue(I, Int<2>{}, s);
    issue(I, Int<1>{}, s);
    issue(I, Int<3>{}, s);
  });
  if constexpr (BK == kCodes) {
    const Source s = source(now.k0 + 2, now, next);
    for_each<4>([&](auto Q) { issue(Int<0>{}, Int<4 + Q>{}, s); });
    // Of 4, 4 and the codes' 4 loads, slot 0's first half of A has landed.
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(2 + Loads, 0));
  } else {
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(2 + Loads, 15));
  }
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  read_a(Int<0>{}, Int<0>{}, Int<0>{});
  read_a(Int<0>{}, Int<1>{}, Int<1>{});
  for_each<4>([&](auto J) { read_b(Int<0>{}, J); });

  while (item >= 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = v4f{0, 0, 0, 0};
    for (int k = now.k0; k < now.k1; k += 2) {
      stage(Int<0>{}, k, now, next);
      stage(Int<1>{}, k + 1, now, next);
    }
    Spot at;
    at.tn = now.tn;
    at.wn = wn;
    at.part = now.part;
    at.lrow = 128 * wm + r16;
    at.lcol = 64 * wn + (BK == kAlong ? 16 : 4) * g;
    at.row0 = (int64_t)now.tm * kTile + at.lrow;
    at.col0 = (int64_t)now.tn * kTile + at.lcol;
    at.to = now.part < 0 ? nullptr
                         : t.split_ws + ((int64_t)now.split_tile * t.parts + now.part) * (kTile * kTile);
    epi.template store<BK == kAlong>(acc, at, t.m, t.n);
    item = item_at(round);
    now = next;
    next = place(item < 0 ? -1 : item_at(++round));
  }
  // No load may be in flight into LDS when the workgroup ends.
  __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));
#endif
}

// ---- host ---------------------------------------------------------------------
inline int64_t tiles_of(int64_t n) { return (n + kTile - 1) / kTile; }
inline int64_t units_of(int64_t K) { return (K + 2 * kStageK - 1) / (2 * kStageK); }

inline TileArgs tile_args(Operand a, Operand b, int64_t m, int64_t n, int64_t K) {
  TileArgs t{};
  t.a = a;
  t.b = b;
  t.m = m;
  t.n = n;
  t.K = K;
  t.tiles_m = (int)tiles_of(m);
  t.tiles_n = (int)tiles_of(n);
  t.units = (int)units_of(K);
  t.full = t.tiles_m * t.tiles_n;
  t.parts = 1;
  return t;
}
inline dim3 tile_grid(const TileArgs& t) {
  const int64_t items = (int64_t)t.full + (int64_t)t.split * t.parts, cus = compute_units();
  return dim3((unsigned)(items < cus ? items : cus));
}

}  // namespace tiles
}  // namespace adahop
