// Products of bf16 operands in tiles fed through LDS, with an epilogue of the
// caller's (gfx950): C[i, j] = sum_k A(i, k) B(j, k) in fp32.
//
// An operand lies along K ([rows][K], row-major) or across it ([K][rows]); B
// may also be MXFP8 codes and scales across K, widened to bf16 on their way into
// LDS. Any sizes; K of an operand along it in 16-byte chunks, rows of one
// across it too (the caller checks).
//
// Large tiles, 256 (192) x 256: a workgroup of 8 waves, two a SIMD, a wave 128
// (96) x 64 of it as 8 (6) x 4 blocks of v_mfma_f32_16x16x32_bf16 (B first, so that
// a lane holds four neighbouring columns of a row). K advances 64 elements a
// stage through two LDS slots of 64 (56) KB. A slot is refilled with the stage
// after next in two parts, as soon as all waves have read them: B and the first
// half of A after the second block row, the other half after the last but two,
// so that every load has more than a stage of time for two barriers a stage (one
// refill a stage leaves the matrix cores waiting; three, with B's own barrier,
// were 1 % slower). LDS reads and loads are spread between the matrix
// instructions: issued together they hold up the wave's own (operands across K:
// 5 % of the time). Workgroups stay: the next tile's first stages are loaded
// during a tile's last ones and its epilogue.
//
// Measured: 8192 x 4096 x 65536 (4.4e12 operations) with A along K and B across
// 1430 .. 1500 TFLOP/s (A of two terms, 32768 each, 1540 .. 1570), 65536 x 4096 x 8192
// with both across 1410 .. 1500 (two terms, 32768 x 4096 x 8192, 1450 .. 1490), the
// matrix cores busy 80 .. 83 % of the time at 1.75 .. 1.77 GHz, the clock that the power
// limit leaves (16x16x32 and 32x32x16 blocks alike); 4096 x 14336 x 32768 (3.8e12) with
// both across 1380 .. 1440, from codes 1280 .. 1390, busy 65 % at 1.87 .. 1.88 GHz. The
// kernel that reads codes keeps four registers in memory from before its tiles to
// their epilogues.
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
#include "tile_plan.h"

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

constexpr int kTile = 256;                 // rows and columns of a large tile
constexpr int kStageK = 64;                // K elements of a stage
constexpr int kThreads = 512;
constexpr int kRingCols = 128;             // columns of a small tile
constexpr int kGroupM = 8;                 // tile rows that run together on one XCD

struct Operand {
  const uint8_t* p;
  int64_t ld;                // bytes from a row to the next
  int64_t chunk;             // bf16: bytes from 64 columns to the next 64 (128: plain rows)
  const uint8_t* scales;     // kCodes: a byte per 32 columns
  int64_t ld_scales;
  int64_t term = 0;          // A of two terms: bytes from the first to the second
};

struct TileArgs {
  Operand a, b;
  int64_t m, n, K;
  int tiles_m, tiles_n;
  int bm, bn;                // rows and columns of a tile
  int units;                 // pairs of stages of K
  // Items 0 .. full - 1 are whole tiles; those after them each one of `parts`
  // parts of K of a tile, whose sums go to split_ws ([tile][part][bm][bn]). All
  // tiles' first parts come first, so that what an XCD runs at once shares K-rows.
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
// row0 + step i, column col0 + (BK == kAlong ? 4 j : 16 j) + e.
struct Spot {
  int64_t row0, col0;
  int64_t group;             // the wave's columns start at 64 group
  float* to;                 // a part's sums [bm][bn]; null: a whole tile
  int step;                  // from a block row to the next
  int lrow, lcol, bn;        // row and column in the tile
};

// Bytes of the 16-byte chunks that hold n elements.
__device__ __forceinline__ int64_t chunks(int64_t n) { return 2 * ((n + 7) & ~(int64_t)7); }
// A stage's rows of an operand: the descriptor starts at its first byte and ends
// with its last, so that rows and K-rows past the ends read as 0. p: the tile's
// first byte at the stage's first k; span: bytes of the tile's rows (across K: columns) but for
// the last one's own; left: elements of K from the stage's first.
template <Kind K>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t source_of(const uint8_t* p, int span, int64_t ld, int left) {
  const int bytes = K == kAlong ? span + (int)chunks(left) : (left - 1) * (int)ld + span;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0, left > 0 ? bytes : 0, kBufferFlags);
}
// First byte of a tile's rows r0 .. (a multiple of 64) and their span, as source_of
// takes them.
template <Kind K>
__device__ __forceinline__ const uint8_t* tile_base(const Operand& o, int64_t r0) {
  return K == kAlong ? o.p + r0 * o.ld : K == kCodes ? o.p + r0 : o.p + r0 / 64 * o.chunk;
}
template <Kind K>
__device__ __forceinline__ int tile_span(const Operand& o, int64_t rows) {
  if constexpr (K == kAlong) return (int)((rows - 1) * o.ld);
  else if constexpr (K == kCodes) return (int)rows;
  else return (int)((rows - 1) / 64 * o.chunk + chunks((rows - 1) % 64 + 1));
}
// 16 K-rows' elements of a lane's column, transposed on their way from LDS: two
// runs of four K-rows, `next` bytes apart.
__device__ __forceinline__ v4i read_across(const uint8_t* p, int next) {
  const v2i lo = __builtin_bit_cast(v2i, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s16*)p));
  const v2i hi = __builtin_bit_cast(v2i, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s16*)(p + next)));
  return v4i{lo[0], lo[1], hi[0], hi[1]};
}
// 8 codes under one scale as 8 bf16 (exact; below 2^-126 possibly 0). The
// instruction takes the scale's exponent alone, so every byte is its E8M0 value.
__device__ __forceinline__ v4i widen8(uint32_t lo, uint32_t hi, uint8_t scale) {
  const float by = __builtin_bit_cast(float, (uint32_t)scale << 23);
  return v4i{__builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, by, false)),
             __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, by, true)),
             __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, by, false)),
             __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, by, true))};
}
__device__ __forceinline__ v4f product16(const v4i& b, const v4i& a, const v4f& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, b), __builtin_bit_cast(v8bf, a), c, 0, 0, 0);
}

template <int Rows>
struct Half {
  uint8_t a[Rows * 128];
};
struct Wide {
  uint8_t b[256 * 128];
};

// Terms: A is the sum of so many matrices of its layout; B is read once for each.
template <Kind AK, Kind BK, typename Epi, int FM, int Terms>
__global__ void __launch_bounds__(kThreads, 1) bf16_tile_kernel(TileArgs t, Epi epi) {
#ifdef __HIP_DEVICE_COMPILE__                        // the host pass needs the launch stub alone
  // Tile rows; a wave's block rows in A's second half; loads of a wave and stage:
  // of A (2 of the first half) and 4 of B.
  constexpr int BM = 32 * FM, Rest = FM - 4, LA = FM / 2, Loads = LA + 4;
  static_assert(FM == 8 || (FM == 6 && AK == kAlong), "");
  static_assert(Terms == 1 || (Terms == 2 && BK != kCodes), "");
  // One LDS object for each part that is filled at once: alias analysis then
  // sees that loads into one do not touch another, and adds no wait before
  // the reads.
  __shared__ __attribute__((aligned(1024))) Half<128> f0, f1;           // a wave row's first 4 block rows
  __shared__ __attribute__((aligned(1024))) Half<32 * Rest> r0, r1;     // and the others
  __shared__ __attribute__((aligned(1024))) Wide w0, w1;
  auto half = [&](auto I, auto H) -> uint8_t* {
    if constexpr (I == 0 && H == 0) return f0.a;
    else if constexpr (I == 0) return r0.a;
    else if constexpr (H == 0) return f1.a;
    else return r1.a;
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
  // An item's place, all scalar: of its tile, and where its operands' stages start.
  // rest: elements of K from its first stage's on; end: the same, once its last
  // stage (of an even number) is taken.
  struct Place {
    int tm, tn, part, split_tile, stages, rest, end;
    const uint8_t* a;
    const uint8_t* b;
    const uint8_t* scales;
    int a_span, b_span;
  };
  // Bytes from a stage to the next.
  const uint32_t step_a = (uint32_t)(AK == kAlong ? t.a.chunk : kStageK * t.a.ld);
  const uint32_t step_b = BK == kAlong ? 128 : (uint32_t)(kStageK * t.b.ld);
  const uint32_t step_scales = (uint32_t)(kStageK * t.b.ld_scales);
  auto place = [&](int item) {
    // Without an item: stages past the end of any K, without an end.
    Place p{0, 0, -1, 0, 0, 0, 1, t.a.p, t.b.p, t.b.scales, 0, 0};
    if (item < 0) return p;
    int tile = item, part = -1;
    if (item >= t.full) {
      const int s = item - t.full;
      part = s / t.split;
      p.split_tile = __builtin_amdgcn_readfirstlane(s - part * t.split);
      tile = t.full + p.split_tile;
    }
    int m_, n_;
    tile_at(tile, t.tiles_m, t.tiles_n, &m_, &n_);
    p.tm = __builtin_amdgcn_readfirstlane(m_);
    p.tn = __builtin_amdgcn_readfirstlane(n_);
    p.part = __builtin_amdgcn_readfirstlane(part);
    int k0 = 0, k1 = 2 * t.units;
    if (p.part >= 0) {
      k0 = 2 * __builtin_amdgcn_readfirstlane((int)((int64_t)t.units * p.part / t.parts));
      k1 = 2 * __builtin_amdgcn_readfirstlane((int)((int64_t)t.units * (p.part + 1) / t.parts));
    }
    p.stages = k1 - k0;
    p.rest = (int)t.K - kStageK * k0;
    p.end = (int)t.K - kStageK * k1;
    const int64_t m0 = (int64_t)p.tm * BM, n0 = (int64_t)p.tn * kTile;
    p.a = tile_base<AK>(t.a, m0) + (int64_t)k0 * step_a;
    p.b = tile_base<BK>(t.b, n0) + (int64_t)k0 * step_b;
    p.a_span = tile_span<AK>(t.a, t.m - m0 < BM ? t.m - m0 : BM);
    p.b_span = tile_span<BK>(t.b, t.n - n0 < kTile ? t.n - n0 : kTile);
    if constexpr (BK == kCodes) p.scales = t.b.scales + n0 / 32 + (int64_t)k0 * step_scales;
    return p;
  };

  // ---- loads: this wave's share of a stage ------------------------------------
  // An operand's stages in the order of their loads. A step on from the last
  // stage is a few scalar instructions between the matrix instructions of a
  // stage's first two block rows; descriptors formed anew from k, some 60 in one
  // run, held the matrix cores up (4 % of the time, beside codes 8 %). Selects keep
  // the stages free of branches.
  struct Cursor {
    const uint8_t* p;
    const uint8_t* scales;
    int span, rest, end;
  };
  struct Source {
    __amdgpu_buffer_rsrc_t v, scales;
    int left;
  };
  // The next stage's descriptors; past an item's last stage, item `next`'s first.
  auto take = [&](auto IsB, Cursor& c, const Place& next) __attribute__((always_inline)) {
    constexpr bool Is = decltype(IsB)::value;
    constexpr Kind K = Is ? BK : AK;
    const bool over = c.rest == c.end;
    c.p = over ? (Is ? next.b : next.a) : c.p;
    c.span = over ? (Is ? next.b_span : next.a_span) : c.span;
    c.rest = over ? next.rest : c.rest;
    c.end = over ? next.end : c.end;
    Source s;
    s.left = c.rest < kStageK ? c.rest : kStageK;        // none: 0 or less
    s.v = source_of<K>(c.p, c.span, Is ? t.b.ld : t.a.ld, s.left);
    c.p += Is ? step_b : step_a;
    if constexpr (K == kCodes) {
      c.scales = over ? next.scales : c.scales;
      s.scales = source_of<K>(c.scales, (int)((unsigned)c.span / 32), t.b.ld_scales, s.left);
      c.scales += step_scales;
    }
    c.rest -= kStageK;
    return s;
  };
  auto take_a = [&](Cursor& c, const Place& next) __attribute__((always_inline)) { return take(Int<0>{}, c, next); };
  auto take_b = [&](Cursor& c, const Place& next) __attribute__((always_inline)) { return take(Int<1>{}, c, next); };
  // Block row i of wave row wm is rows 32 i + 16 wm .. +15 of the tile, so that a
  // tile of few rows has work for both. Along K, load q of this wave fills rows
  // 64 q' + 8 wave + lane / 8 of B or of a half of A (loads 0 and 2 the first, 1 and
  // 3 the other; q' = q / 2), with chunks XORed as they are read; across, K-rows
  // (A) 32 q' + 4 wave + lane / 16 of a half, (B) 16 q + 2 wave + lane / 32.
  const int row8 = 8 * wave + (lane >> 3);
  const int ca = (lane & 7) ^ ((row8 >> 1) & 7);
  const int cb = (lane & 7) ^ (2 * ((row8 >> 4) & 3) + ((row8 >> 1) & 1));
  const int ka = 4 * wave + (lane >> 4), kb = 2 * wave + (lane >> 5);
  const int ga = ((lane & 15) >> 1) ^ ((ka & 3) + 4 * ((ka >> 3) & 1));
  const int gb0 = ((lane & 31) >> 1) ^ ((kb & 3) + 4 * ((kb >> 3) & 1));
  const int chunk_a = BK == kCodes ? 128 : (int)t.a.chunk;   // beside codes, A lies in plain rows
  const int rowa = 32 * (wave >> 1) + 8 * (wave & 1) + (lane >> 3);
  // The second half holds, of 6 block rows, two: 16 rows of each wave row.
  const int rowr = FM == 8 ? 128 + rowa : 128 + 32 * ((wave >> 1) & 1) + 16 * (wave >> 2) + 8 * (wave & 1) + (lane >> 3);
  const int oa = AK == kAlong ? rowa * (int)t.a.ld + 16 * ca
                              : ka * (int)t.a.ld + ((ga & 3) >> 1) * chunk_a + 64 * (ga & 1) + 32 * (ga >> 2) +
                                    16 * (lane & 1);
  const int orest = rowr * (int)t.a.ld + 16 * ca;
  // Codes: two runs of 16 of a stage a thread, K-rows 32 u + thread / 16.
  const int kc = threadIdx.x >> 4, gc = threadIdx.x & 15;
  const int ob = BK == kCodes ? kc * (int)t.b.ld + 16 * gc : BK == kAlong ? row8 * (int)t.b.ld + 16 * cb : kb * (int)t.b.ld + 32 * gb0 + 16 * (lane & 1);
  // Codes of the stage after the next but one, loaded a stage ahead of their
  // widening into the slot that the stage before them frees.
  v4i codes[2];
  uint8_t scale[2];
  const int oc = kc * 512 + 32 * (gc ^ ((kc & 3) + 4 * ((kc >> 3) & 1))) + 16 * ((gc >> 2) & 1);
  // Half h of run u. Of 8 threads, 4 begin with their second half, so that a
  // write's 16-byte pieces lie 16 bytes apart over 128.
  const int sw = (gc >> 2) & 1;
  auto widen = [&](auto I, auto U, auto H) __attribute__((always_inline)) {
    constexpr int u = decltype(U)::value, h = decltype(H)::value;
    const bool last = h != sw;
    const v4i w = widen8((uint32_t)(last ? codes[u][2] : codes[u][0]), (uint32_t)(last ? codes[u][3] : codes[u][1]), scale[u]);
    *reinterpret_cast<v4i*>(wide(I).b + (oc ^ (16 * h)) + 16384 * u) = w;
  };
  // Across K, a row's last bytes are followed by the next row's: columns past
  // the tile's end reach only sums that are not stored.
  auto issue = [&](auto I, auto Q, const Source& s) __attribute__((always_inline)) {
    constexpr int q = decltype(Q)::value;
    if constexpr (q < 4) {
      int v;
      if constexpr (AK == kAlong) v = 8 * ca < s.left ? (q % 2 == 0 ? oa : orest) + 16 * (q / 2) * (int)t.a.ld : kPastEnd;
      else v = oa + 32 * (q / 2) * (int)t.a.ld + 2 * (q % 2) * chunk_a;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(s.v, (lds_void*)(half(I, Int<q % 2>{}) + 1024 * (8 * (q / 2) + wave)),
                                               16, v, 0, 0, 0);
    } else if constexpr (BK == kCodes) {
      constexpr int u = (q - 4) / 2;
      if constexpr (q % 2 == 0)
        codes[u] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(s.v, ob + 32 * u * (int)t.b.ld, 0, 0));
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
      __builtin_amdgcn_raw_ptr_buffer_load_lds(s.v, (lds_void*)&wide(I).b[1024 * (8 * j + wave)], 16, v, 0, 0, 0);
    }
  };

  // ---- fragments --------------------------------------------------------------
  const int q4 = r16 >> 2, sub = r16 & 3;
  const int hk = q4 + 4 * (g & 1);                   // h(k) of this lane's K-rows
  const int fa = AK == kAlong ? (64 * wm + r16) * 128 + 16 * (g ^ ((r16 >> 1) & 7))
                              : (8 * g + q4) * 256 + 8 * sub;
  const int fb = BK == kAlong ? (64 * wn + 16 * q4 + sub) * 128 + 16 * (g ^ (2 * q4 + (sub >> 1)))
                              : (8 * g + q4) * 512 + 8 * sub;
  // Across K: the first block's address; block i's differs in the bits of 32 i.
  const int xa = fa + 32 * ((4 * wm) ^ hk), xb = fb + 32 * ((4 * wn) ^ hk);
  const int fr = FM == 8 ? fa : fa - 32 * 128 * wm;  // in A's second half
  v4f acc[FM][4];
  v4i A[4][2], B[4][2];
  auto read_a = [&](auto I, auto Buf, auto R) __attribute__((always_inline)) {
    constexpr int b = decltype(Buf)::value, i = decltype(R)::value;
    const uint8_t* p = half(I, Int<i / 4>{});
    if constexpr (AK == kAlong) {
      const int at = i < 4 ? fa : fr;
      A[b][0] = *reinterpret_cast<const v4i*>(p + 2048 * (i % 4) + at);
      A[b][1] = *reinterpret_cast<const v4i*>(p + 2048 * (i % 4) + (at ^ 64));
    } else {
      A[b][0] = read_across(p + (xa ^ (32 * (i % 4))), 1024);
      A[b][1] = read_across(p + (xa ^ (32 * (i % 4))) + 8192, 1024);
    }
  };
  auto read_b = [&](auto I, auto J) __attribute__((always_inline)) {
    constexpr int j = decltype(J)::value;
    const uint8_t* p = wide(I).b;
    if constexpr (BK == kAlong) {
      B[j][0] = *reinterpret_cast<const v4i*>(p + 512 * j + fb);
      B[j][1] = *reinterpret_cast<const v4i*>(p + 512 * j + (fb ^ 64));
    } else {
      B[j][0] = read_across(p + (xb ^ (32 * j)), 2048);
      B[j][1] = read_across(p + (xb ^ (32 * j)) + 16384, 2048);
    }
  };
  auto mma = [&](auto R, auto Buf, auto S, auto J) __attribute__((always_inline)) {
    constexpr int i = decltype(R)::value, b = decltype(Buf)::value, s = decltype(S)::value, j = decltype(J)::value;
    acc[i][j] = product16(B[j][s], A[b][s], acc[i][j]);
  };
  constexpr int ReadsA = AK == kAlong ? 2 : 4;       // LDS reads of a block row's fragments

  Cursor cur_a, cur_b;
  // A stage in slot I: enters with its B fragments and first two A fragments
  // read; leaves with the next stage's. Fragment i of A sits in buffer
  // (i + Off) % 4. Loads still in flight at the first and the last wait: a
  // stage's, issued since those of the parts that are due.
  auto stage = [&](auto I, const Place& next) __attribute__((always_inline)) {
    using Next = Int<1 - decltype(I)::value>;
    constexpr int Off = (FM * decltype(I)::value) % 4;
    auto read = [&](auto R) { read_a(I, Int<(decltype(R)::value + Off) % 4>{}, R); };
    // A block row's matrix instructions with its LDS reads, the widening of the
    // codes' run `Run` (two LDS writes) and `Count` loads from `First` on (of A
    // every other) between them.
    auto step = [&](auto R, auto Reads, auto Run, auto First, auto Count, const Source& from) __attribute__((always_inline)) {
      constexpr int r = decltype(R)::value, run = decltype(Run)::value, count = decltype(Count)::value;
      for_each<2>([&](auto S) { for_each<4>([&](auto J) { mma(R, Int<(r + Off) % 4>{}, S, J); }); });
      if constexpr (run >= 0) for_each<2>([&](auto H) { widen(I, Run, H); });
      for_each<count>([&](auto C) {
        constexpr int first = decltype(First)::value;
        issue(I, Int<first + decltype(C)::value * (first < 4 ? 2 : 1)>{}, from);
      });
      for_each<8>([&](auto X) {
        constexpr int x = decltype(X)::value;
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                                          // MFMA
        if constexpr (r < 2) __builtin_amdgcn_sched_group_barrier(0x004, 3, 0);                     // SALU
        if constexpr (x < decltype(Reads)::value) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // DS read
        if constexpr (run >= 0) __builtin_amdgcn_sched_group_barrier(0x002, 3, 0);                  // VALU
        if constexpr (run >= 0 && x % 4 == 3) __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);    // DS write
        if constexpr (x >= 4 && x - 4 < count) __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);   // VMEM
      });
      __builtin_amdgcn_sched_barrier(0);
    };
    constexpr bool Codes = BK == kCodes;
    read(Int<2>{});
    read(Int<3>{});
    const Source sb = take_b(cur_b, next);
    step(Int<0>{}, Int<2 * ReadsA>{}, Int<-1>{}, Int<0>{}, Int<0>{}, sb);
    const Source s = take_a(cur_a, next);
    step(Int<1>{}, Int<0>{}, Int<-1>{}, Int<0>{}, Int<0>{}, s);
    // B and A's first half are read, its second half has landed.
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(Loads, 0));
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (Codes) {
      // A run's codes of the stage after, once those before are widened; all of
      // them before A's loads: waiting for them then waits for none of those that
      // are due later.
      read(Int<4>{});
      step(Int<2>{}, Int<ReadsA>{}, Int<0>{}, Int<0>{}, Int<0>{}, s);
      read(Int<5>{});
      step(Int<3>{}, Int<ReadsA>{}, Int<1>{}, Int<4>{}, Int<2>{}, sb);
      read(Int<6>{});
      step(Int<4>{}, Int<ReadsA>{}, Int<-1>{}, Int<6>{}, Int<2>{}, sb);
      read(Int<7>{});
      step(Int<5>{}, Int<ReadsA>{}, Int<-1>{}, Int<0>{}, Int<2>{}, s);
    } else {
      read(Int<4>{});
      step(Int<2>{}, Int<ReadsA>{}, Int<-1>{}, Int<4>{}, Int<2>{}, sb);
      read(Int<5>{});
      step(Int<3>{}, Int<ReadsA>{}, Int<-1>{}, Int<6>{}, Int<2>{}, sb);
      if constexpr (FM == 8) {
        read(Int<6>{});
        step(Int<4>{}, Int<ReadsA>{}, Int<-1>{}, Int<0>{}, Int<1>{}, s);
        read(Int<7>{});
        step(Int<5>{}, Int<ReadsA>{}, Int<-1>{}, Int<2>{}, Int<1>{}, s);
      } else {
        issue(I, Int<0>{}, s);
        issue(I, Int<2>{}, s);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(Loads, 0));
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    constexpr int X = FM - 2, Y = FM - 1;                      // the last two block rows
    read_a(Next{}, Int<(FM + Off) % 4>{}, Int<0>{});
    read_a(Next{}, Int<(FM + 1 + Off) % 4>{}, Int<1>{});
    for_each<4>([&](auto J) {
      for_each<2>([&](auto S) {
        mma(Int<X>{}, Int<(X + Off) % 4>{}, S, J);
        mma(Int<Y>{}, Int<(Y + Off) % 4>{}, S, J);
      });
      read_b(Next{}, J);
      if constexpr (J == 1) issue(I, Int<1>{}, s);
      if constexpr (J == 2 && FM == 8) issue(I, Int<3>{}, s);
      for_each<4>([&](auto) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, (J == 0 ? 3 : 1) * (ReadsA / 2) / 2, 0);
      });
      __builtin_amdgcn_sched_barrier(0);
    });
  };

  int item = item_at(0);
  if (item < 0) return;
  Place now = place(item), next = place(item_at(1));
  int round = 1;
  cur_a = {now.a, nullptr, now.a_span, now.rest, now.end};
  cur_b = {now.b, now.scales, now.b_span, now.rest, now.end};
  if constexpr (BK == kCodes) {
    // The order of the loads after slot 0's is a stage's, so that the waits for
    // codes are as loose here as there.
    const Source b0 = take_b(cur_b, next), b1 = take_b(cur_b, next), b2 = take_b(cur_b, next);
    const Source s = take_a(cur_a, next), s1 = take_a(cur_a, next);
    auto whole = [&](auto I) __attribute__((always_inline)) {
      for_each<4>([&](auto X) { widen(I, Int<decltype(X)::value / 2>{}, Int<decltype(X)::value % 2>{}); });
      __builtin_amdgcn_sched_barrier(0);
    };
    for_each<4>([&](auto Q) { issue(Int<0>{}, Int<4 + Q>{}, b0); });
    for_each<4>([&](auto Q) { issue(Int<0>{}, Q, s); });
    whole(Int<0>{});
    for_each<4>([&](auto Q) { issue(Int<1>{}, Int<4 + Q>{}, b1); });
    whole(Int<1>{});
    for_each<4>([&](auto Q) { issue(Int<0>{}, Int<4 + Q>{}, b2); });
    __builtin_amdgcn_sched_barrier(0);
    issue(Int<1>{}, Int<0>{}, s1);
    issue(Int<1>{}, Int<2>{}, s1);
    __builtin_amdgcn_sched_barrier(0);               // the waits count loads in this order
    issue(Int<1>{}, Int<1>{}, s1);
    issue(Int<1>{}, Int<3>{}, s1);
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(Loads, 0));
  } else {
    for_each<2>([&](auto I) {
      const Source s = take_a(cur_a, next), sb = take_b(cur_b, next);
      for_each<4>([&](auto Q) { issue(I, Int<4 + Q>{}, sb); });
      issue(I, Int<0>{}, s);
      issue(I, Int<2>{}, s);
      __builtin_amdgcn_sched_barrier(0);               // the waits count loads in this order
      issue(I, Int<1>{}, s);
      if constexpr (FM == 8) issue(I, Int<3>{}, s);
      __builtin_amdgcn_sched_barrier(0);
    });
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(Rest / 2 + Loads, 15));
  }
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  read_a(Int<0>{}, Int<0>{}, Int<0>{});
  read_a(Int<0>{}, Int<1>{}, Int<1>{});
  for_each<4>([&](auto J) { read_b(Int<0>{}, J); });

  while (item >= 0) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = v4f{0, 0, 0, 0};
    if constexpr (Terms == 1) {
      for (int k = 0; k < now.stages; k += 2) {
        stage(Int<0>{}, next);
        stage(Int<1>{}, next);
      }
    } else {
      // The first term's last stages load the second's first, whose own the next item's.
      Place to = now;
      to.a += t.a.term;
#pragma unroll 1
      for (int term = 0; term < Terms; ++term) {
        for (int k = 0; k < now.stages; k += 2) {
          stage(Int<0>{}, to);
          stage(Int<1>{}, to);
        }
        to = next;
      }
    }
    Spot at;
    at.lrow = 16 * wm + r16;
    at.lcol = 64 * wn + (BK == kAlong ? 16 : 4) * g;
    at.bn = kTile;
    at.step = 32;
    at.row0 = (int64_t)now.tm * BM + at.lrow;
    at.col0 = (int64_t)now.tn * kTile + at.lcol;
    at.group = (int64_t)now.tn * (kTile / 64) + wn;
    at.to = now.part < 0 ? nullptr
                         : t.split_ws + ((int64_t)now.split_tile * t.parts + now.part) * (BM * kTile);
    epi.template store<BK == kAlong>(acc, at, t.m, t.n);
    item = item_at(round);
    now = next;
    next = place(item < 0 ? -1 : item_at(++round));
  }
  // No load may be in flight into LDS when the workgroup ends.
  __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));
#endif
}

// Small tiles, one a workgroup: 16 FM WM rows by 64 WN = 128 columns, for
// products whose large tiles would leave compute units without work. K advances
// through four LDS slots, filled four stages ahead; a stage's last two block rows
// run while the next stage's first fragments are read and the slot is refilled.
// Layouts as above, of a K-row across K 256 bytes.
template <bool Across, int Rows>
struct RingPart {
  uint8_t v[Rows * 128];
  static_assert(!Across || Rows == 128, "K-rows of 256 bytes");
};

template <Kind AK, Kind BK, typename Epi, int WM, int WN, int FM, int Terms>
__global__ void __launch_bounds__(64 * WM * WN, 1) bf16_ring_kernel(TileArgs t, Epi epi) {
#ifdef __HIP_DEVICE_COMPILE__
  constexpr int Waves = WM * WN, BM = 16 * FM * WM, BN = 64 * WN;
  constexpr int Runs = 8 / Waves;                      // of 16 codes, a thread and stage
  constexpr int LA = BM / 8 / Waves, LB = BK == kCodes ? 2 * Runs : BN / 8 / Waves, Loads = LA + LB;
  static_assert(BN == kRingCols && FM >= 2 && FM % 2 == 0 && 3 * Loads < 64, "");
  using PartA = RingPart<AK != kAlong, BM>;
  using PartB = RingPart<BK != kAlong, BN>;
  __shared__ __attribute__((aligned(1024))) PartA a0, a1, a2, a3;
  __shared__ __attribute__((aligned(1024))) PartB b0, b1, b2, b3;
  auto pa = [&](auto I) -> uint8_t* {
    if constexpr (I == 0) return a0.v;
    else if constexpr (I == 1) return a1.v;
    else if constexpr (I == 2) return a2.v;
    else return a3.v;
  };
  auto pb = [&](auto I) -> uint8_t* {
    if constexpr (I == 0) return b0.v;
    else if constexpr (I == 1) return b1.v;
    else if constexpr (I == 2) return b2.v;
    else return b3.v;
  };
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int r16 = lane & 15, g = lane >> 4;

  // ---- place ------------------------------------------------------------------
  const int item = xcd_band(blockIdx.x, gridDim.x);
  const bool split = item >= t.full;
  const int s_ = split ? item - t.full : 0;
  const int part = split ? s_ / t.split : 0, split_tile = split ? s_ - part * t.split : 0;
  int m_, n_;
  tile_at(split ? t.full + split_tile : item, t.tiles_m, t.tiles_n, &m_, &n_);
  const int tm = __builtin_amdgcn_readfirstlane(m_), tn = __builtin_amdgcn_readfirstlane(n_);
  const int k0 = __builtin_amdgcn_readfirstlane(split ? 2 * (int)((int64_t)t.units * part / t.parts) : 0);
  const int end = __builtin_amdgcn_readfirstlane(2 * (split ? (int)((int64_t)t.units * (part + 1) / t.parts) : t.units));
  const int stages = ((int)t.K + kStageK - 1) / kStageK, k1 = end < stages ? end : stages;
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
  const uint8_t* base_a = tile_base<AK>(t.a, m0);
  const uint8_t* base_b = tile_base<BK>(t.b, n0);
  const int span_a = tile_span<AK>(t.a, t.m - m0 < BM ? t.m - m0 : BM);
  const int span_b = tile_span<BK>(t.b, t.n - n0 < BN ? t.n - n0 : BN);

  // ---- loads --------------------------------------------------------------------
  // As above, an operand's stages in the order of their loads; past k1 A's second
  // term follows, if there is one, and past that nothing is loaded. All in 32 bits (K below 2^30) but the addresses: what 64-bit
  // comparisons yield lies in vector registers, and a descriptor made from it
  // turns every load into a loop over lanes.
  const int end_rest = (int)t.K - kStageK * k1;
  const uint32_t step_a = (uint32_t)(AK == kAlong ? t.a.chunk : kStageK * t.a.ld);
  const uint32_t step_b = BK == kAlong ? 128 : (uint32_t)(kStageK * t.b.ld);
  const uint32_t step_scales = (uint32_t)(kStageK * t.b.ld_scales);
  struct Cursor {
    const uint8_t* p;
    const uint8_t* scales;
    int rest;
    int terms;               // still to come
  };
  const int first_rest = (int)t.K - kStageK * k0;
  const uint8_t* first_a = base_a + (int64_t)k0 * step_a;
  const uint8_t* first_b = base_b + (int64_t)k0 * step_b;
  Cursor cur_a{first_a, nullptr, first_rest, Terms - 1};
  Cursor cur_b{first_b, nullptr, first_rest, Terms - 1};
  if constexpr (BK == kCodes) cur_b.scales = t.b.scales + n0 / 32 + (int64_t)k0 * step_scales;
  struct Source {
    __amdgpu_buffer_rsrc_t v, scales;
    int left;
  };
  auto take = [&](auto IsB, Cursor& c) __attribute__((always_inline)) {
    constexpr bool Is = decltype(IsB)::value;
    constexpr Kind K = Is ? BK : AK;
    if constexpr (Terms > 1) {
      const bool over = c.rest == end_rest && c.terms > 0;
      c.p = over ? (Is ? first_b : first_a + t.a.term) : c.p;
      c.rest = over ? first_rest : c.rest;
      c.terms = over ? 0 : c.terms;
    }
    Source s;
    s.left = c.rest <= end_rest ? 0 : c.rest < kStageK ? c.rest : kStageK;
    s.v = source_of<K>(c.p, Is ? span_b : span_a, Is ? t.b.ld : t.a.ld, s.left);
    c.p += Is ? step_b : step_a;
    if constexpr (K == kCodes) {
      s.scales = source_of<K>(c.scales, (int)((unsigned)span_b / 32), t.b.ld_scales, s.left);
      c.scales += step_scales;
    }
    c.rest -= kStageK;
    return s;
  };
  // Load q of an operand along K: rows 8 (Waves q + wave) + lane / 8; across:
  // K-rows 4 (Waves q + wave) + lane / 16. The XOR keys of load q are those of
  // load 0 but for the bits that Waves q brings.
  const int row8 = 8 * wave + (lane >> 3);
  const int ca = (lane & 7) ^ ((row8 >> 1) & 7);
  const int cb = (lane & 7) ^ (2 * ((row8 >> 4) & 3) + ((row8 >> 1) & 1));
  const int k4 = 4 * wave + (lane >> 4);
  const int gx = ((lane & 15) >> 1) ^ ((k4 & 3) + 4 * ((k4 >> 3) & 1));
  const int oa = AK == kAlong ? row8 * (int)t.a.ld + 16 * ca : k4 * (int)t.a.ld + 16 * (lane & 1);
  const int ob = BK == kAlong ? row8 * (int)t.b.ld : k4 * (int)t.b.ld + 16 * (lane & 1);
  const int kc = threadIdx.x >> 3, gc = threadIdx.x & 7;     // + 8 Waves K-rows a run
  // A slot's next codes, loaded four stages before they are widened into it.
  v4i codes[4][Runs];
  uint8_t scale[4][Runs];
  const int sw = (gc >> 2) & 1;
  auto widen = [&](auto I) __attribute__((always_inline)) {
    for_each<Runs>([&](auto U) {
      constexpr int u = decltype(U)::value;
      constexpr int slot = decltype(I)::value;
      uint8_t* to = pb(I) + kc * 256 + 32 * (gc ^ ((kc & 3) + 4 * ((kc >> 3) & 1))) + 2048 * Waves * u;
      for_each<2>([&](auto H) {
        const bool last = decltype(H)::value != sw;
        *reinterpret_cast<v4i*>(to + (last ? 16 : 0)) =
            widen8((uint32_t)(last ? codes[slot][u][2] : codes[slot][u][0]), (uint32_t)(last ? codes[slot][u][3] : codes[slot][u][1]), scale[slot][u]);
      });
    });
  };
  auto load_a = [&](auto I, auto Q, const Source& s) __attribute__((always_inline)) {
    constexpr int q = decltype(Q)::value;
    int v;
    if constexpr (AK == kAlong) {
      v = 8 * ca < s.left ? oa + 8 * Waves * q * (int)t.a.ld : kPastEnd;
    } else {
      const int c = gx ^ (4 * ((Waves / 2 * q) & 1));      // 16 columns
      v = oa + (c >> 2) * (int)t.a.chunk + 32 * (c & 3) + 4 * Waves * q * (int)t.a.ld;
    }
    __builtin_amdgcn_raw_ptr_buffer_load_lds(s.v, (lds_void*)(pa(I) + 1024 * (Waves * q + wave)), 16, v, 0, 0, 0);
  };
  auto load_b = [&](auto I, auto Q, const Source& s) __attribute__((always_inline)) {
    constexpr int q = decltype(Q)::value;
    if constexpr (BK == kCodes) {
      constexpr int u = q / 2;
      if constexpr (q % 2 == 0)
        codes[decltype(I)::value][u] = __builtin_bit_cast(
            v4i, __builtin_amdgcn_raw_buffer_load_b128(s.v, (kc + 8 * Waves * u) * (int)t.b.ld + 16 * gc, 0, 0));
      else
        scale[decltype(I)::value][u] = __builtin_amdgcn_raw_buffer_load_b8(s.scales, (kc + 8 * Waves * u) * (int)t.b.ld_scales + gc / 2, 0,
                                                       0);
    } else {
      int v;
      if constexpr (BK == kAlong) {
        const int c = cb ^ (2 * ((Waves / 2 * q) & 3));
        v = 8 * c < s.left ? ob + 16 * c + 8 * Waves * q * (int)t.b.ld : kPastEnd;
      } else {
        v = ob + 32 * (gx ^ (4 * ((Waves / 2 * q) & 1))) + 4 * Waves * q * (int)t.b.ld;
      }
      __builtin_amdgcn_raw_ptr_buffer_load_lds(s.v, (lds_void*)(pb(I) + 1024 * (Waves * q + wave)), 16, v, 0, 0, 0);
    }
  };

  // ---- fragments ------------------------------------------------------------------
  const int q4 = r16 >> 2, sub = r16 & 3, hk = q4 + 4 * (g & 1);
  const int fa = AK == kAlong ? (16 * FM * wm + r16) * 128 + 16 * (g ^ ((r16 >> 1) & 7)) : (8 * g + q4) * 256 + 8 * sub;
  const int fb = BK == kAlong ? (64 * wn + 16 * q4 + sub) * 128 + 16 * (g ^ (2 * q4 + (sub >> 1)))
                              : (8 * g + q4) * 256 + 8 * sub;
  v4f acc[FM][4];
  v4i A[4][2], B[4][2];
  auto read_a = [&](auto I, auto Buf, auto R) __attribute__((always_inline)) {
    constexpr int b = decltype(Buf)::value, i = decltype(R)::value;
    const uint8_t* p = pa(I);
    if constexpr (AK == kAlong) {
      A[b][0] = *reinterpret_cast<const v4i*>(p + 2048 * i + fa);
      A[b][1] = *reinterpret_cast<const v4i*>(p + 2048 * i + (fa ^ 64));
    } else {
      const int at = fa + 32 * ((FM * wm + i) ^ hk);
      A[b][0] = read_across(p + at, 1024);
      A[b][1] = read_across(p + at + 8192, 1024);
    }
  };
  auto read_b = [&](auto I, auto J) __attribute__((always_inline)) {
    constexpr int j = decltype(J)::value;
    const uint8_t* p = pb(I);
    if constexpr (BK == kAlong) {
      B[j][0] = *reinterpret_cast<const v4i*>(p + 512 * j + fb);
      B[j][1] = *reinterpret_cast<const v4i*>(p + 512 * j + (fb ^ 64));
    } else {
      const int at = fb + 32 * ((4 * wn + j) ^ hk);
      B[j][0] = read_across(p + at, 1024);
      B[j][1] = read_across(p + at + 8192, 1024);
    }
  };
  constexpr int ReadsA = AK == kAlong ? 2 : 4, ReadsB = BK == kAlong ? 2 : 4;   // LDS reads of a block's fragments
  // First of the loads issued with block column j; codes' after their widening,
  // all with column 2.
  constexpr auto first = [](int j) { return BK != kCodes ? Loads * j / 4 : j < 3 ? 0 : j == 3 ? LB : Loads; };
  // A stage in slot I: enters with its B fragments and its first two A fragments
  // read; leaves with the next stage's. Fragment i of A sits in buffer
  // (i + Off) % 4. Codes are loaded eight stages ahead, and widened into the slot
  // after four (a stage ahead they made a stage as long as a load: 0.8 us instead
  // of 0.6).
  auto stage = [&](auto I) __attribute__((always_inline)) {
    constexpr int slot = decltype(I)::value;
    using Next = Int<(slot + 1) % 4>;
    constexpr int Off = (FM * slot) % 4;
    const Source sb = take(Int<1>{}, cur_b), s = take(Int<0>{}, cur_a);
    for_each<FM - 2>([&](auto R) {
      constexpr int i = decltype(R)::value;
      read_a(I, Int<(i + 2 + Off) % 4>{}, Int<i + 2>{});
      for_each<8>([&](auto X) {
        constexpr int x = decltype(X)::value;
        acc[i][x % 4] = product16(B[x % 4][x / 4], A[(i + Off) % 4][x / 4], acc[i][x % 4]);
      });
      for_each<8>([&](auto X) {
        constexpr int x = decltype(X)::value;
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x004, 4, 0);
        if constexpr (x < ReadsA) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      });
      __builtin_amdgcn_sched_barrier(0);
    });
    // All of this slot's reads are in; the next stage's loads of this wave have
    // landed when only the two later stages' are in flight. The barrier
    // publishes the next stage and frees this slot.
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(2 * Loads, 0));
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    for_each<4>([&](auto J) {
      if constexpr (J < 2) read_a(Next{}, Int<(FM + J + Off) % 4>{}, Int<J>{});
      constexpr int j = decltype(J)::value;
      for_each<2>([&](auto S) {
        constexpr int x = decltype(S)::value;
        acc[FM - 2][j] = product16(B[j][x], A[(FM - 2 + Off) % 4][x], acc[FM - 2][j]);
        acc[FM - 1][j] = product16(B[j][x], A[(FM - 1 + Off) % 4][x], acc[FM - 1][j]);
      });
      read_b(Next{}, J);
      if constexpr (BK == kCodes && j == 1) widen(I);
      for_each<first(j + 1) - first(j)>([&](auto Q) {
        constexpr int q = first(j) + decltype(Q)::value;
        if constexpr (q < LB) load_b(I, Int<q>{}, sb);
        else load_a(I, Int<q - LB>{}, s);
      });
      // One by one between the matrix instructions (3 to 5 % of a wave of tiles).
      constexpr int reads = (J < 2 ? ReadsA : 0) + ReadsB, loads = first(j + 1) - first(j);
      for_each<4>([&](auto X) {
        constexpr int x = decltype(X)::value;
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                                            // MFMA
        __builtin_amdgcn_sched_group_barrier(0x100, reads * (x + 1) / 4 - reads * x / 4, 0);          // DS read
        if constexpr (BK == kCodes && j == 1) {
          __builtin_amdgcn_sched_group_barrier(0x002, 8 * Runs, 0);                                   // VALU
          if constexpr (Runs > 1 || x % 2 == 0) __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);    // DS write
        }
        __builtin_amdgcn_sched_group_barrier(0x010, loads * (x + 1) / 4 - loads * x / 4, 0);          // VMEM
      });
      __builtin_amdgcn_sched_barrier(0);
    });
  };

#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = v4f{0, 0, 0, 0};
  if constexpr (BK == kCodes) {
    for_each<4>([&](auto I) {
      const Source sb = take(Int<1>{}, cur_b);
      for_each<LB>([&](auto Q) { load_b(I, Q, sb); });
    });
    for_each<4>([&](auto I) { widen(I); });
    __builtin_amdgcn_sched_barrier(0);
    // From here on in a stage's order, so that the waits for codes are as loose.
    for_each<4>([&](auto I) {
      const Source sb = take(Int<1>{}, cur_b), s = take(Int<0>{}, cur_a);
      for_each<LB>([&](auto Q) { load_b(I, Q, sb); });
      __builtin_amdgcn_sched_barrier(0);
      for_each<LA>([&](auto Q) { load_a(I, Q, s); });
      __builtin_amdgcn_sched_barrier(0);
    });
  } else {
    for_each<4>([&](auto I) {
      const Source sb = take(Int<1>{}, cur_b), s = take(Int<0>{}, cur_a);
      for_each<LB>([&](auto Q) { load_b(I, Q, sb); });
      for_each<LA>([&](auto Q) { load_a(I, Q, s); });
      __builtin_amdgcn_sched_barrier(0);               // the waits count loads in this order
    });
  }
  __builtin_amdgcn_s_waitcnt(waitcnt_imm(3 * Loads, 0));
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  read_a(Int<0>{}, Int<0>{}, Int<0>{});
  read_a(Int<0>{}, Int<1>{}, Int<1>{});
  for_each<4>([&](auto J) { read_b(Int<0>{}, J); });
  const int last = Terms == 1 ? k1 : k0 + Terms * (k1 - k0);
  int k = k0;
  for (; k + 4 <= last; k += 4) for_each<4>([&](auto I) { stage(I); });
  for_each<3>([&](auto I) {
    if (k + I < last) stage(I);
  });
  Spot at;
  at.lrow = 16 * FM * wm + r16;
  at.lcol = 64 * wn + (BK == kAlong ? 16 : 4) * g;
  at.bn = BN;
  at.step = 16;
  at.row0 = m0 + at.lrow;
  at.col0 = n0 + at.lcol;
  at.group = (int64_t)tn * WN + wn;
  at.to = !split ? nullptr : t.split_ws + ((int64_t)split_tile * t.parts + part) * (BM * BN);
  epi.template store<BK == kAlong>(acc, at, t.m, t.n);
  // No load may be in flight into LDS when the workgroup ends.
  __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));
#endif
}

// ---- host ---------------------------------------------------------------------
inline int64_t units_of(int64_t K) { return (K + 2 * kStageK - 1) / (2 * kStageK); }

inline TileArgs tile_args(const ProductPlan& p, Operand a, Operand b, int64_t m, int64_t n, int64_t K) {
  TileArgs t{};
  t.a = a;
  t.b = b;
  t.m = m;
  t.n = n;
  t.K = K;
  t.bm = tile_rows(p.tile);
  t.bn = tile_cols(p.tile);
  t.tiles_m = (int)((m + t.bm - 1) / t.bm);
  t.tiles_n = (int)((n + t.bn - 1) / t.bn);
  t.units = (int)units_of(K);
  t.full = (int)p.full;
  t.split = (int)p.split;
  t.parts = p.parts;
  return t;
}

template <Kind AK, Kind BK, int Terms = 1, typename Epi>
void tile_launch(const ProductPlan& p, TileArgs t, const Epi& epi, hipStream_t stream) {
  const int64_t items = p.full + p.split * p.parts, cus = compute_units();
  const dim3 most((unsigned)(items < cus ? items : cus)), all((unsigned)items);
  switch (p.tile) {
    case k256x256:
      // Codes are loaded three stages ahead, which has to stay within the next tile.
      if (BK == kCodes && t.units < 2) t.units = 2;
      bf16_tile_kernel<AK, BK, Epi, 8, Terms><<<most, dim3(kThreads), 0, stream>>>(t, epi);
      break;
    case k192x256:
      if constexpr (AK == kAlong) bf16_tile_kernel<AK, BK, Epi, 6, Terms><<<most, dim3(kThreads), 0, stream>>>(t, epi);
      break;
    case k64x128:
      if constexpr (AK == kAlong) bf16_ring_kernel<AK, BK, Epi, 2, 2, 2, Terms><<<all, dim3(256), 0, stream>>>(t, epi);
      break;
    default: bf16_ring_kernel<AK, BK, Epi, 4, 2, 2, Terms><<<all, dim3(512), 0, stream>>>(t, epi);
  }
}

}  // namespace tiles
}  // namespace adahop
