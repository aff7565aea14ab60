// Shared pieces of the MXFP8 operators (norm, quantizer, linear layer and
// their gradients): element loads and stores, the E8M0 / E4M3 conversion,
// cross-lane sums and maxima, the activation functions. gfx950 only.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstring>

namespace adahop {
namespace mx8 {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float bf16_to_f32(uint16_t h) {
  return __builtin_bit_cast(float, (uint32_t)h << 16);
}
// Round to nearest even in hardware (a NaN stays a NaN).
__device__ __forceinline__ uint16_t f32_to_bf16(float v) {
  return __builtin_bit_cast(uint16_t, (__bf16)v);
}
__device__ __forceinline__ uint32_t f32x2_to_bf16x2(float a, float b) {
  const bf16x2 p = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, p);
}

// ---- elements in groups of 8 ------------------------------------------------
// Rows start at any element, so a group's address is aligned to its element
// only: the memcpy keeps the access one 16-byte load or store, which the
// hardware takes at any address.
template <bool F32>
struct Elem;
template <>
struct Elem<false> {
  using type = uint16_t;
  static __device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
    u32x4 w;
    __builtin_memcpy(&w, p, 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __builtin_bit_cast(float, w[i] << 16);
      v[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ float load(const uint16_t* p) { return bf16_to_f32(*p); }
  static __device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = f32x2_to_bf16x2(v[2 * i], v[2 * i + 1]);
    __builtin_memcpy(p, &w, 16);
  }
  static __device__ __forceinline__ void store(uint16_t* p, float v) { *p = f32_to_bf16(v); }
  // v as the type holds it.
  static __device__ __forceinline__ float rounded(float v) { return (float)(__bf16)v; }
};
template <>
struct Elem<true> {
  using type = float;
  static __device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    f32x4 a, b;
    __builtin_memcpy(&a, p, 16);
    __builtin_memcpy(&b, p + 4, 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
  }
  static __device__ __forceinline__ float load(const float* p) { return *p; }
  static __device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
    const f32x4 a = {v[0], v[1], v[2], v[3]}, b = {v[4], v[5], v[6], v[7]};
    __builtin_memcpy(p, &a, 16);
    __builtin_memcpy(p + 4, &b, 16);
  }
  static __device__ __forceinline__ void store(float* p, float v) { *p = v; }
  static __device__ __forceinline__ float rounded(float v) { return v; }
};

// The k < 8 elements at p as 8 elements' words, 0 after them, and back: in
// pieces of 4, 2 and 1.
template <typename T>
__device__ __forceinline__ T read_as(const void* p) {
  T v;
  __builtin_memcpy(&v, p, sizeof(T));
  return v;
}
template <bool F32, int N>
__device__ __forceinline__ void load_part(const typename Elem<F32>::type* p, int k, uint32_t (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = 0;
  if constexpr (F32) {
    const int two = k & 4, one = k & 6;
    if (k & 4) {
      const u32x4 v = read_as<u32x4>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = v[i];
    }
    if (k & 2) {
      const u32x2 v = read_as<u32x2>(p + two);
      const uint32_t a = v[0], b = v[1];
      (two ? x[4] : x[0]) = a;
      (two ? x[5] : x[1]) = b;
    }
    if (k & 1) {
      const uint32_t v = read_as<uint32_t>(p + one);
      (one == 0 ? x[0] : one == 2 ? x[2] : one == 4 ? x[4] : x[6]) = v;
    }
  } else {
    const int two = k & 4, one = k & 6;
    if (k & 4) {
      const u32x2 v = read_as<u32x2>(p);
      x[0] = v[0];
      x[1] = v[1];
    }
    if (k & 2) (two ? x[2] : x[0]) = read_as<uint32_t>(p + two);
    if (k & 1) {
      const uint32_t v = read_as<uint16_t>(p + one);
      (one == 0 ? x[0] : one == 2 ? x[1] : one == 4 ? x[2] : x[3]) = v;
    }
  }
}
template <bool F32, int N>
__device__ __forceinline__ void store_part(typename Elem<F32>::type* p, int k, const uint32_t (&x)[N]) {
  const int two = k & 4, one = k & 6;
  if constexpr (F32) {
    if (k & 4) {
      const u32x4 v = {x[0], x[1], x[2], x[3]};
      __builtin_memcpy(p, &v, 16);
    }
    if (k & 2) {
      const u32x2 v = {two ? x[4] : x[0], two ? x[5] : x[1]};
      __builtin_memcpy(p + two, &v, 8);
    }
    if (k & 1) {
      const uint32_t v = one == 0 ? x[0] : one == 2 ? x[2] : one == 4 ? x[4] : x[6];
      __builtin_memcpy(p + one, &v, 4);
    }
  } else {
    if (k & 4) {
      const u32x2 v = {x[0], x[1]};
      __builtin_memcpy(p, &v, 8);
    }
    if (k & 2) {
      const uint32_t v = two ? x[2] : x[0];
      __builtin_memcpy(p + two, &v, 4);
    }
    if (k & 1) {
      const uint16_t v = (uint16_t)(one == 0 ? x[0] : one == 2 ? x[1] : one == 4 ? x[2] : x[3]);
      __builtin_memcpy(p + one, &v, 2);
    }
  }
}

// Elements c .. c + 7 of a row of `cols`; those past the end read as 0 and
// are not stored.
template <bool F32>
__device__ __forceinline__ void load_group(const typename Elem<F32>::type* row, int64_t c,
                                           int64_t cols, float (&v)[8]) {
  if (c + 8 <= cols) {
    Elem<F32>::load8(row + c, v);
  } else {
    uint32_t x[F32 ? 8 : 4];
    load_part<F32>(row + c, c < cols ? (int)(cols - c) : 0, x);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = __builtin_bit_cast(float, F32 ? x[F32 ? i : 0] : i % 2 ? x[i / 2] & 0xFFFF0000u : x[i / 2] << 16);
  }
}
template <bool F32>
__device__ __forceinline__ void store_group(typename Elem<F32>::type* row, int64_t c, int64_t cols,
                                            const float (&v)[8]) {
  if (c + 8 <= cols) {
    Elem<F32>::store8(row + c, v);
  } else if (c < cols) {
    uint32_t x[F32 ? 8 : 4];
#pragma unroll
    for (int i = 0; i < (F32 ? 8 : 4); ++i) {
      if constexpr (F32) x[i] = __builtin_bit_cast(uint32_t, v[i]);
      else x[i] = f32x2_to_bf16x2(v[2 * i], v[2 * i + 1]);
    }
    store_part<F32>(row + c, (int)(cols - c), x);
  }
}

// Elements c .. c + 7 as they are stored, for loads issued long before their
// use. A row's last group is the row's last 8 elements, moved into place when
// they are used: loads under a branch would be waited for in it (a row of 8191
// then costs its last wave a latency for each: 2050 x 8191 in 39 us instead of
// 26). Once: nontemporal, where whole cache lines are read at once and not
// again (reads stream at 6.9 TB/s instead of 6.1; lines read in pieces are
// fetched again: 2050 x 8191 in 48 us instead of 36).
typedef u32x4 u32x4_any __attribute__((aligned(2)));
template <bool F32>
struct Raw8 {
  u32x4 w[F32 ? 2 : 1];
  template <bool Once>
  __device__ __forceinline__ void load(const typename Elem<F32>::type* row, int64_t c, int64_t cols) {
    if (cols >= 8) {
      const u32x4_any* p = reinterpret_cast<const u32x4_any*>(row + (c + 8 <= cols ? c : cols - 8));
#pragma unroll
      for (int i = 0; i < (F32 ? 2 : 1); ++i) {
        // (an fp32 group's two loads each read half of every 32 bytes)
        if constexpr (Once && !F32) w[i] = __builtin_nontemporal_load(p + i);
        else w[i] = p[i];
      }
    } else {
      uint32_t x[F32 ? 8 : 4];
      load_part<F32>(row + c, c < cols ? (int)(cols - c) : 0, x);
#pragma unroll
      for (int i = 0; i < (F32 ? 2 : 1); ++i) w[i] = u32x4{x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]};
    }
  }
  // The elements, 0 past the end of the row.
  __device__ __forceinline__ void get(float (&v)[8], int64_t c, int64_t cols) const {
    constexpr int N = F32 ? 8 : 4;
    uint32_t x[N + 1];
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = w[i / 4][i % 4];
    x[N] = 0;
    if (cols >= 8 && c + 8 > cols) {
      const int s = c < cols ? (int)(c + 8 - cols) : 8;      // elements to move by
      constexpr int W = F32 ? 1 : 2;                         // elements of a word
#pragma unroll
      for (int b = 8; b >= W; b /= 2)
        if (s & b) {
#pragma unroll
          for (int i = 0; i < N; ++i) x[i] = i + b / W < N ? x[i + b / W < N ? i + b / W : 0] : 0u;
        }
      if (!F32 && (s & 1)) {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = x[i] >> 16 | x[i + 1] << 16;
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = __builtin_bit_cast(float, F32 ? x[F32 ? i : 0] : i % 2 ? x[i / 2] & 0xFFFF0000u : x[i / 2] << 16);
  }
};

// Codes c .. c + 7 of an MXFP8 row and their block's scale, loaded long before
// their use; c and cols are multiples of 8, and past the row's end the last
// group is read. `first`: the row's first column counted from a multiple of 32.
struct RawMx8 {
  u32x2 w;
  uint8_t byte;
  __device__ __forceinline__ void load(const uint8_t* codes, const uint8_t* scales, int64_t first, int64_t c,
                                       int64_t cols) {
    const int64_t at = first + (c < cols ? c : cols - 8);
    __builtin_memcpy(&w, codes + at, 8);
    byte = scales[at / 32];
  }
  // The values, 0 past the end of the row.
  __device__ __forceinline__ void get(float (&v)[8], int64_t c, int64_t cols) const;
};

// Whether every row of a matrix starts at a cache line.
inline bool line_aligned(const void* p, int64_t ld, int f32) {
  return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(ld * (f32 ? 4 : 2))) & 127u) == 0;
}

// ---- cross-lane -------------------------------------------------------------
template <int Ctrl>
__device__ __forceinline__ int dpp(int v) {
  return __builtin_amdgcn_update_dpp(0, v, Ctrl, 0xF, 0xF, false);
}
constexpr int kDppXor1 = 0xB1, kDppXor2 = 0x4E;          // quad_perm [1,0,3,2], [2,3,0,1]
constexpr int kDppHalfMirror = 0x141, kDppMirror = 0x140;   // within 8, within 16 lanes

// Sum over the wave, in every lane; a fixed tree, so the result is the same
// on every run.
__device__ __forceinline__ float wave_sum(float v) {
  v += __builtin_bit_cast(float, dpp<kDppXor1>(__builtin_bit_cast(int, v)));
  v += __builtin_bit_cast(float, dpp<kDppXor2>(__builtin_bit_cast(int, v)));
  v += __builtin_bit_cast(float, dpp<kDppHalfMirror>(__builtin_bit_cast(int, v)));
  v += __builtin_bit_cast(float, dpp<kDppMirror>(__builtin_bit_cast(int, v)));
  v += __shfl_xor(v, 16);
  v += __shfl_xor(v, 32);
  return v;
}
// Maximum of unsigned values over groups of 4 lanes.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  uint32_t o = (uint32_t)dpp<kDppXor1>((int)v);
  v = v > o ? v : o;
  o = (uint32_t)dpp<kDppXor2>((int)v);
  return v > o ? v : o;
}

// ---- MXFP8 ------------------------------------------------------------------
// Magnitudes are compared as bit patterns: they order as the values do, with
// infinity and then NaN above every finite one.
__device__ __forceinline__ uint32_t abs_bits(float v) {
  return __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu;
}
constexpr uint32_t kInfBits = 0x7F800000u;

// E8M0 byte of a block from the bits of its largest magnitude: the least e
// with amax <= 448 * 2^e, as e + 127 in 0 .. 254; 255 (NaN) for a block that
// holds an infinity or a NaN. 448 = 1.75 * 2^8, so the exponent goes up by
// one where the mantissa is above 1.75 (0x600000): one addition that carries
// into the exponent. The rule of MXFP4 here (floor(log2 amax) - emax) would
// let magnitudes in (448, 512) * 2^e saturate, up to 12.5 % off; this one
// never saturates, at the cost of one bit of range in the blocks it moves.
__device__ __forceinline__ uint32_t mx8_scale_byte(uint32_t amax_bits) {
  if (amax_bits >= kInfBits) return 255u;
  const int e = (int)((amax_bits + 0x1FFFFFu) >> 23) - 8;
  return e < 0 ? 0u : (uint32_t)e;
}
// 2^-(byte - 127) for bytes 0 .. 254 (byte 254 cannot come from finite fp32:
// the largest is 247, so the result is never below 2^-120).
__device__ __forceinline__ float mx8_inverse(uint32_t byte) {
  return __builtin_bit_cast(float, (254u - byte) << 23);
}
// 2^(byte - 127); byte 0 is the subnormal 2^-127, byte 255 a NaN.
__device__ __forceinline__ float mx8_scale(uint32_t byte) {
  const uint32_t b = byte == 0 ? 0x00400000u : byte == 255 ? 0x7FC00000u : byte << 23;
  return __builtin_bit_cast(float, b);
}
// 8 codes' values under the scale s.
__device__ __forceinline__ void mx8_unpack8(u32x2 w, float s, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[j], false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[j], true);
    v[4 * j] = lo[0] * s;
    v[4 * j + 1] = lo[1] * s;
    v[4 * j + 2] = hi[0] * s;
    v[4 * j + 3] = hi[1] * s;
  }
}
__device__ __forceinline__ void RawMx8::get(float (&v)[8], int64_t c, int64_t cols) const {
  const bool in = c < cols;
  mx8_unpack8(in ? w : u32x2{0, 0}, in ? mx8_scale(byte) : 0.0f, v);
}
// Four E4M3 codes of v / 2^e, nearest even (hardware conversion; the scaled
// magnitudes are at most 448). A block with byte 255 gets NaN codes.
__device__ __forceinline__ uint32_t mx8_pack4(const float* v, float inv, bool nan) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * inv, v[1] * inv, 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(v[2] * inv, v[3] * inv, w, true);
  return nan ? 0x7F7F7F7Fu : (uint32_t)w;
}
// 8 values of a lane, four lanes to a block: writes the codes and (one lane
// of the four) the block's scale byte.
__device__ __forceinline__ void mx8_store_quad(const float (&v)[8], uint8_t* codes, uint8_t* scale) {
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = abs_bits(v[i]);
    a = a > b ? a : b;
  }
  const uint32_t byte = mx8_scale_byte(quad_max(a));
  const bool nan = byte == 255u;
  const float inv = mx8_inverse(nan ? 127u : byte);
  u32x2 w = {mx8_pack4(v, inv, nan), mx8_pack4(v + 4, inv, nan)};
  __builtin_memcpy(codes, &w, 8);
  if ((threadIdx.x & 3) == 0) *scale = (uint8_t)byte;
}

// ---- activations ------------------------------------------------------------
// enum values of adahop_act.
constexpr int kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4;
constexpr float kSqrt8OverPi = 1.5957691216057308f, kGeluA = 0.044715f;

// 1 / (1 + exp(-t)): exp overflows to infinity for very negative t, and the
// reciprocal is then 0.
__device__ __forceinline__ float sigmoid(float t) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * t));
}
// t limited to [-32, 32], where every activation's slope has reached 0 or 1
// (squares and cubes beyond would overflow); a NaN stays a NaN.
__device__ __forceinline__ float bounded(float t) {
  return t < -32.0f ? -32.0f : (t > 32.0f ? 32.0f : t);
}

// Phi(z), the normal distribution function, without branches: erfc(x) =
// exp(-x^2) q(t) with x = |z| / sqrt(2), t = 1 / (1 + 0.4 x) and q the
// polynomial t (c0 + .. + c7 t^7) of least relative error on 0 <= x <= 5.5
// (fitted here: 7e-8, with fp32's roundings 4e-7). *density: exp(-z^2 / 2).
__device__ __forceinline__ float normal_cdf(float z, float* density) {
  const float a = __builtin_fabsf(z);
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.28284271247461903f, a, 1.0f));
  float q = 0.07073937356472015f;
  q = __builtin_fmaf(q, t, -0.3785628080368042f);
  q = __builtin_fmaf(q, t, 0.6544638276100159f);
  q = __builtin_fmaf(q, t, -0.34386175870895386f);
  q = __builtin_fmaf(q, t, 0.39126431941986084f);
  q = __builtin_fmaf(q, t, 0.14554718136787415f);
  q = __builtin_fmaf(q, t, 0.23538021743297577f);
  q = __builtin_fmaf(q, t, 0.2250295728445053f);
  const float e = __builtin_amdgcn_exp2f(-0.7213475204444817f * z * z);
  *density = e;
  const float tail = 0.5f * (q * t) * e;
  return z < 0.0f ? tail : 1.0f - tail;
}

template <int Act>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (Act == kActRelu) return z < 0.0f ? 0.0f : z;
  if constexpr (Act == kActSilu) return z * sigmoid(z);
  if constexpr (Act == kActGelu) {
    float e;
    return z * normal_cdf(z, &e);
  }
  // 1/2 (1 + tanh u) = sigmoid(2 u)
  if constexpr (Act == kActGeluTanh) {
    const float t = bounded(z);
    return z * sigmoid(kSqrt8OverPi * (t + kGeluA * t * t * t));
  }
  return z;
}

// The activation's value and slope at z.
template <int Act>
__device__ __forceinline__ void act_both(float z, float* value, float* slope) {
  if constexpr (Act == kActRelu) {
    *value = z < 0.0f ? 0.0f : z;
    *slope = z > 0.0f ? 1.0f : 0.0f;
  } else if constexpr (Act == kActSilu) {
    const float s = sigmoid(z), t = bounded(z);
    *value = z * s;
    *slope = s + t * s * (1.0f - s);
  } else if constexpr (Act == kActGelu) {
    float e;
    const float t = bounded(z), cdf = normal_cdf(t, &e);
    *value = z * cdf;
    *slope = cdf + t * 0.3989422804014327f * e;
  } else if constexpr (Act == kActGeluTanh) {
    const float t = bounded(z);
    const float p = sigmoid(kSqrt8OverPi * (t + kGeluA * t * t * t));
    *value = z * p;
    *slope = p + t * p * (1.0f - p) * kSqrt8OverPi * (1.0f + 3.0f * kGeluA * t * t);
  } else {
    *value = z;
    *slope = 1.0f;
  }
}

}  // namespace mx8
}  // namespace adahop
