// Rows of bf16 / fp32 elements and of the storage formats, eight elements at a time: what the
// kernels of rows.hip and norm.hip share.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>

#include "common.h"
#include "launch.h"

namespace hk {

typedef unsigned u32x2 __attribute__((ext_vector_type(2)));

// Workgroups along the rows: one per `per` rows, at most 2^21 (a launch holds
// fewer than 2^32 threads); the kernels walk the rest in steps of so many.
constexpr int64_t kMostBlocks = int64_t(1) << 21;
inline unsigned row_blocks(int64_t n, int64_t per) {
  return (unsigned)std::min<int64_t>((n + per - 1) / per, kMostBlocks);
}

inline int rows_bytes(int dtype) { return dtype == kRowsBF16 ? 2 : 4; }

inline bool aligned16(const void* p, int64_t ts, int64_t hs, int dtype) {
  const int64_t b = rows_bytes(dtype);
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ts * b % 16 == 0 && hs * b % 16 == 0;
}

// ------------------------------------------------------- element access

__device__ __forceinline__ float bf16_float(uint32_t bits) { return __uint_as_float(bits << 16); }

// Two floats rounded to bf16 (to nearest, ties to even), a in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  bf16x2 v;
  v[0] = (__bf16)a;
  v[1] = (__bf16)b;
  return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ void unpack_bf16(const u32x4& v, float* o) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[2 * i] = bf16_float(v[i] & 0xffffu);
    o[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
  }
}

// Eight consecutive elements as stored; VEC: 16-byte aligned.
template <int DT>
struct Raw8 {
  u32x4 w[DT == kRowsBF16 ? 1 : 2];

  __device__ __forceinline__ void zero() {
    for (u32x4& x : w) x = u32x4{0u, 0u, 0u, 0u};
  }
  template <bool VEC>
  __device__ __forceinline__ void load(const void* base, int64_t at) {
    if constexpr (DT == kRowsBF16) {
      const uint16_t* p = static_cast<const uint16_t*>(base) + at;
      if constexpr (VEC) {
        w[0] = *reinterpret_cast<const u32x4*>(p);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[0][i] = (uint32_t)p[2 * i] | ((uint32_t)p[2 * i + 1] << 16);
      }
    } else {
      const uint32_t* p = static_cast<const uint32_t*>(base) + at;
      if constexpr (VEC) {
        w[0] = *reinterpret_cast<const u32x4*>(p);
        w[1] = *reinterpret_cast<const u32x4*>(p + 4);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i >> 2][i & 3] = p[i];
      }
    }
  }
  __device__ __forceinline__ void floats(float* o) const {
    if constexpr (DT == kRowsBF16) {
      unpack_bf16(w[0], o);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = __uint_as_float(w[i >> 2][i & 3]);
    }
  }
  // The signs flipped where `flip` is all ones.
  __device__ __forceinline__ void negate(uint32_t flip) {
    const uint32_t m = flip & (DT == kRowsBF16 ? 0x80008000u : 0x80000000u);
    for (u32x4& x : w) x ^= u32x4{m, m, m, m};
  }
  // What another lane of the wave holds.
  __device__ __forceinline__ Raw8 of_lane(int lane) const {
    Raw8 r;
#pragma unroll
    for (unsigned i = 0; i < sizeof(w) / sizeof(w[0]); ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        r.w[i][j] = (uint32_t)__builtin_amdgcn_ds_bpermute(lane * 4, (int)w[i][j]);
    return r;
  }
};

// Eight consecutive elements as floats.
template <int DT, bool VEC>
__device__ __forceinline__ void load8(const void* base, int64_t at, float* o) {
  if constexpr (DT == kRowsBF16) {
    const uint16_t* p = static_cast<const uint16_t*>(base) + at;
    if constexpr (VEC) {
      unpack_bf16(*reinterpret_cast<const u32x4*>(p), o);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = bf16_float(p[i]);
    }
  } else {
    const float* p = static_cast<const float*>(base) + at;
    if constexpr (VEC) {
      const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) { o[i] = a[i]; o[4 + i] = b[i]; }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = p[i];
    }
  }
}

template <int DT>
__device__ __forceinline__ float load1(const void* base, int64_t at) {
  if constexpr (DT == kRowsBF16) return bf16_float(static_cast<const uint16_t*>(base)[at]);
  else return static_cast<const float*>(base)[at];
}

// Eight elements to 16-byte aligned memory; PAST: not kept in the caches.
template <int DT, bool PAST = false>
__device__ __forceinline__ void store8(void* base, int64_t at, const float* v) {
  auto put = [](void* p, const u32x4& w) {
    if constexpr (PAST) __builtin_nontemporal_store(w, static_cast<u32x4*>(p));
    else *static_cast<u32x4*>(p) = w;
  };
  u32x4 w;
  if constexpr (DT == kRowsBF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    put(static_cast<uint16_t*>(base) + at, w);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(v[4 * h + i]);
      put(static_cast<float*>(base) + at + 4 * h, w);
    }
  }
}

template <int DT>
__device__ __forceinline__ void store1(void* base, int64_t at, float v) {
  if constexpr (DT == kRowsBF16)
    static_cast<uint16_t*>(base)[at] = (uint16_t)(pack_bf16(v, 0.0f) & 0xffffu);
  else
    static_cast<float*>(base)[at] = v;
}

// ------------------------------------------------------ storage formats

typedef short short2v __attribute__((ext_vector_type(2)));

// Four values of at most 448 (or what rounds to it) as E4M3 bytes, to nearest, ties to even.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

// The scale of an FP8 row whose largest magnitude is m: max(m / 448, 2^-126), 1 for a row of zeros.  The quotient is rounded
// as a division's: a product with the rounded 1 / 448 and one correction by the exact remainder (all 2^23
// significands compared with the division's).  An infinite m has no remainder, and its scale is infinite, so that the whole row reads as
// NaN: it comes from the product less 2^-20 of it, which is below every other quotient.
__device__ __forceinline__ float e4m3_scale(float m) {
  constexpr float kInv = 1.0f / 448.0f;
  const float q = m * kInv;
  return m > 0.0f ? fmaxf(fmaxf(fmaf(fmaf(-448.0f, q, m), kInv, q), 0x1p-126f), m * (kInv * (1.0f - 0x1p-20f))) : 1.0f;
}

// The E4M3 bytes of four exact quotients x / scale.  `below` and `above` are 1 / scale less and plus 2^-21 of it, so x
// times them lies on either side of the quotient, and its code is one of the two's.  Where they differ, the quotient
// lies near the tie between them, half of a + b: x - (a + b) / 2 scale, one fused operation, has the exact difference's sign
// (rows far below 1 are raised by 2^64 first, so that none is lost below the smallest number).  Rows of bf16 meet ties often:
// where the largest's significand is a multiple of 7, one element in some thirty.
struct Reciprocal {
  float scale, below, above;
  __device__ __forceinline__ explicit Reciprocal(float s) : scale(s) {
    const float inv = __builtin_amdgcn_rcpf(s);  // within 2^-23 of it, each of the two products within 2^-24
    below = inv * (1.0f - 0x1p-21f);
    above = inv * (1.0f + 0x1p-21f);
  }
};
__device__ __forceinline__ uint32_t e4m3x4_quotient(const float* x, const Reciprocal& r) {
  const uint32_t lo = e4m3x4(x[0] * r.below, x[1] * r.below, x[2] * r.below, x[3] * r.below);
  const uint32_t hi = e4m3x4(x[0] * r.above, x[1] * r.above, x[2] * r.above, x[3] * r.above);
  if (lo == hi) return lo;
  const float raise = r.scale < 1.0f ? 0x1p64f : 1.0f, half = r.scale * raise * 0.5f;
  auto pair = [](uint32_t codes, int i) {
    return i == 0 ? __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, false) : __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, true);
  };
  uint32_t take = 0;  // the bytes of `hi` that are taken
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const auto a = pair(lo, i), b = pair(hi, i);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float over = fmaf(-(a[j] + b[j]), half, x[i + j] * raise);
      // beyond the tie, or on it with an odd code below
      const bool up = over == 0.0f ? (lo >> (8 * (i + j))) & 1u : (__float_as_uint(over) ^ __float_as_uint(x[i + j])) >> 31 == 0;
      take |= up ? 0xffu << (8 * (i + j)) : 0u;
    }
  }
  return lo ^ ((lo ^ hi) & take);
}

// The exponent that a block of an MX format shares, where m is its largest magnitude: floor(log2(m)) less the
// largest element's, clamped (frexp's exponent is floor(log2(m)) + 1); 2^-127 for a block of zeros.
template <int FMT>
__device__ __forceinline__ int mx_exponent(float m) {
  const int x = __builtin_amdgcn_frexp_expf(m) - 1 - (FMT == kMXFP8 ? 8 : 2);
  return m > 0.0f ? max(-127, min(127, x)) : -127;
}

// Eight values over 2^e as E4M3 bytes; what lies over 448 would turn to NaN and saturates first.
__device__ __forceinline__ u32x2 mx_e4m3x8(const float* y, int e) {
  const float by = __uint_as_float((unsigned)(e + 127) << 23);  // the conversions divide by this: the scale's exponent in an fp32
  const float top = ldexpf(448.0f, e);
  u32x2 w;
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    float z[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) z[j] = __builtin_amdgcn_fmed3f(y[4 * p + j], -top, top);
    short2v t = {0, 0};
    t = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(t, z[0], z[1], by, false);
    t = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(t, z[2], z[3], by, true);
    w[p] = __builtin_bit_cast(uint32_t, t);
  }
  return w;
}

// Eight values over 2^e as E2M1 nibbles; the conversion saturates by itself.
__device__ __forceinline__ uint32_t mx_e2m1x8(const float* y, int e) {
  const float by = __uint_as_float((unsigned)(e + 127) << 23);
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[0], y[1], by, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[2], y[3], by, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[4], y[5], by, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[6], y[7], by, 3);
}

// Eight elements of a cache row, as stored.
template <int FMT>
struct Stored8 {
  u32x4 w;    // bf16 uses all four words, E4M3 two, E2M1 one
  float s;    // FP8: the row's scale
  unsigned b;  // MX: the block's scale byte

  // e0: the first element's place in the cache, of row `row`.
  __device__ __forceinline__ void load(const uint8_t* codes, const void* scale, int64_t row, int64_t e0) {
    if constexpr (FMT == kBF16) {
      w = *reinterpret_cast<const u32x4*>(codes + e0 * 2);
    } else if constexpr (FMT == kMXFP4) {
      w[0] = *reinterpret_cast<const uint32_t*>(codes + (e0 >> 1));
    } else {
      const u32x2 t = *reinterpret_cast<const u32x2*>(codes + e0);
      w[0] = t[0];
      w[1] = t[1];
    }
    if constexpr (FMT == kFP8) s = static_cast<const float*>(scale)[row];
    if constexpr (FMT == kMXFP8 || FMT == kMXFP4) b = static_cast<const uint8_t*>(scale)[e0 >> 5];
  }

  __device__ __forceinline__ void decode(float* o) const {
    if constexpr (FMT == kBF16) {
      unpack_bf16(w, o);
    } else if constexpr (FMT == kFP8) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false);
        const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
        o[4 * i] = lo[0] * s;
        o[4 * i + 1] = lo[1] * s;
        o[4 * i + 2] = hi[0] * s;
        o[4 * i + 3] = hi[1] * s;
      }
    } else {
      const float by = __uint_as_float(b << 23);  // 2^(b - 127): the conversions multiply by it
      if constexpr (FMT == kMXFP8) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const auto lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[i], by, false);
          const auto hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[i], by, true);
          o[4 * i] = lo[0];
          o[4 * i + 1] = lo[1];
          o[4 * i + 2] = hi[0];
          o[4 * i + 3] = hi[1];
        }
      } else {
        const auto p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[0], by, 0);
        const auto p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[0], by, 1);
        const auto p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[0], by, 2);
        const auto p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[0], by, 3);
        o[0] = p0[0]; o[1] = p0[1]; o[2] = p1[0]; o[3] = p1[1];
        o[4] = p2[0]; o[5] = p2[1]; o[6] = p3[0]; o[7] = p3[1];
      }
      if (b == 255u) {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = __builtin_nanf("");
      }
    }
  }
};

// ------------------------------------------------- across a row's lanes

// The largest of m over groups of P neighbouring lanes (4 <= P <= 64): quads and
// rows of 16 by lane permutations inside the vector instruction.
template <int CTRL>
__device__ __forceinline__ float max_dpp(float m) {
  return fmaxf(m, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(m), CTRL, 0xf, 0xf, true)));
}
__device__ __forceinline__ float quad_max(float m) {
  return max_dpp<0x4e>(max_dpp<0xb1>(m));  // neighbours, then pairs of neighbours
}
__device__ __forceinline__ float lanes_max(float m, int P) {
  m = quad_max(m);
  if (P > 4) m = max_dpp<0x141>(m);  // the other quad of eight lanes (mirrored)
  if (P > 8) m = max_dpp<0x140>(m);  // the other eight of sixteen
  if (P > 16) m = fmaxf(m, __shfl_xor(m, 16));
  if (P > 32) m = fmaxf(m, __shfl_xor(m, 32));
  return m;
}

}  // namespace hk
