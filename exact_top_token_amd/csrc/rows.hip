// Rows on their way into and out of the selection: rotary positions, and the
// four storage formats of q and k written from and read back to bf16 / fp32
// rows.  Every kernel here moves each row once and is bound by memory.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "common.h"
#include "launch.h"

namespace hk {

namespace {

constexpr int kRowThreads = 256;  // threads of a workgroup (a write of long rows takes up to 1,024)

typedef unsigned u32x2 __attribute__((ext_vector_type(2)));

// Workgroups along the rows: one per `per` rows, at most 2^21 (a launch holds
// fewer than 2^32 threads); the kernels walk the rest in steps of so many.
constexpr int64_t kMostBlocks = int64_t(1) << 21;
unsigned row_blocks(int64_t n, int64_t per) {
  return (unsigned)std::min<int64_t>((n + per - 1) / per, kMostBlocks);
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

// ------------------------------------------------------------- rotation

// Quarter turns a position, less whole turns (positions are whole numbers), as a sum of two doubles: one double's
// rounding, times 2^31 positions, would be 2^-24 of a turn.
struct Turns {
  double hi, lo;
  __device__ __forceinline__ explicit Turns(double freq) {  // radians a position
#pragma clang fp contract(off)  // t is the rounded product wherever it stands
    constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;  // 1 / (2 pi)
    const double t = freq * kHi;
    lo = 4.0 * fma(freq, kLo, fma(freq, kHi, -t));
    hi = 4.0 * (t - rint(t));
  }
};

// Cosine and sine of q + r quarter turns, |r| <= 1/2 (or what rounds to it).  sin(pi/2 r) = r (pi/2 + P(r^2)) and
// cos(pi/2 r) = 1 + r^2 Q(r^2), P and Q interpolated at the Chebyshev nodes of [0, 1/4] (off by 2.4e-9 and 2e-10;
// pi/2 is rounded to fp32 and P holds the rest); q swaps and signs the two.
__device__ __forceinline__ float2 turn_cos_sin(int q, float r) {
  const float z = r * r;
  float s = fmaf(z, -0.004602149128913879f, 0.07968021929264069f);
  s = fmaf(z, s, -0.6459634900093079f);
  s = fmaf(z, s, -4.8553051357203e-08f);
  s = fmaf(r, 1.5707963705062866f, r * s);
  float c = fmaf(z, 0.0009067399078048766f, -0.02086152881383896f);
  c = fmaf(z, c, 0.253669410943985f);
  c = fmaf(z, c, -1.2337005138397217f);
  c = fmaf(z, c, 1.0f);
  const float cc = q & 1 ? s : c, ss = q & 1 ? c : s;
  return make_float2(__uint_as_float(__float_as_uint(cc) ^ (((unsigned)(q + 1) & 2u) << 30)),
                     __uint_as_float(__float_as_uint(ss) ^ (((unsigned)q & 2u) << 30)));
}

// (gain cos, turn sin) at position pos.  The angle is formed in 64 bits and reduced to the nearest quarter turn
// there, so that at any int32 position its rounding to fp32 is 2^-28 of a turn.  1.5 * 2^52 more leaves
// a number of quarter turns below 2^33 rounded to a whole one, its last 32 bits the sum's.
__device__ __forceinline__ float2 rot_entry(const RotArgs& r, const Turns& f, int pos) {
  constexpr double kWhole = 6755399441055744.0;
  const double p = (double)pos, n = fma(p, f.hi, kWhole);
  const double rest = fma(p, f.lo, fma(p, f.hi, kWhole - n));
  const float2 c = turn_cos_sin((int)__double_as_longlong(n), (float)rest);
  return make_float2(c.x * r.gain, c.y * r.turn);
}

// One half of a rotated pair: v cos -+ w sin.  Written as one product and one fused
// step, so that every path (alignment, layout, on its way into a cache) gives
// the same bits.
__device__ __forceinline__ float rot_lo(float v, float w, float2 f) { return fmaf(v, f.x, -(w * f.y)); }
__device__ __forceinline__ float rot_hi(float v, float w, float2 f) { return fmaf(v, f.x, w * f.y); }

// u / by for u * by < 2^22 (the error of the rounded-up reciprocal stays below 1 / by).
struct SmallDiv {
  unsigned by, mul;
  __host__ __device__ SmallDiv(unsigned d, unsigned m) : by(d), mul(m) {}
  __host__ explicit SmallDiv(unsigned d) : SmallDiv(d, ((1u << 22) + d - 1) / d) {}
  __device__ __forceinline__ unsigned operator()(unsigned u) const {
    return (unsigned)(((uint64_t)u * mul) >> 22);
  }
};

// A token's entries in LDS, [dim/2] float2.  With 16-byte access a thread reads W pairs at
// once (eight of the half layout, four of the interleaved one), two to a 16-byte read: pair
// 2 j + b of unit u lies in the (j * units + u)-th 16 bytes, so that neighbouring threads
// read neighbouring pieces without bank conflicts (in plain order their 64-byte steps met
// in the same banks, and the LDS bounded the quantised write: 66 us of 8,192 x 64 x 128).
template <int W>
__device__ __forceinline__ int rot_slot(int i, int half) {
  if constexpr (W == 1) return i;
  const int u = i / W, w = i % W;
  return 2 * ((w >> 1) * (half / W) + u) + (w & 1);
}
template <int W>
__device__ __forceinline__ void rot_read(const float2* cs, int half, int u, float2* f) {
  const f32x4* p = reinterpret_cast<const f32x4*>(cs) + u;
#pragma unroll
  for (int j = 0; j < W / 2; ++j) {
    const f32x4 v = p[j * (half / W)];
    f[2 * j] = make_float2(v[0], v[1]);
    f[2 * j + 1] = make_float2(v[2], v[3]);
  }
}

// The entries of tokens t0 .. t0 + nt - 1, once for all their heads: [nt][dim/2]
// (at most 2,048 entries, or one token's).
template <int W>
__device__ __forceinline__ void rot_table(const RotArgs& r, int64_t t0, int nt, int threads, float2* cs) {
  const int half = r.dim >> 1;
  // a thread keeps its pair, whose frequency it loads once, and walks over tokens
  const int cols = min(half, threads), steps = threads / cols;
  const int first = threadIdx.x / cols;
  if (first >= steps) return;
  for (int i = threadIdx.x - first * cols; i < half; i += cols) {
    const Turns f(r.freq[i]);
    float2* to = cs + rot_slot<W>(i, half);
    for (int t = first; t < nt; t += steps) {
      const int pos = r.pos ? r.pos[t0 + t] : r.pos0 + (int)t0 + t;  // below 2^31
      to[t * half] = rot_entry(r, f, pos);
    }
  }
}

}  // namespace

// Rotary positions: y = rotation of x, elements outside the rotated part copied.
// A workgroup takes `tb` tokens by `hb` heads and computes the tokens'
// cosines and sines once, in LDS, for all those heads.  A thread keeps one
// unit of the head (its pairs) and walks over (token, head) rows.  A unit is, with 16-byte
// access (VEC), eight pairs of the half layout (two 16-byte pieces), four pairs of
// the interleaved one, or eight elements outside the rotated part; else one pair or one element.
struct RotaryGrid {
  uint16_t tb, hb;    // tokens and heads of a workgroup: at most 1,024 and 32,768
  uint16_t units;     // units of a head, at most 256
  uint16_t rows;      // (token, head) rows in flight: threads / units
};
static_assert(sizeof(RotaryArgs) + sizeof(RotaryGrid) <= 112, "launches");

namespace {

template <int IN, int OUT, int LAYOUT, bool VEC>
__global__ void __launch_bounds__(kRowThreads) rotary_kernel(RotaryArgs a, RotaryGrid g) {
  extern __shared__ __attribute__((aligned(16))) float2 cs[];
  const RotArgs& r = a.rot;
  const int half = r.dim >> 1;
  const int h0 = blockIdx.y * g.hb, nh = min((int)g.hb, a.heads - h0);
  const int ts = g.rows / nh, hs = g.rows - ts * nh;
  constexpr int W = VEC ? 8 : 1;                            // elements of a copy unit
  constexpr int PW = VEC ? (LAYOUT == kRotHalf ? 8 : 4) : 1;  // pairs of a rotated unit
  const int nrot = half / PW;
  for (int64_t tile = blockIdx.x; tile * g.tb < a.n; tile += kMostBlocks) {
    const int t0 = (int)(tile * g.tb), nt = min((int)g.tb, a.n - t0);
    if (tile != blockIdx.x) __syncthreads();  // the last tile's entries are read
    rot_table<PW>(r, t0, nt, kRowThreads, cs);
    __syncthreads();
    // Units wider than the workgroup (heads of many elements without 16-byte
    // access) are walked in steps of the workgroup.
    for (int u = threadIdx.x % g.units; u < nrot + (a.d - r.dim) / W; u += kRowThreads) {
      int row = threadIdx.x / g.units;
      if (row >= g.rows) break;
      const bool rot = u < nrot;
      int e;  // the unit's first element in the head
      if (rot) {
        e = a.first + (LAYOUT == kRotHalf ? u * PW : 2 * u * PW);
      } else {
        e = (u - nrot) * W;
        if (e >= a.first) e += r.dim;
      }
      int t = row / nh, h = row - t * nh;
      while (t < nt) {
        const int64_t xi = (int64_t)(t0 + t) * a.xts + (int64_t)(h0 + h) * a.xhs + e;
        const int64_t yi = (int64_t)(t0 + t) * a.yts + (int64_t)(h0 + h) * a.yhs + e;
        if constexpr (VEC) {
          float v[8];
          load8<IN, true>(a.x, xi, v);
          if (rot) {
            float2 c[8];
            rot_read<PW>(cs + t * half, half, u, c);
            if constexpr (LAYOUT == kRotHalf) {
              float w[8];
              load8<IN, true>(a.x, xi + half, w);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float2 f = c[i];
                const float p = v[i], q = w[i];
                v[i] = rot_lo(p, q, f);
                w[i] = rot_hi(q, p, f);
              }
              store8<OUT>(a.y, yi + half, w);
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float2 f = c[i];
                const float p = v[2 * i], q = v[2 * i + 1];
                v[2 * i] = rot_lo(p, q, f);
                v[2 * i + 1] = rot_hi(q, p, f);
              }
            }
          }
          store8<OUT>(a.y, yi, v);
        } else {
          const float p = load1<IN>(a.x, xi);
          if (rot) {
            const int off = LAYOUT == kRotHalf ? half : 1;
            const float2 f = cs[t * half + u];
            const float q = load1<IN>(a.x, xi + off);
            store1<OUT>(a.y, yi, rot_lo(p, q, f));
            store1<OUT>(a.y, yi + off, rot_hi(q, p, f));
          } else {
            store1<OUT>(a.y, yi, p);
          }
        }
        t += ts;
        h += hs;
        if (h >= nh) { h -= nh; ++t; }
      }
    }
  }
}

template <int IN, int OUT>
hipError_t rotary_io(const RotaryArgs& a, int layout, bool vec, hipStream_t s) {
  const RotArgs& r = a.rot;
  const int pw = vec ? (layout == kRotHalf ? 8 : 4) : 1, w = vec ? 8 : 1;
  const int units = std::min(r.dim / 2 / pw + (a.d - r.dim) / w, kRowThreads);
  const int rows = kRowThreads / units;
  // Four rows a thread where that leaves 512 workgroups or more, else one: 8,192 x 64 x 128 53 us
  // against 66, 1,000 x 64 x 128 8.4 against 9.7, but 300 x 64 x 128 5.0 against 4.6.
  const int64_t rows_all = (int64_t)a.n * a.heads;
  const int per = rows_all / (4 * rows) >= 512 ? 4 * rows : rows;
  int hb = std::min(a.heads, per), tb = 1;
  if ((a.heads + hb - 1) / hb > 65535) hb = (a.heads + 65534) / 65535;
  if (hb == a.heads) {
    const int lds_tokens = std::max(1, 2048 / (r.dim / 2));  // at most 16 KiB of entries
    tb = std::max(1, std::min(per / a.heads, lds_tokens));
  }
  const RotaryGrid g{(uint16_t)tb, (uint16_t)hb, (uint16_t)units, (uint16_t)rows};
  const dim3 grid(row_blocks(a.n, tb), (unsigned)((a.heads + hb - 1) / hb));
  const size_t lds = (size_t)tb * (r.dim / 2) * sizeof(float2);
  if (layout == kRotHalf) {
    if (vec) hipLaunchKernelGGL((rotary_kernel<IN, OUT, kRotHalf, true>), grid, dim3(kRowThreads), lds, s, a, g);
    else hipLaunchKernelGGL((rotary_kernel<IN, OUT, kRotHalf, false>), grid, dim3(kRowThreads), lds, s, a, g);
  } else {
    if (vec) hipLaunchKernelGGL((rotary_kernel<IN, OUT, kRotInterleaved, true>), grid, dim3(kRowThreads), lds, s, a, g);
    else hipLaunchKernelGGL((rotary_kernel<IN, OUT, kRotInterleaved, false>), grid, dim3(kRowThreads), lds, s, a, g);
  }
  return hipGetLastError();
}

int rows_bytes(int dtype) { return dtype == kRowsBF16 ? 2 : 4; }

bool aligned16(const void* p, int64_t ts, int64_t hs, int dtype) {
  const int64_t b = rows_bytes(dtype);
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ts * b % 16 == 0 && hs * b % 16 == 0;
}

// Whether the units of 16-byte access tile the head: pieces of eight elements
// that lie wholly inside or outside the rotated part (and, in the half layout,
// inside one half of it).
bool rot_in_eights(int dim, int first, int layout, int d) {
  return d % 8 == 0 && first % 8 == 0 && dim % (layout == kRotHalf ? 16 : 8) == 0;
}

}  // namespace

hipError_t launch_rotary(const RotaryArgs& a, int layout, int in_dtype, int out_dtype, hipStream_t s) {
  if (a.n <= 0) return hipSuccess;
  const bool vec = rot_in_eights(a.rot.dim, a.first, layout, a.d) && aligned16(a.x, a.xts, a.xhs, in_dtype) &&
                   aligned16(a.y, a.yts, a.yhs, out_dtype);
  if (in_dtype == kRowsBF16) {
    return out_dtype == kRowsBF16 ? rotary_io<kRowsBF16, kRowsBF16>(a, layout, vec, s)
                                  : rotary_io<kRowsBF16, kRowsFP32>(a, layout, vec, s);
  }
  return out_dtype == kRowsBF16 ? rotary_io<kRowsFP32, kRowsBF16>(a, layout, vec, s)
                                : rotary_io<kRowsFP32, kRowsFP32>(a, layout, vec, s);
}

// --------------------------------------------------------- cache writing

namespace {

typedef short short2v __attribute__((ext_vector_type(2)));

// Four values of at most 448 (or what rounds to it) as E4M3 bytes, to nearest, ties to even.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

// x / scale with an inexact result's last bit set: rounding that to a short
// format equals rounding the exact quotient (the 64-bit quotient of two 24-bit
// numbers cannot round onto a tie of fewer bits unless it is one).
__device__ __forceinline__ float quotient_odd(float x, float scale) {
  const double q = (double)x / (double)scale;
  const float f = (float)q;
  const double df = (double)f;
  if (df == q || !isfinite(f)) return f;
  uint32_t u = __float_as_uint(f);
  if (fabs(df) > fabs(q)) --u;  // toward zero
  return __uint_as_float(u | 1u);
}

// The E4M3 bytes of four exact quotients x / scale.  x * inv is within 2^-22
// of the quotient; only where the codes of its two ends differ, near a tie, is the
// quotient formed in 64 bits.
__device__ __forceinline__ uint32_t e4m3x4_quotient(const float* x, float scale, float inv) {
  constexpr float kLo = 1.0f - 0x1p-22f, kHi = 1.0f + 0x1p-22f;
  float q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = x[i] * inv;
  const uint32_t lo = e4m3x4(q[0] * kLo, q[1] * kLo, q[2] * kLo, q[3] * kLo);
  const uint32_t hi = e4m3x4(q[0] * kHi, q[1] * kHi, q[2] * kHi, q[3] * kHi);
  if (lo == hi) return lo;
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = quotient_odd(x[i], scale);
  return e4m3x4(q[0], q[1], q[2], q[3]);
}

// A thread's eight elements e0 .. e0 + 7 of a head, on one side of every border of the rotation.
struct Eight {
  bool in;        // in the rotated part
  uint32_t flip;  // half layout: all ones in its first half, whose partners count negative
  int other;      // half layout: how far the partners lie
  int unit;       // its entries in LDS

  template <int LAYOUT>
  __device__ __forceinline__ void place(int dim, int first, int e0) {
    const int half = dim >> 1, e = e0 - first;
    in = e >= 0 && e < dim;
    const bool lo = e < half;
    flip = lo ? ~0u : 0u;
    other = lo ? half : -half;
    unit = LAYOUT == kRotHalf ? (lo ? e : e - half) >> 3 : e >> 3;
  }
};

// Rotated values of eight elements v; w: their partners of the half layout, signed; f: the
// entries of the unit.
template <int LAYOUT>
__device__ __forceinline__ void rotate_eight(const float* w, const float2* f, float* v) {
  if constexpr (LAYOUT == kRotHalf) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = fmaf(v[i], f[i].x, w[i] * f[i].y);  // rot_lo or rot_hi
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float p = v[2 * i], q = v[2 * i + 1];
      v[2 * i] = rot_lo(p, q, f[i]);
      v[2 * i + 1] = rot_hi(q, p, f[i]);
    }
  }
}

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

// The same one element at a time, for any rotated part and alignment (cs: the token's entries in
// plain order).
template <int IN>
__device__ __forceinline__ void rotate_each(int dim, int first, bool halves, const void* x, int64_t at, int e0,
                                            const float2* cs, float* v) {
  const int half = dim >> 1;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = e0 - first + i;
    if (e < 0 || e >= dim) continue;
    const bool lo = halves ? e < half : (e & 1) == 0;
    const int off = halves ? half : 1;
    const float2 f = cs[halves ? (lo ? e : e - half) : e >> 1];
    const float w = load1<IN>(x, at + e0 + i + (lo ? off : -off));
    v[i] = lo ? rot_lo(v[i], w, f) : rot_hi(v[i], w, f);
  }
}

// How the rows of a write lie on threads: P = 1 << log_p threads take a row, a
// workgroup takes `rounds` times 256 / P rows at once.
struct WriteGrid {
  uint32_t pieces : 10;  // of eight elements of a head, less one
  uint32_t heads : 8;    // less one
  uint32_t log_p : 4;
  uint32_t rounds : 3;
  uint32_t near : 1;     // no head straddles two waves: partners are a lane's to give
  uint32_t halves : 1;   // the layout, for rows without 16-byte access
  uint32_t mul;          // SmallDiv of a head's pieces
};
static_assert(sizeof(CacheWriteArgs) + sizeof(WriteGrid) <= 112, "launches");

constexpr int kMaxWriteThreads = 1024;
constexpr int kWriteEntries = 2048;  // cosines and sines of a workgroup's rows

// Rows written into a cache.  P threads (a power of two, 4..256; up to 1,024 for FP8) take
// a row in pieces of eight elements, K of them at a time, so a row is read once and its
// scale comes from registers: a reduction over the row (FP8), or over the four
// lanes of a 32-element block (MX).  K is 4 for rows of more than 256 pieces whose
// heads repeat every P pieces (`same`): a thread's pieces then share their cosines and
// sines, their place in the head and the row's set-up.  Other long rows are walked 256
// pieces at a time (FP8: 1,024 threads a row).  8,192 x 64 x 128 to MXFP4, rotated: with
// K = 4 47 us, one piece at a time 64 (bound by the instructions around the
// elements), 1,024 threads a row 65 (waiting for each other).
template <int IN, int FMT, int K, bool VEC, int LAYOUT>
__global__ void __launch_bounds__(FMT == kFP8 && K == 1 ? kMaxWriteThreads : kRowThreads)
cache_write_kernel(CacheWriteArgs a, WriteGrid g) {
  __shared__ __attribute__((aligned(16))) float2 cs[kWriteEntries];
  __shared__ float red[2][kMaxWriteThreads / kWave];
  __shared__ int later[kRowThreads / 4];
  constexpr int KV = FMT == kFP8 ? K : 1;  // pieces whose values are held at once
  const SmallDiv head(g.pieces + 1u, g.mul);
  const int log_p = g.log_p, P = 1 << log_p, threads = max(kRowThreads, P), RB = threads >> log_p;
  const int rl = threadIdx.x >> log_p;
  const int chunks = (int)((g.heads + 1u) * head.by), half = a.rot.dim >> 1;
  const int segs = (chunks + K * P - 1) / (K * P), rounds = g.rounds;  // steps of K P pieces that a row takes
  // A thread's (first) piece of the row: chunk lr, eight elements from e0 of a head, at `at` in
  // a row of x.  Piece k of K lies k P chunks and k `step` elements on.
  struct Piece {
    int lr, e0;
    int64_t at;
  };
  const int64_t step = K > 1 ? (int64_t)head(P) * a.hs : 0;
  auto piece = [&](int seg) {
    Piece p;
    p.lr = (int)(threadIdx.x & (P - 1)) + (seg << log_p);
    const unsigned h = head((unsigned)p.lr);
    p.e0 = (p.lr - (int)(h * head.by)) * 8;
    p.at = (int64_t)h * a.hs + p.e0;
    return p;
  };
  int flip = 0;
  for (int64_t i0 = (int64_t)blockIdx.x * RB * rounds; i0 < a.n; i0 += kMostBlocks * RB * rounds) {
    const int tile = (int)min((int64_t)RB * rounds, a.n - i0);
    Raw8<IN> raw[K];  // the next step's elements and slot, under way while this one is worked on
    int slot = -1;
    auto fetch = [&](const Piece& p, int r0) {
      const bool have = r0 + rl < tile;
      const int64_t at = (i0 + r0 + rl) * a.ts + p.at;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        raw[k].zero();
        if (have && p.lr + k * P < chunks) raw[k].template load<VEC>(a.x, at + k * step);
      }
      slot = -1;
      if (have) slot = a.slots ? a.slots[i0 + r0 + rl] : a.start + (int)i0 + r0 + rl;
    };
    Piece ahead = piece(0);
    fetch(ahead, 0);
    if (a.rot.freq) {
      __syncthreads();  // the last rows' entries are read
      rot_table<!VEC ? 1 : LAYOUT == kRotHalf ? 8 : 4>(a.rot, i0, tile, threads, cs);
      __syncthreads();
    }
    for (int r0 = 0, seg = 0; r0 < tile;) {
      const bool have = r0 + rl < tile;
      const int i = (int)i0 + r0 + rl;
      const Piece my = ahead;
      Raw8<IN> now[K];
#pragma unroll
      for (int k = 0; k < K; ++k) now[k] = raw[k];
      // The row's place; negative where nothing is written.
      int row = slot < a.L ? slot : -1;
      const int r1 = r0;
      if (++seg == segs) {
        seg = 0;
        r0 += RB;
      }
      if (r0 < tile) {
        if (segs > 1) ahead = piece(seg);
        fetch(ahead, r0);
      }
      if (a.claim && row >= 0 && a.claim[row] != i) row = -1;
      if (a.slots && !a.claim) {  // few rows: look for a later row of the same slot
        __syncthreads();
        if ((int)threadIdx.x < RB) later[threadIdx.x] = 0;
        __syncthreads();
        if (row >= 0) {
          bool dup = false;
          for (int j = i + 1 + (my.lr & (P - 1)); j < a.n; j += P) dup |= a.slots[j] == row;
          if (dup) later[rl] = 1;
        }
        __syncthreads();
        if (later[rl]) row = -1;
      }

      const float2* entries = cs + (have ? r1 + rl : 0) * half;
      Eight part;
      part.template place<LAYOUT>(a.rot.dim, a.first, my.e0);
      float2 f[8];
      if (VEC && a.rot.freq && part.in) rot_read<LAYOUT == kRotHalf ? 8 : 4>(entries, half, part.unit, f);
      // The k-th piece's values, rotated.
      auto values = [&](int k, float* v) {
        now[k].floats(v);
        if (!a.rot.freq) return;
        if constexpr (VEC) {
          float w[8];
          if constexpr (LAYOUT == kRotHalf) {
            Raw8<IN> other = now[k];
            if (g.near) other = now[k].of_lane(lane_id() + (part.in ? part.other / 8 : 0));
            else if (part.in && have && my.lr + k * P < chunks)
              other.template load<true>(a.x, (int64_t)i * a.ts + my.at + k * step + part.other);
            other.negate(part.flip);
            other.floats(w);
          }
          if (part.in) rotate_eight<LAYOUT>(w, f, v);
        } else if (have && my.lr + k * P < chunks) {
          rotate_each<IN>(a.rot.dim, a.first, g.halves, a.x, (int64_t)i * a.ts + my.at + k * step - my.e0, my.e0, entries, v);
        }
      };

      float v[KV][8];
      float scale = 1.0f, inv = 1.0f;
      if constexpr (FMT == kFP8) {
        float m = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
          values(k, v[k]);
#pragma unroll
          for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[k][j]));
        }
        m = lanes_max(m, P);
        if (P > kWave) {  // uniform over the launch
          float* sums = red[flip];  // the other half is read by waves still in the last round
          flip ^= 1;
          if (lane_id() == 0) sums[threadIdx.x >> 6] = m;
          __syncthreads();
          const int w0 = rl * (P / kWave);
          for (int w = 0; w < P / kWave; ++w) m = fmaxf(m, sums[w0 + w]);
        }
        scale = m > 0.0f ? fmaxf(m / 448.0f, 0x1p-126f) : 1.0f;
        inv = 1.0f / scale;
        if (row >= 0 && my.lr == 0) static_cast<float*>(a.scale)[row] = scale;
      }

      const int64_t chunk0 = (int64_t)((uint64_t)(unsigned)row * (unsigned)chunks) + my.lr;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        float* y = v[FMT == kFP8 ? k : 0];
        if constexpr (FMT != kFP8) values(k, y);
        int e = 0;
        if constexpr (FMT == kMXFP8 || FMT == kMXFP4) {
          float m = 0.0f;
#pragma unroll
          for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(y[j]));
          m = quad_max(m);
          // floor(log2(m)) - emax, clamped; frexp's exponent is floor(log2(m)) + 1
          const int x = __builtin_amdgcn_frexp_expf(m) - 1 - (FMT == kMXFP8 ? 8 : 2);
          e = m > 0.0f ? max(-127, min(127, x)) : -127;
        }
        const int64_t chunk = chunk0 + k * P;
        if (row < 0 || my.lr + k * P >= chunks) {
          // nothing to write
        } else if constexpr (FMT == kBF16) {
          store8<kRowsBF16>(a.codes, chunk * 8, y);
        } else if constexpr (FMT == kFP8) {
          const u32x2 w = {e4m3x4_quotient(y, scale, inv), e4m3x4_quotient(y + 4, scale, inv)};
          *reinterpret_cast<u32x2*>(a.codes + chunk * 8) = w;
        } else {
          if ((my.lr & 3) == 0)
            static_cast<uint8_t*>(a.scale)[chunk >> 2] = (uint8_t)(e + 127);
          // the conversions divide by this: the scale's exponent in an fp32
          const float by = __uint_as_float((unsigned)(e + 127) << 23);
          if constexpr (FMT == kMXFP8) {  // what lies over 448 would turn to NaN
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
            *reinterpret_cast<u32x2*>(a.codes + chunk * 8) = w;
          } else {  // saturates by itself
            uint32_t w = 0;
            w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[0], y[1], by, 0);
            w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[2], y[3], by, 1);
            w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[4], y[5], by, 2);
            w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[6], y[7], by, 3);
            *reinterpret_cast<uint32_t*>(a.codes + chunk * 4) = w;
          }
        }
      }
    }
  }
}

// claim[slot] = the last row that names the slot, for the slots named.
__global__ void __launch_bounds__(kRowThreads)
claim_kernel(const int* slots, int n, int L, int* claim, bool clear) {
  for (int64_t i = (int64_t)blockIdx.x * kRowThreads + threadIdx.x; i < n; i += kMostBlocks * kRowThreads) {
    const int s = slots[i];
    if (s < 0 || s >= L) continue;
    if (clear) claim[s] = -1;
    else atomicMax(&claim[s], (int)i);
  }
}

// A write's rows: heads of `pieces` pieces of eight elements, and the rotation's layout.
struct WriteShape {
  int heads, pieces, layout;
  bool vec;
};

template <int IN, int FMT, int K>
hipError_t cache_write_k(const CacheWriteArgs& a, const WriteShape& w, int log_p, hipStream_t s) {
  const int threads = std::max(kRowThreads, 1 << log_p), rb = threads >> log_p;
  // Rounds share the set-up and the entries of a workgroup's rows; as many (up to
  // four) as leave 2,048 workgroups and fit the table (8,192 x 64 x 128 to MXFP4 and back with
  // 1, 2, 4, 16 rounds: 100, 85, 81, 79 us; 131,072 x 128 to MXFP8 and back 32.5, 29.4, 29.2, 29.0).
  int rounds = 1;
  const int fit = a.rot.freq ? kWriteEntries / (rb * (a.rot.dim / 2)) : 4;
  while (rounds < 4 && 2 * rounds <= fit && a.n / ((int64_t)rb * 2 * rounds) >= 2048) rounds *= 2;
  WriteGrid g{};
  g.pieces = (uint32_t)w.pieces - 1;
  g.heads = (uint32_t)w.heads - 1;
  g.log_p = (uint32_t)log_p;
  g.rounds = (uint32_t)rounds;
  g.near = kWave % w.pieces == 0;
  g.halves = w.layout == kRotHalf;
  g.mul = SmallDiv((unsigned)w.pieces).mul;
  const dim3 grid(row_blocks(a.n, rb * rounds)), block((unsigned)threads);
  if (!w.vec)  // the layout is a branch there
    hipLaunchKernelGGL((cache_write_kernel<IN, FMT, K, false, kRotHalf>), grid, block, 0, s, a, g);
  else if (w.layout == kRotHalf)
    hipLaunchKernelGGL((cache_write_kernel<IN, FMT, K, true, kRotHalf>), grid, block, 0, s, a, g);
  else
    hipLaunchKernelGGL((cache_write_kernel<IN, FMT, K, true, kRotInterleaved>), grid, block, 0, s, a, g);
  return hipGetLastError();
}

template <int IN, int FMT>
hipError_t cache_write_fmt(const CacheWriteArgs& a, const WriteShape& w, hipStream_t s) {
  const int chunks = w.heads * w.pieces;
  const bool four = chunks > kRowThreads && kRowThreads % w.pieces == 0;
  int log_p = 2;
  while ((1 << log_p) < chunks && log_p < (FMT == kFP8 && !four ? 10 : 8)) ++log_p;
  return four ? cache_write_k<IN, FMT, 4>(a, w, log_p, s) : cache_write_k<IN, FMT, 1>(a, w, log_p, s);
}

template <int IN>
hipError_t cache_write_in(const CacheWriteArgs& a, const WriteShape& w, int fmt, hipStream_t s) {
  if (fmt == kBF16) return cache_write_fmt<IN, kBF16>(a, w, s);
  if (fmt == kFP8) return cache_write_fmt<IN, kFP8>(a, w, s);
  if (fmt == kMXFP8) return cache_write_fmt<IN, kMXFP8>(a, w, s);
  if (fmt == kMXFP4) return cache_write_fmt<IN, kMXFP4>(a, w, s);
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_cache_write(const CacheWriteArgs& a, int heads, int d, int layout, int in_dtype, int fmt,
                              hipStream_t s) {
  if (a.n <= 0) return hipSuccess;
  if (d % 8 || d <= 0 || heads <= 0 || heads > 256 || d > 8192) return hipErrorInvalidValue;  // WriteGrid's fields
  if (a.slots && a.claim) {
    const dim3 grid(row_blocks(a.n, kRowThreads)), block(kRowThreads);
    for (int clear = 1; clear >= 0; --clear) {
      hipLaunchKernelGGL(claim_kernel, grid, block, 0, s, a.slots, a.n, a.L, a.claim, clear == 1);
      hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  }
  const bool vec = aligned16(a.x, a.ts, a.hs, in_dtype) && (!a.rot.freq || rot_in_eights(a.rot.dim, a.first, layout, d));
  const WriteShape w{heads, d / 8, layout, vec};
  return in_dtype == kRowsBF16 ? cache_write_in<kRowsBF16>(a, w, fmt, s)
                               : cache_write_in<kRowsFP32>(a, w, fmt, s);
}

// --------------------------------------------------------- cache reading

namespace {

// Eight elements of a cache row, as stored.
template <int FMT>
struct Stored8 {
  u32x4 w;    // bf16 uses all four words, E4M3 two, E2M1 one
  float s;    // FP8: the row's scale
  unsigned b;  // MX: the block's scale byte

  __device__ __forceinline__ void load(const CacheReadArgs& a, int64_t row, int e) {
    const int64_t e0 = row * a.row + e;
    if constexpr (FMT == kBF16) {
      w = *reinterpret_cast<const u32x4*>(a.codes + e0 * 2);
    } else if constexpr (FMT == kMXFP4) {
      w[0] = *reinterpret_cast<const uint32_t*>(a.codes + (e0 >> 1));
    } else {
      const u32x2 t = *reinterpret_cast<const u32x2*>(a.codes + e0);
      w[0] = t[0];
      w[1] = t[1];
    }
    if constexpr (FMT == kFP8) s = static_cast<const float*>(a.scale)[row];
    if constexpr (FMT == kMXFP8 || FMT == kMXFP4) b = static_cast<const uint8_t*>(a.scale)[e0 >> 5];
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

// Pieces of eight elements a thread has in flight (eight: 91 us for 1M FP8 rows of 128 against 81).
constexpr int kReadUnits = 4;

// Rows read back, `rows` of them a workgroup: a thread decodes eight elements at a time, so that
// a wave stores one contiguous kilobyte of bf16.
template <int OUT, int FMT, bool PAST>
__global__ void __launch_bounds__(kRowThreads) cache_read_kernel(CacheReadArgs a, int rows, SmallDiv pieces) {
  for (int64_t i0 = (int64_t)blockIdx.x * rows; i0 < a.n; i0 += kMostBlocks * rows) {
    const unsigned end = (unsigned)min((int64_t)rows, a.n - i0) * pieces.by;
    Stored8<FMT> x[kReadUnits];
    int64_t to[kReadUnits];
    bool live[kReadUnits];
#pragma unroll
    for (int k = 0; k < kReadUnits; ++k) {
      const unsigned u = threadIdx.x + k * kRowThreads;
      const unsigned r = pieces(u), e = (u - r * pieces.by) * 8;
      const int64_t i = i0 + r;
      to[k] = u < end ? i * a.row + e : -1;
      live[k] = false;
      if (u < end) {
        const int64_t row = a.slots ? (int64_t)a.slots[i] : (int64_t)a.start + i;
        live[k] = row >= 0 && row < a.L;
        if (live[k]) x[k].load(a, row, (int)e);
      }
    }
#pragma unroll
    for (int k = 0; k < kReadUnits; ++k) {
      if (to[k] < 0) continue;
      float v[8];
      if (live[k]) {
        x[k].decode(v);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.0f;
      }
      store8<OUT, PAST>(a.out, to[k], v);
    }
  }
}

template <int OUT, bool PAST>
hipError_t cache_read_past(const CacheReadArgs& a, int fmt, hipStream_t s) {
  const SmallDiv pieces((unsigned)a.row / 8);           // at most 1,024
  const int rows = kReadUnits * kRowThreads / (int)pieces.by;  // whole rows, at least one
  const dim3 grid(row_blocks(a.n, rows)), block(kRowThreads);
  if (fmt == kBF16) hipLaunchKernelGGL((cache_read_kernel<OUT, kBF16, PAST>), grid, block, 0, s, a, rows, pieces);
  else if (fmt == kFP8) hipLaunchKernelGGL((cache_read_kernel<OUT, kFP8, PAST>), grid, block, 0, s, a, rows, pieces);
  else if (fmt == kMXFP8) hipLaunchKernelGGL((cache_read_kernel<OUT, kMXFP8, PAST>), grid, block, 0, s, a, rows, pieces);
  else if (fmt == kMXFP4) hipLaunchKernelGGL((cache_read_kernel<OUT, kMXFP4, PAST>), grid, block, 0, s, a, rows, pieces);
  else return hipErrorInvalidValue;
  return hipGetLastError();
}

// Results larger than the chip's L2 caches (32 MiB) go past them: 1M FP8 rows of 128 read to
// bf16 (256 MiB) 74 us against 81, 131,072 MXFP8 rows (32 MiB) written and read 29.4 against 30.0;
// smaller ones stay for their reader.
template <int OUT>
hipError_t cache_read_out(const CacheReadArgs& a, int fmt, hipStream_t s) {
  const int64_t bytes = (int64_t)a.n * a.row * rows_bytes(OUT);
  return bytes >= int64_t(32) << 20 ? cache_read_past<OUT, true>(a, fmt, s) : cache_read_past<OUT, false>(a, fmt, s);
}

}  // namespace

hipError_t launch_cache_read(const CacheReadArgs& a, int out_dtype, int fmt, hipStream_t s) {
  if (a.n <= 0) return hipSuccess;
  return out_dtype == kRowsBF16 ? cache_read_out<kRowsBF16>(a, fmt, s)
                                : cache_read_out<kRowsFP32>(a, fmt, s);
}

}  // namespace hk
