// Rows on their way into and out of the selection: rotary positions, and the
// four storage formats of q and k written from and read back to bf16 / fp32
// rows.  Every kernel here moves each row once and is bound by memory.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "common.h"
#include "launch.h"

namespace hk {

namespace {

constexpr int kRowThreads = 256;

typedef unsigned u32x2 __attribute__((ext_vector_type(2)));

// Workgroups along the rows: one per `per` rows, at most 2^22 (a launch holds
// fewer than 2^32 threads); the kernels walk the rest.
unsigned row_blocks(int64_t n, int64_t per) {
  return (unsigned)std::min<int64_t>((n + per - 1) / per, int64_t(1) << 22);
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

// Eight consecutive elements; VEC: 16-byte aligned.
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

template <int DT>
__device__ __forceinline__ void store8(void* base, int64_t at, const float* v) {
  if constexpr (DT == kRowsBF16) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(base) + at) = w;
  } else {
    float* p = static_cast<float*>(base) + at;
    *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
    *reinterpret_cast<f32x4*>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
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

// gain * (cos, sign * sin) of pos * f.  The angle in turns is formed and
// reduced to [-1/2, 1/2] in 64 bits: at 2^31 positions its error is below
// 1e-7 turns, at 2^20 below 1e-10, where 32 bits would keep none of it.
__device__ __forceinline__ float2 rot_entry(const RotArgs& r, int i, int64_t pos) {
  double t = (double)pos * (r.freq[i] * 0.15915494309189533577);
  t -= rint(t);
  float s, c;
  sincospif(2.0f * (float)t, &s, &c);
  return make_float2(c * r.gain, s * (r.gain * r.sign));
}

// One half of a rotated pair: v cos -+ w sin.  Written as one product and one fused
// step, so that every path (alignment, layout, on its way into a cache) gives
// the same bits.
__device__ __forceinline__ float rot_lo(float v, float w, float2 f) { return fmaf(v, f.x, -(w * f.y)); }
__device__ __forceinline__ float rot_hi(float v, float w, float2 f) { return fmaf(v, f.x, w * f.y); }

// The entries of tokens t0 .. t0 + nt - 1, once for all their heads: [nt][dim/2].
__device__ __forceinline__ void rot_table(const RotArgs& r, int t0, int nt, float2* cs) {
  const int half = r.dim >> 1;
  for (int e = threadIdx.x; e < nt * half; e += blockDim.x) {
    const int t = e / half, i = e - t * half;
    const int64_t pos = r.pos ? (int64_t)r.pos[t0 + t] : r.pos0 + t0 + t;
    cs[e] = rot_entry(r, i, pos);
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
  int tb, hb;    // tokens and heads of a workgroup
  int units;     // units of a head
  int rows;      // (token, head) rows in flight: threads / units
};

namespace {

template <int IN, int OUT, int LAYOUT, bool VEC>
__global__ void __launch_bounds__(kRowThreads) rotary_kernel(RotaryArgs a, RotaryGrid g) {
  extern __shared__ float2 cs[];
  const RotArgs& r = a.rot;
  const int half = r.dim >> 1;
  const int h0 = blockIdx.y * g.hb, nh = min(g.hb, a.heads - h0);
  const int ts = g.rows / nh, hs = g.rows - ts * nh;
  constexpr int W = VEC ? 8 : 1;                            // elements of a copy unit
  constexpr int PW = VEC ? (LAYOUT == kRotHalf ? 8 : 4) : 1;  // pairs of a rotated unit
  const int nrot = half / PW;
  for (int64_t tile = blockIdx.x; tile * g.tb < a.n; tile += gridDim.x) {
    const int t0 = (int)(tile * g.tb), nt = min(g.tb, a.n - t0);
    if (tile != blockIdx.x) __syncthreads();  // the last tile's entries are read
    rot_table(r, t0, nt, cs);
    __syncthreads();
    // Units wider than the workgroup (heads of many elements without 16-byte
    // access) are walked in steps of the workgroup.
    for (int u = threadIdx.x % g.units; u < nrot + (a.d - r.dim) / W; u += kRowThreads) {
      int row = threadIdx.x / g.units;
      if (row >= g.rows) break;
      const bool rot = u < nrot;
      int e;  // the unit's first element in the head
      if (rot) {
        e = r.first + (LAYOUT == kRotHalf ? u * PW : 2 * u * PW);
      } else {
        e = (u - nrot) * W;
        if (e >= r.first) e += r.dim;
      }
      int t = row / nh, h = row - t * nh;
      while (t < nt) {
        const int64_t xi = (int64_t)(t0 + t) * a.xts + (int64_t)(h0 + h) * a.xhs + e;
        const int64_t yi = (int64_t)(t0 + t) * a.yts + (int64_t)(h0 + h) * a.yhs + e;
        if constexpr (VEC) {
          float v[8];
          load8<IN, true>(a.x, xi, v);
          if (rot) {
            const float2* c = cs + t * half + u * PW;
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
hipError_t rotary_io(const RotaryArgs& a, bool vec, hipStream_t s) {
  const RotArgs& r = a.rot;
  const int pw = vec ? (r.layout == kRotHalf ? 8 : 4) : 1, w = vec ? 8 : 1;
  const int units = r.dim / 2 / pw + (a.d - r.dim) / w;
  RotaryGrid g;
  g.units = std::min(units, kRowThreads);
  g.rows = kRowThreads / g.units;
  // Four rows a thread where that leaves over 1,024 workgroups, else one.
  const int64_t rows_all = (int64_t)a.n * a.heads;
  const int per = rows_all / (4 * g.rows) >= 1024 ? 4 * g.rows : g.rows;
  g.hb = std::min(a.heads, per);
  if ((a.heads + g.hb - 1) / g.hb > 65535) g.hb = (a.heads + 65534) / 65535;
  g.tb = 1;
  if (g.hb == a.heads) {
    const int lds_tokens = std::max(1, 2048 / (r.dim / 2));  // at most 16 KiB of entries
    g.tb = std::max(1, std::min(per / a.heads, lds_tokens));
  }
  const dim3 grid(row_blocks(a.n, g.tb), (unsigned)((a.heads + g.hb - 1) / g.hb));
  const size_t lds = (size_t)g.tb * (r.dim / 2) * sizeof(float2);
  if (r.layout == kRotHalf) {
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
bool rot_in_eights(const RotArgs& r, int d) {
  return d % 8 == 0 && r.first % 8 == 0 && r.dim % (r.layout == kRotHalf ? 16 : 8) == 0;
}

}  // namespace

hipError_t launch_rotary(const RotaryArgs& a, int in_dtype, int out_dtype, hipStream_t s) {
  if (a.n <= 0) return hipSuccess;
  const bool vec = rot_in_eights(a.rot, a.d) && aligned16(a.x, a.xts, a.xhs, in_dtype) &&
                   aligned16(a.y, a.yts, a.yhs, out_dtype);
  if (in_dtype == kRowsBF16) {
    return out_dtype == kRowsBF16 ? rotary_io<kRowsBF16, kRowsBF16>(a, vec, s)
                                  : rotary_io<kRowsBF16, kRowsFP32>(a, vec, s);
  }
  return out_dtype == kRowsBF16 ? rotary_io<kRowsFP32, kRowsBF16>(a, vec, s)
                                : rotary_io<kRowsFP32, kRowsFP32>(a, vec, s);
}

// --------------------------------------------------------- cache writing

namespace {

// Four values, clamped to +-448, as E4M3 bytes (to nearest, ties to even).
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  a = fminf(fmaxf(a, -448.0f), 448.0f);
  b = fminf(fmaxf(b, -448.0f), 448.0f);
  c = fminf(fmaxf(c, -448.0f), 448.0f);
  d = fminf(fmaxf(d, -448.0f), 448.0f);
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
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

// E2M1 code of v: magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6 (codes 0..7), to
// nearest, ties to the even code, saturating at 6; bit 3 is the sign.
__device__ __forceinline__ uint32_t e2m1(float v) {
  const float a = fminf(fabsf(v), 6.0f);
  const float c = a < 2.0f ? rintf(2.0f * a) : (a < 4.0f ? rintf(a) + 2.0f : rintf(0.5f * a) + 4.0f);
  return (uint32_t)c | ((__float_as_uint(v) >> 31) << 3);
}

// Rotated values of elements e0 .. e0 + 7 of a head (v holds them unrotated;
// `at` is the head's offset in x, cs the token's entries).
template <int IN, bool VEC>
__device__ __forceinline__ void rotate8(const RotArgs& r, const void* x, int64_t at, int e0,
                                        const float2* cs, float* v) {
  const int half = r.dim >> 1;
  const int e = e0 - r.first;
  if constexpr (VEC) {  // all eight lie on one side of every border
    if (e < 0 || e >= r.dim) return;
    if (r.layout == kRotHalf) {
      const bool lo = e < half;
      const float2* c = cs + (lo ? e : e - half);
      float w[8];
      load8<IN, true>(x, at + e0 + (lo ? half : -half), w);  // the partners, in cache by now
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 f = c[i];
        v[i] = lo ? rot_lo(v[i], w[i], f) : rot_hi(v[i], w[i], f);
      }
    } else {
      const float2* c = cs + (e >> 1);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = c[i];
        const float p = v[2 * i], q = v[2 * i + 1];
        v[2 * i] = rot_lo(p, q, f);
        v[2 * i + 1] = rot_hi(q, p, f);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int ei = e + i;
      if (ei < 0 || ei >= r.dim) continue;
      const bool lo = r.layout == kRotHalf ? ei < half : (ei & 1) == 0;
      const int off = r.layout == kRotHalf ? half : 1;
      const float2 f = cs[r.layout == kRotHalf ? (lo ? ei : ei - half) : ei >> 1];
      const float w = load1<IN>(x, at + e0 + i + (lo ? off : -off));
      v[i] = lo ? rot_lo(v[i], w, f) : rot_hi(v[i], w, f);
    }
  }
}

// Rows written into a cache.  P threads (a power of two, 4..256) take a row in
// chunks of eight elements, K chunks each, so a row is read once and its
// scale comes from registers: a lane reduction over the row (FP8), or over the four
// lanes of a 32-element block (MX).
template <int IN, int FMT, int K, bool VEC>
__global__ void __launch_bounds__(kRowThreads)
cache_write_kernel(CacheWriteArgs a, int log_p) {
  __shared__ float2 cs[1024];
  __shared__ float red[kRowThreads / kWave];
  __shared__ int later[kRowThreads / 4];
  const int P = 1 << log_p, RB = kRowThreads >> log_p;
  const int rl = threadIdx.x >> log_p, lr = threadIdx.x & (P - 1);
  const int chunks = a.heads * a.d / 8;
  for (int64_t tile = blockIdx.x; tile * RB < a.n; tile += gridDim.x) {
    const int i0 = (int)(tile * RB);
    const int i = rl < a.n - i0 ? i0 + rl : a.n;
    const bool have = i < a.n;
    if (tile != blockIdx.x) __syncthreads();  // LDS of the last rows is read

    float v[K][8];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = lr + k * P;
      if (have && c < chunks) {
        const int h = a.heads == 1 ? 0 : c * 8 / a.d, e0 = c * 8 - h * a.d;
        load8<IN, VEC>(a.x, (int64_t)i * a.ts + (int64_t)h * a.hs + e0, v[k]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[k][j] = 0.0f;
      }
    }

    // The row's place; -1 where nothing is written.
    int64_t row = -1;
    if (have) {
      row = a.slots ? (int64_t)a.slots[i] : a.start + i;
      if (row >= a.L || row < 0) row = -1;
      if (row >= 0 && a.claim && a.claim[row] != i) row = -1;
    }
    if (a.slots && !a.claim) {  // few rows: look for a later row of the same slot
      for (int t = threadIdx.x; t < RB; t += kRowThreads) later[t] = 0;
      __syncthreads();
      if (row >= 0) {
        bool dup = false;
        for (int j = i + 1 + lr; j < a.n; j += P) dup |= (int64_t)a.slots[j] == row;
        if (dup) later[rl] = 1;
      }
      __syncthreads();
      if (later[rl]) row = -1;
    }

    if (a.rot.freq) {
      rot_table(a.rot, i0, min(RB, a.n - i0), cs);
      __syncthreads();
      const float2* my = cs + rl * (a.rot.dim >> 1);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int c = lr + k * P;
        if (have && c < chunks) {
          const int h = a.heads == 1 ? 0 : c * 8 / a.d, e0 = c * 8 - h * a.d;
          rotate8<IN, VEC>(a.rot, a.x, (int64_t)i * a.ts + (int64_t)h * a.hs, e0, my, v[k]);
        }
      }
    }

    float scale = 1.0f, inv = 1.0f;
    if constexpr (FMT == kFP8) {
      float m = 0.0f;
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[k][j]));
      for (int off = min(P, kWave) >> 1; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
      if (P > kWave) {  // uniform over the launch
        if (lane_id() == 0) red[threadIdx.x >> 6] = m;
        __syncthreads();
        const int w0 = rl * (P / kWave);
        for (int w = 0; w < P / kWave; ++w) m = fmaxf(m, red[w0 + w]);
      }
      scale = m > 0.0f ? fmaxf(m / 448.0f, 0x1p-126f) : 1.0f;
      inv = 1.0f / scale;
      if (row >= 0 && lr == 0) static_cast<float*>(a.scale)[row] = scale;
    }

#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = lr + k * P;
      int e = 0;
      if constexpr (FMT == kMXFP8 || FMT == kMXFP4) {
        float m = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[k][j]));
        m = fmaxf(m, __shfl_xor(m, 1));
        m = fmaxf(m, __shfl_xor(m, 2));
        int x;
        (void)frexpf(m, &x);  // floor(log2(m)) + 1
        e = m > 0.0f ? max(-127, min(127, x - 1 - (FMT == kMXFP8 ? 8 : 2))) : -127;
      }
      if (row < 0 || c >= chunks) {
        // nothing to write
      } else if constexpr (FMT == kBF16) {
        store8<kRowsBF16>(a.codes, (row * chunks + c) * 8, v[k]);
      } else if constexpr (FMT == kFP8) {
        const u32x2 w = {e4m3x4_quotient(v[k], scale, inv), e4m3x4_quotient(v[k] + 4, scale, inv)};
        *reinterpret_cast<u32x2*>(a.codes + (row * chunks + c) * 8) = w;
      } else {
        if ((lr & 3) == 0)
          static_cast<uint8_t*>(a.scale)[(row * chunks + c) >> 2] = (uint8_t)(e + 127);
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = ldexpf(v[k][j], -e);
        if constexpr (FMT == kMXFP8) {
          const u32x2 w = {e4m3x4(y[0], y[1], y[2], y[3]), e4m3x4(y[4], y[5], y[6], y[7])};
          *reinterpret_cast<u32x2*>(a.codes + (row * chunks + c) * 8) = w;
        } else {
          uint32_t w = 0;
#pragma unroll
          for (int j = 0; j < 8; ++j) w |= e2m1(y[j]) << (4 * j);
          *reinterpret_cast<uint32_t*>(a.codes + (row * chunks + c) * 4) = w;
        }
      }
    }
  }
}

// claim[slot] = the last row that names the slot, for the slots named.
__global__ void __launch_bounds__(kRowThreads)
claim_kernel(const int* slots, int n, int L, int* claim, bool clear) {
  for (int64_t i = (int64_t)blockIdx.x * kRowThreads + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * kRowThreads) {
    const int s = slots[i];
    if (s < 0 || s >= L) continue;
    if (clear) claim[s] = -1;
    else atomicMax(&claim[s], (int)i);
  }
}

template <int IN, int FMT>
hipError_t cache_write_fmt(const CacheWriteArgs& a, bool vec, hipStream_t s) {
  const int chunks = a.heads * a.d / 8;
  int log_p = 2;
  while ((1 << log_p) < chunks && log_p < 8) ++log_p;
  const int per = (chunks + (1 << log_p) - 1) >> log_p;
  const int rb = kRowThreads >> log_p;
  const dim3 grid(row_blocks(a.n, rb)), block(kRowThreads);
  if (vec) {
    if (per == 1) hipLaunchKernelGGL((cache_write_kernel<IN, FMT, 1, true>), grid, block, 0, s, a, log_p);
    else if (per == 2) hipLaunchKernelGGL((cache_write_kernel<IN, FMT, 2, true>), grid, block, 0, s, a, log_p);
    else hipLaunchKernelGGL((cache_write_kernel<IN, FMT, 4, true>), grid, block, 0, s, a, log_p);
  } else {
    if (per == 1) hipLaunchKernelGGL((cache_write_kernel<IN, FMT, 1, false>), grid, block, 0, s, a, log_p);
    else hipLaunchKernelGGL((cache_write_kernel<IN, FMT, 4, false>), grid, block, 0, s, a, log_p);
  }
  return hipGetLastError();
}

template <int IN>
hipError_t cache_write_in(const CacheWriteArgs& a, int fmt, bool vec, hipStream_t s) {
  if (fmt == kBF16) return cache_write_fmt<IN, kBF16>(a, vec, s);
  if (fmt == kFP8) return cache_write_fmt<IN, kFP8>(a, vec, s);
  if (fmt == kMXFP8) return cache_write_fmt<IN, kMXFP8>(a, vec, s);
  if (fmt == kMXFP4) return cache_write_fmt<IN, kMXFP4>(a, vec, s);
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_cache_write(const CacheWriteArgs& a, int in_dtype, int fmt, hipStream_t s) {
  if (a.n <= 0) return hipSuccess;
  if (a.slots && a.claim) {
    const dim3 grid(row_blocks(a.n, kRowThreads)), block(kRowThreads);
    for (int clear = 1; clear >= 0; --clear) {
      hipLaunchKernelGGL(claim_kernel, grid, block, 0, s, a.slots, a.n, a.L, a.claim, clear == 1);
      hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  }
  const bool vec = aligned16(a.x, a.ts, a.hs, in_dtype) && (!a.rot.freq || rot_in_eights(a.rot, a.d));
  return in_dtype == kRowsBF16 ? cache_write_in<kRowsBF16>(a, fmt, vec, s)
                               : cache_write_in<kRowsFP32>(a, fmt, vec, s);
}

// --------------------------------------------------------- cache reading

namespace {

// Sixteen elements of a cache row.
template <int FMT>
__device__ __forceinline__ void decode16(const CacheReadArgs& a, int64_t row, int c, float* o) {
  const int64_t e0 = row * a.row + c * 16;
  if constexpr (FMT == kBF16) {
    const u32x4* p = reinterpret_cast<const u32x4*>(a.codes + e0 * 2);
    unpack_bf16(p[0], o);
    unpack_bf16(p[1], o + 8);
    return;
  }
  if constexpr (FMT == kFP8 || FMT == kMXFP8) {
    const u32x4 w = *reinterpret_cast<const u32x4*>(a.codes + e0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false);
      const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
      o[4 * i] = lo[0];
      o[4 * i + 1] = lo[1];
      o[4 * i + 2] = hi[0];
      o[4 * i + 3] = hi[1];
    }
  }
  if constexpr (FMT == kMXFP4) {
    const u32x2 w = *reinterpret_cast<const u32x2*>(a.codes + (e0 >> 1));
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t n = (w[i >> 3] >> (4 * (i & 7))) & 15u, m = n & 7u;
      // exponent and mantissa bits of the E2M1 code in an fp32 (code 1 is 0.5, the one subnormal)
      const float f = m < 2u ? 0.5f * (float)m : __uint_as_float(((m >> 1) + 126u) << 23 | (m & 1u) << 22);
      o[i] = (n & 8u) ? -f : f;
    }
  }
  if constexpr (FMT == kFP8) {
    const float s = static_cast<const float*>(a.scale)[row];
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] *= s;
  } else {
    const int b = static_cast<const uint8_t*>(a.scale)[e0 >> 5];
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = b == 255 ? __builtin_nanf("") : ldexpf(o[i], b - 127);
  }
}

// Rows read back: a thread decodes sixteen elements.
template <int OUT, int FMT>
__global__ void __launch_bounds__(kRowThreads) cache_read_kernel(CacheReadArgs a, int rows) {
  const int chunks = a.row / 16;
  for (int64_t i0 = (int64_t)blockIdx.x * rows; i0 < a.n; i0 += (int64_t)gridDim.x * rows) {
    const int nr = (int)min((int64_t)rows, a.n - i0);
    for (int u = threadIdx.x; u < nr * chunks; u += kRowThreads) {
      const int r = u / chunks, c = u - r * chunks;
      const int64_t i = i0 + r;
      const int64_t row = a.slots ? (int64_t)a.slots[i] : a.start + i;
      float v[16];
      if (row >= 0 && row < a.L) {
        decode16<FMT>(a, row, c, v);
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = 0.0f;
      }
      store8<OUT>(a.out, i * a.row + c * 16, v);
      store8<OUT>(a.out, i * a.row + c * 16 + 8, v + 8);
    }
  }
}

template <int OUT>
hipError_t cache_read_out(const CacheReadArgs& a, int fmt, hipStream_t s) {
  const int chunks = a.row / 16;
  const int rows = std::max(1, 4 * kRowThreads / chunks);
  const dim3 grid(row_blocks(a.n, rows)), block(kRowThreads);
  if (fmt == kBF16) hipLaunchKernelGGL((cache_read_kernel<OUT, kBF16>), grid, block, 0, s, a, rows);
  else if (fmt == kFP8) hipLaunchKernelGGL((cache_read_kernel<OUT, kFP8>), grid, block, 0, s, a, rows);
  else if (fmt == kMXFP8) hipLaunchKernelGGL((cache_read_kernel<OUT, kMXFP8>), grid, block, 0, s, a, rows);
  else if (fmt == kMXFP4) hipLaunchKernelGGL((cache_read_kernel<OUT, kMXFP4>), grid, block, 0, s, a, rows);
  else return hipErrorInvalidValue;
  return hipGetLastError();
}

}  // namespace

hipError_t launch_cache_read(const CacheReadArgs& a, int out_dtype, int fmt, hipStream_t s) {
  if (a.n <= 0) return hipSuccess;
  return out_dtype == kRowsBF16 ? cache_read_out<kRowsBF16>(a, fmt, s)
                                : cache_read_out<kRowsFP32>(a, fmt, s);
}

}  // namespace hk
