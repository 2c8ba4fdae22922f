// Layer norm of rows on their way to the rotation, forward and backward, with
// checkpoints of its input in 8 bits.  Every kernel here moves each row once and is
// bound by memory.
#include <hip/hip_runtime.h>

#include "rows.h"

namespace hk {

namespace {

constexpr int kNormThreads = 256;  // threads of a forward workgroup
constexpr int kBackThreads = 512;  // and of a backward one

// Elements whose type is read from the arguments and which are accessed one by one: rows off
// 16 bytes and widths that are no multiple of eight.
constexpr int kAny = 2;
// A backward's x from a checkpoint (kRowsBF16, kRowsFP32, kAny: rows).
constexpr int kCodesFP8 = 3, kCodesMXFP8 = 4;

// Eight consecutive elements of a row, as loaded; `e` of them counts where only whole pieces exist
// (16-byte access) as eight.
template <int T>
struct Piece {
  Raw8<T> raw;
  __device__ __forceinline__ void zero() { raw.zero(); }
  __device__ __forceinline__ void load(const void* base, int64_t at, int, bool) { raw.template load<true>(base, at); }
  __device__ __forceinline__ void floats(float* v) const { raw.floats(v); }
};
template <>
struct Piece<kAny> {
  float v[8];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (float& x : v) x = 0.0f;
  }
  __device__ __forceinline__ void load(const void* base, int64_t at, int e, bool fp32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = 0.0f;
      if (i < e) v[i] = fp32 ? load1<kRowsFP32>(base, at + i) : load1<kRowsBF16>(base, at + i);
    }
  }
  __device__ __forceinline__ void floats(float* o) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = v[i];
  }
};

template <int T>
__device__ __forceinline__ void put(void* base, int64_t at, int e, bool fp32, const float* v) {
  if constexpr (T == kAny) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i >= e) continue;
      if (fp32) store1<kRowsFP32>(base, at + i, v[i]);
      else store1<kRowsBF16>(base, at + i, v[i]);
    }
  } else {
    store8<T>(base, at, v);
  }
}

// `e` elements of a weight or bias from element `at`, or `other` without one; `whole`: all eight, 16-byte aligned.
__device__ __forceinline__ void parameters(const void* p, bool fp32, bool whole, int at, int e, float other, float* v) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = other;
  if (!p || e == 0) return;
  if (whole) {
    if (fp32) load8<kRowsFP32, true>(p, at, v);
    else load8<kRowsBF16, true>(p, at, v);
    return;
  }
  for (int i = 0; i < e; ++i) {
    const float x = fp32 ? load1<kRowsFP32>(p, at + i) : load1<kRowsBF16>(p, at + i);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j == i ? x : v[j];
  }
}

// The sum over groups of P neighbouring lanes (a power of two up to 64), in each of them.
template <int CTRL>
__device__ __forceinline__ float add_dpp(float x) {
  return x + __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), CTRL, 0xf, 0xf, true));
}
// The sum with the lane 16 or 32 lanes away.
__device__ __forceinline__ float add_16(float x) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}
__device__ __forceinline__ float add_32(float x) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}
__device__ __forceinline__ float lanes_add(float x, int P) {
  if (P > 1) x = add_dpp<0xb1>(x);
  if (P > 2) x = add_dpp<0x4e>(x);
  if (P > 4) x = add_dpp<0x141>(x);
  if (P > 8) x = add_dpp<0x140>(x);
  if (P > 16) x = add_16(x);
  if (P > 32) x = add_32(x);
  return x;
}

// Joins what the waves of a row hold (P > 64 threads a row; `flip` alternates between two
// halves, so that one barrier a step is enough: the other half is read by waves still in the last step).
template <typename Join>
__device__ __forceinline__ float2 join_waves(float2 (*red)[kBackThreads / kWave], int& flip, int P, float2 v, Join join) {
  float2* part = red[flip];
  flip ^= 1;
  if (lane_id() == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  const int waves = P / kWave, w0 = (threadIdx.x >> 6) & ~(waves - 1);
  v = part[w0];
  for (int w = 1; w < waves; ++w) v = join(v, part[w0 + w]);
  return v;
}

// 1 / sqrt(v) within 2^-23; the instruction takes subnormal arguments as 0.
__device__ __forceinline__ float inverse_root(float v) {
  const bool low = v < 0x1p-96f;
  return __builtin_amdgcn_rsqf(low ? v * 0x1p96f : v) * (low ? 0x1p48f : 1.0f);
}

}  // namespace

// How rows lie on threads: P = 1 << log_p threads take a row in K pieces of eight elements each, piece k of
// thread t being the (t + k P)-th.
struct NormGrid {
  uint32_t d : 14;      // at most 8,192
  uint32_t log_p : 4;
  uint32_t rounds : 11;  // times threads / P rows of a workgroup
  uint32_t fp32 : 1;     // weight and bias; whether both can be read 16 bytes at a time
  uint32_t whole : 1;
  uint32_t x32 : 1;      // x, y (rows accessed one element at a time)
  uint32_t y32 : 1;
};
static_assert(sizeof(NormArgs) + sizeof(NormGrid) <= 112, "launches");

namespace {

// y = (x - mean) / sqrt(var + eps) * weight + bias of each row.  A row is read once and stays in registers: a
// first sum gives m0, the mean but for that sum's rounding; the sums of x - m0 and its square then give the rest of
// the mean and the variance about m0, less that rest's square, so neither an offset of the row nor its sum's
// rounding reaches the deviations.  SAVE: the row is also quantised as a cache row of its own.
template <int IN, int OUT, int SAVE, int K>
__global__ void __launch_bounds__(kNormThreads) layer_norm_kernel(NormArgs a, NormGrid g) {
#pragma clang fp contract(off)  // every path (alignment, types, checkpoint) gives the same bits
  __shared__ float2 red[2][kBackThreads / kWave];
  const int d = g.d, P = 1 << g.log_p, RB = kNormThreads >> g.log_p;
  const int lr = threadIdx.x & (P - 1), rl = threadIdx.x >> g.log_p;
  const float inv_d = 1.0f / (float)d;
  auto count = [&](int k) { return min(max(d - 8 * (lr + k * P), 0), 8); };  // elements of the thread's k-th piece
  float w[K][8], b[K][8];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    parameters(a.weight, g.fp32, g.whole, 8 * (lr + k * P), count(k), 1.0f, w[k]);
    parameters(a.bias, g.fp32, g.whole, 8 * (lr + k * P), count(k), 0.0f, b[k]);
  }
  const int64_t row0 = (int64_t)blockIdx.x * RB * g.rounds + rl;
  // The token and head of a row (one head: rows `ts` apart).
  auto place = [&](int64_t row, int64_t ts, int64_t hs) {
    if (a.heads == 1) return row * ts;
    const unsigned t = (unsigned)row / (unsigned)a.heads;
    return (int64_t)t * ts + (int64_t)((unsigned)row - t * (unsigned)a.heads) * hs;
  };
  Piece<IN> raw[K];  // the next row's elements, under way while this one is worked on
  auto fetch = [&](int64_t row) {
    const int64_t at = row < a.rows ? place(row, a.xts, a.xhs) : 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      raw[k].zero();
      if (row < a.rows && count(k) > 0) raw[k].load(a.x, at + 8 * (lr + k * P), count(k), g.x32);
    }
  };
  fetch(row0);
  int flip = 0;
  for (int r = 0; r < (int)g.rounds; ++r) {
    const int64_t row = row0 + (int64_t)r * RB;
    if (row - rl >= a.rows) break;  // the whole workgroup
    float v[K][8];
#pragma unroll
    for (int k = 0; k < K; ++k) raw[k].floats(v[k]);
    if (r + 1 < (int)g.rounds) fetch(row + RB);

    float sum = 0.0f, top = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sum += v[k][i];
        if constexpr (SAVE == kFP8) top = fmaxf(top, fabsf(v[k][i]));
      }
    sum = lanes_add(sum, P);
    if constexpr (SAVE == kFP8) top = lanes_max(top, P);
    if (P > kWave) {
      const float2 s = join_waves(red, flip, P, make_float2(sum, top),
                                  [](float2 x, float2 y) { return make_float2(x.x + y.x, fmaxf(x.y, y.y)); });
      sum = s.x;
      top = s.y;
    }
    const float m0 = sum * inv_d;
    if constexpr (SAVE == kFP8) {
      const float scale = top > 0.0f ? fmaxf(top / 448.0f, 0x1p-126f) : 1.0f, inv = 1.0f / scale;
      if (row < a.rows && lr == 0) static_cast<float*>(a.scale)[row] = scale;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (row >= a.rows || count(k) == 0) continue;
        const u32x2 c = {e4m3x4_quotient(v[k], scale, inv), e4m3x4_quotient(v[k] + 4, scale, inv)};
        *reinterpret_cast<u32x2*>(a.codes + row * d + 8 * (lr + k * P)) = c;
      }
    } else if constexpr (SAVE == kMXFP8) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[k][i]));
        const int e = mx_exponent<kMXFP8>(quad_max(m));  // the four lanes of a block
        if (row >= a.rows || count(k) == 0) continue;
        const int64_t at = row * d + 8 * (lr + k * P);
        if ((lr & 3) == 0) static_cast<uint8_t*>(a.scale)[at >> 5] = (uint8_t)(e + 127);
        *reinterpret_cast<u32x2*>(a.codes + at) = mx_e4m3x8(v[k], e);
      }
    }

    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int n = count(k);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float c = i < (IN == kAny ? n : 8 * min(n, 1)) ? v[k][i] - m0 : 0.0f;
        v[k][i] = c;
        s1 += c;
        s2 = fmaf(c, c, s2);
      }
    }
    s1 = lanes_add(s1, P);
    s2 = lanes_add(s2, P);
    if (P > kWave) {
      const float2 s = join_waves(red, flip, P, make_float2(s1, s2),
                                  [](float2 x, float2 y) { return make_float2(x.x + y.x, x.y + y.y); });
      s1 = s.x;
      s2 = s.y;
    }
    const float rest = s1 * inv_d, var = fmaf(-rest, rest, s2 * inv_d);
    const float rstd = inverse_root(fmaxf(var, 0.0f) + a.eps);
    if (row >= a.rows) continue;
    if (a.stats && lr == 0) a.stats[row] = make_float2(m0 + rest, rstd);
    const int64_t at = place(row, a.yts, a.yhs);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (count(k) == 0) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[k][i] = fmaf((v[k][i] - rest) * rstd, w[k][i], b[k][i]);
      put<OUT>(a.y, at + 8 * (lr + k * P), count(k), g.y32, v[k]);
    }
  }
}

// Threads and pieces a row of d elements: the fewest slots that hold it, on 16 threads or more (rows shorter
// than that: one piece a thread), so that neighbouring threads read neighbouring pieces and the four
// pieces of an MX block lie on neighbouring lanes; of equals the most threads up to 1 << best_log_p, else the fewest.
struct RowShape {
  int log_p, k;
};
RowShape row_shape(int d, int most_log_p, int most_k, int best_log_p) {
  const int pieces = (d + 7) / 8;
  RowShape best{0, 0};
  for (int log_p = 0; log_p <= most_log_p; ++log_p)
    for (int k = 1; k <= most_k; ++k) {
      const int slots = k << log_p, had = best.k << best.log_p;
      if (slots < pieces || (log_p < 4 && k > 1)) continue;
      if (best.k == 0 || slots < had || (slots == had && log_p <= best_log_p)) best = RowShape{log_p, k};
    }
  return best;
}

template <int IN, int OUT, int SAVE>
hipError_t layer_norm_k(const NormArgs& a, NormGrid g, int k, hipStream_t s) {
  const int64_t rb = kNormThreads >> g.log_p;
  int64_t rounds = 1;
  while (rounds < 4 && a.rows / (rb * 2 * rounds) >= 2048) rounds *= 2;
  rounds = std::max(rounds, (a.rows / rb + kMostBlocks) / kMostBlocks);
  g.rounds = (uint32_t)rounds;
  const dim3 grid((unsigned)((a.rows + rb * rounds - 1) / (rb * rounds))), block(kNormThreads);
  switch (k) {
    case 1: hipLaunchKernelGGL((layer_norm_kernel<IN, OUT, SAVE, 1>), grid, block, 0, s, a, g); break;
    case 2: hipLaunchKernelGGL((layer_norm_kernel<IN, OUT, SAVE, 2>), grid, block, 0, s, a, g); break;
    case 3: hipLaunchKernelGGL((layer_norm_kernel<IN, OUT, SAVE, 3>), grid, block, 0, s, a, g); break;
    case 4: hipLaunchKernelGGL((layer_norm_kernel<IN, OUT, SAVE, 4>), grid, block, 0, s, a, g); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

template <int IN, int OUT>
hipError_t layer_norm_save(const NormArgs& a, const NormGrid& g, int k, int save, hipStream_t s) {
  if (save == kBF16) return layer_norm_k<IN, OUT, kBF16>(a, g, k, s);  // none
  if (save == kFP8) return layer_norm_k<IN, OUT, kFP8>(a, g, k, s);
  if (save == kMXFP8) return layer_norm_k<IN, OUT, kMXFP8>(a, g, k, s);
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_layer_norm(const NormArgs& args, int d, bool weight32, int in_dtype, int out_dtype, int save,
                             hipStream_t s) {
  if (args.rows <= 0) return hipSuccess;
  if (d <= 0 || d > kMaxNorm) return hipErrorInvalidValue;
  NormArgs a = args;
  // rows that lie evenly over tokens and heads are one axis
  if (a.heads > 1 && a.xts == a.heads * a.xhs && a.yts == a.heads * a.yhs) {
    a.heads = 1;
    a.xts = a.xhs;
    a.yts = a.yhs;
  }
  const RowShape shape = row_shape(d, 8, 4, 6);  // one wave where it fits: no barrier
  NormGrid g{};
  g.d = (uint32_t)d;
  g.log_p = (uint32_t)shape.log_p;
  g.fp32 = weight32;
  g.whole = d % 8 == 0 && aligned16(a.weight, 0, 0, kRowsBF16) && aligned16(a.bias, 0, 0, kRowsBF16);
  g.x32 = in_dtype == kRowsFP32;
  g.y32 = out_dtype == kRowsFP32;
  const int64_t xhs = a.heads == 1 ? 0 : a.xhs, yhs = a.heads == 1 ? 0 : a.yhs;
  const int64_t xts = a.rows == a.heads ? 0 : a.xts, yts = a.rows == a.heads ? 0 : a.yts;  // one token: no stride
  if (d % 8 || !aligned16(a.x, xts, xhs, in_dtype) || !aligned16(a.y, yts, yhs, out_dtype))
    return layer_norm_save<kAny, kAny>(a, g, shape.k, save, s);
  if (in_dtype == kRowsBF16) {
    return out_dtype == kRowsBF16 ? layer_norm_save<kRowsBF16, kRowsBF16>(a, g, shape.k, save, s)
                                  : layer_norm_save<kRowsBF16, kRowsFP32>(a, g, shape.k, save, s);
  }
  return out_dtype == kRowsBF16 ? layer_norm_save<kRowsFP32, kRowsBF16>(a, g, shape.k, save, s)
                                : layer_norm_save<kRowsFP32, kRowsFP32>(a, g, shape.k, save, s);
}

// --------------------------------------------------------------- backward

struct NormBackGrid {
  uint32_t d : 14;
  uint32_t log_p : 4;
  uint32_t fp32 : 1;  // weight; whether it can be read 16 bytes at a time
  uint32_t whole : 1;
  uint32_t x32 : 1;   // rows accessed one element at a time
  uint32_t dy32 : 1;
  uint32_t dx32 : 1;
  uint32_t blocks;    // workgroups
};
static_assert(sizeof(NormBackArgs) + sizeof(NormBackGrid) <= 112, "launches");

namespace {

template <int X>
struct XPiece {
  Piece<X> raw;
  __device__ __forceinline__ void zero() { raw.zero(); }
  __device__ __forceinline__ void load(const NormBackArgs& a, int64_t, int64_t at, int, int e0, int e, bool fp32) {
    raw.load(a.x, at + e0, e, fp32);
  }
  __device__ __forceinline__ void floats(float* v) const { raw.floats(v); }
};
template <int FMT>
struct CodePiece {
  Stored8<FMT> raw;
  __device__ __forceinline__ void zero() { raw = Stored8<FMT>{}; }
  __device__ __forceinline__ void load(const NormBackArgs& a, int64_t row, int64_t, int d, int e0, int, bool) {
    raw.load(static_cast<const uint8_t*>(a.x), a.scale, row, row * d + e0);
  }
  __device__ __forceinline__ void floats(float* v) const { raw.decode(v); }
};
template <>
struct XPiece<kCodesFP8> : CodePiece<kFP8> {};
template <>
struct XPiece<kCodesMXFP8> : CodePiece<kMXFP8> {};

// dx = rstd (g - mean(g) - h mean(g h)) with g = dy weight and h = (x - mean) rstd of each row, and this
// workgroup's sums over its rows of dy h and dy, [2][d] behind those of the ones before it.  Statistics are the
// forward's, so both of a row's sums are formed at once; each row is read once and stays in registers, and a thread keeps the sums
// of its columns over all its rows.
template <int X, int DY, int DX, int K>
__global__ void __launch_bounds__(kBackThreads) layer_norm_backward_kernel(NormBackArgs a, NormBackGrid g) {
#pragma clang fp contract(off)  // as forward
  __shared__ float2 red[2][kBackThreads / kWave];
  __shared__ float cols[kBackThreads / kWave][kWave * 8];
  const int d = g.d, P = 1 << g.log_p, RB = kBackThreads >> g.log_p;
  const int lr = threadIdx.x & (P - 1), rl = threadIdx.x >> g.log_p;
  const float inv_d = 1.0f / (float)d;
  auto count = [&](int k) { return min(max(d - 8 * (lr + k * P), 0), 8); };
  float w[K][8], dw[K][8], db[K][8];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    parameters(a.weight, g.fp32, g.whole, 8 * (lr + k * P), count(k), 1.0f, w[k]);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[k][i] = db[k][i] = 0.0f;
  }
  auto place = [&](int64_t row, int64_t ts, int64_t hs) {
    if (a.heads == 1) return row * ts;
    const unsigned t = (unsigned)row / (unsigned)a.heads;
    return (int64_t)t * ts + (int64_t)((unsigned)row - t * (unsigned)a.heads) * hs;
  };
  XPiece<X> xr[K];  // the next row's elements and statistics, under way while this one is worked on
  Piece<DY> yr[K];
  float2 stats;
  auto fetch = [&](int64_t row) {
    const bool have = row < a.rows;
    const int64_t ya = have ? place(row, a.dyts, a.dyhs) : 0;
    const int64_t xa = have && X < kCodesFP8 ? place(row, a.xts, a.xhs) : 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      xr[k].zero();
      yr[k].zero();
      const int e0 = 8 * (lr + k * P);
      if (have && count(k) > 0) {
        yr[k].load(a.dy, ya + e0, count(k), g.dy32);
        xr[k].load(a, row, xa, d, e0, count(k), g.x32);
      }
    }
    stats = have ? a.stats[row] : make_float2(0.0f, 0.0f);
  };
  int64_t row = (int64_t)blockIdx.x * RB + rl;
  fetch(row);
  int flip = 0;
  for (; row - rl < a.rows; row += (int64_t)g.blocks * RB) {
    float h[K][8], dy[K][8];
    const float mean = stats.x, rstd = stats.y;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      xr[k].floats(h[k]);
      yr[k].floats(dy[k]);
    }
    fetch(row + (int64_t)g.blocks * RB);
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        h[k][i] = (h[k][i] - mean) * rstd;
        dw[k][i] = fmaf(dy[k][i], h[k][i], dw[k][i]);
        db[k][i] += dy[k][i];
        dy[k][i] *= w[k][i];
        s1 += dy[k][i];
        s2 = fmaf(dy[k][i], h[k][i], s2);
      }
    if (!a.dx) continue;
    s1 = lanes_add(s1, P);
    s2 = lanes_add(s2, P);
    if (P > kWave) {
      const float2 s = join_waves(red, flip, P, make_float2(s1, s2),
                                  [](float2 x, float2 y) { return make_float2(x.x + y.x, x.y + y.y); });
      s1 = s.x;
      s2 = s.y;
    }
    s1 *= inv_d;
    s2 *= inv_d;
    if (row >= a.rows) continue;
    const int64_t at = place(row, a.dxts, a.dxhs);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (count(k) == 0) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) dy[k][i] = rstd * fmaf(-h[k][i], s2, dy[k][i] - s1);
      put<DX>(a.dx, at + 8 * (lr + k * P), count(k), g.dx32, dy[k]);
    }
  }
  if (!a.part) return;
  // The columns' sums over the workgroup's row groups: over the wave's lanes, then over the waves.
  const int dp = norm_columns(d);
  float* to = a.part + (int64_t)blockIdx.x * 2 * dp;
#pragma unroll
  for (int k = 0; k < K; ++k) {
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      float* c = side ? db[k] : dw[k];
      for (int off = P; off < kWave; off <<= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] += __shfl_xor(c[i], off);
      const int e0 = 8 * (lr + k * P);
      auto store = [&] {
#pragma unroll
        for (int i = 0; i < 8; i += 4)
          if (e0 + i < dp) *reinterpret_cast<f32x4*>(to + side * dp + e0 + i) = f32x4{c[i], c[i + 1], c[i + 2], c[i + 3]};
      };
      if (P == kBackThreads) {  // one row at a time: nothing to join
        store();
        continue;
      }
      __syncthreads();  // the last piece's sums are read
#pragma unroll
      for (int i = 0; i < 8; ++i) cols[threadIdx.x >> 6][i * kWave + lane_id()] = c[i];
      __syncthreads();
      if (rl != 0) continue;
      const int step = max(P / kWave, 1);  // waves of a row group
      for (int wv = (threadIdx.x >> 6) + step; wv < kBackThreads / kWave; wv += step)
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] += cols[wv][i * kWave + lane_id()];
      store();
    }
  }
}

// The sums of the workgroups' columns, [blocks][2][dp], in a fixed order: Q threads of a workgroup take four columns each,
// its other threads further rows, so that all loads of a thread are under way together.
constexpr int kColumnThreads = 1024;
template <int Q>
__global__ void __launch_bounds__(kColumnThreads) norm_columns_kernel(const float* part, float* dw, float* db, int d, int blocks) {
  constexpr int kRows = kColumnThreads / Q, kWaves = kColumnThreads / kWave;
  __shared__ f32x4 sums[kWaves][Q];
  const int dp = norm_columns(d);
  const int c = threadIdx.x % Q, r = threadIdx.x / Q, col = (blockIdx.x * Q + c) * 4;
  f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
  if (col < 2 * dp) {
    constexpr int kFlight = 512 / kRows;
    const float* p = part + col;
    for (int b0 = r; b0 < blocks; b0 += kFlight * kRows) {
      f32x4 v[kFlight];
#pragma unroll
      for (int i = 0; i < kFlight; ++i) {
        v[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (b0 + i * kRows < blocks) v[i] = *reinterpret_cast<const f32x4*>(p + (int64_t)(b0 + i * kRows) * 2 * dp);
      }
#pragma unroll
      for (int i = 0; i < kFlight; ++i) s += v[i];
    }
  }
  // over the rows of a wave, then over the waves
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (Q < 8) s[i] += __shfl_xor(s[i], 4);
    if (Q < 16) s[i] += __shfl_xor(s[i], 8);
    s[i] = add_32(add_16(s[i]));
  }
  if (lane_id() < Q) sums[threadIdx.x / kWave][c] = s;
  __syncthreads();
  if (r != 0 || col >= 2 * dp) return;
  s = sums[0][c];
  for (int i = 1; i < kWaves; ++i) s += sums[i][c];
  float* to = col < dp ? dw : db;
  const int e0 = col < dp ? col : col - dp;
  if (!to) return;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (e0 + i < d) to[e0 + i] = s[i];
}

template <int X, int DY, int DX>
hipError_t backward_k(const NormBackArgs& a, const NormBackGrid& g, int k, hipStream_t s) {
  const dim3 grid(g.blocks), block(kBackThreads);
  switch (k) {
    case 1: hipLaunchKernelGGL((layer_norm_backward_kernel<X, DY, DX, 1>), grid, block, 0, s, a, g); break;
    case 2: hipLaunchKernelGGL((layer_norm_backward_kernel<X, DY, DX, 2>), grid, block, 0, s, a, g); break;
    case 3: hipLaunchKernelGGL((layer_norm_backward_kernel<X, DY, DX, 3>), grid, block, 0, s, a, g); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

template <int X>
hipError_t backward_io(const NormBackArgs& a, const NormBackGrid& g, int k, int dy, int dx, hipStream_t s) {
  if (dy == kRowsBF16) {
    return dx == kRowsBF16 ? backward_k<X, kRowsBF16, kRowsBF16>(a, g, k, s)
                           : backward_k<X, kRowsBF16, kRowsFP32>(a, g, k, s);
  }
  return dx == kRowsBF16 ? backward_k<X, kRowsFP32, kRowsBF16>(a, g, k, s)
                         : backward_k<X, kRowsFP32, kRowsFP32>(a, g, k, s);
}

RowShape back_shape(int d) { return row_shape(d, 9, 3, 9); }

}  // namespace

int norm_backward_blocks(int64_t rows, int d) {
  const int64_t rb = kBackThreads >> back_shape(d).log_p;
  return (int)std::min<int64_t>((rows + rb - 1) / rb, back_shape(d).k == 1 ? 512 : 256);
}

hipError_t launch_layer_norm_backward(const NormBackArgs& args, int d, bool weight32, int x_dtype, int codes, int dy_dtype,
                                      int dx_dtype, float* dweight, float* dbias, hipStream_t s) {
  if (d <= 0 || d > kMaxNorm) return hipErrorInvalidValue;
  NormBackArgs a = args;
  const bool rows = codes == kBF16;  // else a checkpoint's
  const int blocks = norm_backward_blocks(a.rows, d);
  if (blocks > 0 && (a.dx || a.part)) {
    // rows that lie evenly over tokens and heads are one axis
    if (a.heads > 1 && a.dyts == a.heads * a.dyhs && (!rows || a.xts == a.heads * a.xhs) &&
        (!a.dx || a.dxts == a.heads * a.dxhs)) {
      a.heads = 1;
      a.dyts = a.dyhs;
      if (rows) a.xts = a.xhs;
      a.dxts = a.dxhs;
    }
    const RowShape shape = back_shape(d);
    NormBackGrid g{};
    g.d = (uint32_t)d;
    g.log_p = (uint32_t)shape.log_p;
    g.fp32 = weight32;
    g.whole = d % 8 == 0 && aligned16(a.weight, 0, 0, kRowsBF16);
    g.x32 = x_dtype == kRowsFP32;
    g.dy32 = dy_dtype == kRowsFP32;
    g.dx32 = dx_dtype == kRowsFP32;
    g.blocks = (uint32_t)blocks;
    auto ok = [&](const void* p, int64_t ts, int64_t hs, int dtype) {
      return aligned16(p, a.rows == a.heads ? 0 : ts, a.heads == 1 ? 0 : hs, dtype);
    };
    const bool vec = d % 8 == 0 && ok(a.dy, a.dyts, a.dyhs, dy_dtype) && (!rows || ok(a.x, a.xts, a.xhs, x_dtype)) &&
                     (!a.dx || ok(a.dx, a.dxts, a.dxhs, dx_dtype));
    hipError_t e;
    if (!vec) {
      e = rows ? backward_k<kAny, kAny, kAny>(a, g, shape.k, s)
               : codes == kFP8 ? backward_k<kCodesFP8, kAny, kAny>(a, g, shape.k, s)
                               : backward_k<kCodesMXFP8, kAny, kAny>(a, g, shape.k, s);
    } else if (codes == kFP8) {
      e = backward_io<kCodesFP8>(a, g, shape.k, dy_dtype, dx_dtype, s);
    } else if (codes == kMXFP8) {
      e = backward_io<kCodesMXFP8>(a, g, shape.k, dy_dtype, dx_dtype, s);
    } else {
      e = x_dtype == kRowsBF16 ? backward_io<kRowsBF16>(a, g, shape.k, dy_dtype, dx_dtype, s)
                               : backward_io<kRowsFP32>(a, g, shape.k, dy_dtype, dx_dtype, s);
    }
    if (e != hipSuccess) return e;
  }
  if (!dweight && !dbias) return hipSuccess;
  // 256 contiguous bytes a row where that leaves 32 workgroups or more, else 64
  const int quads = norm_columns(d) / 2;
  if (quads >= 512)
    hipLaunchKernelGGL((norm_columns_kernel<16>), dim3((quads + 15) / 16), dim3(kColumnThreads), 0, s, a.part, dweight, dbias, d, blocks);
  else
    hipLaunchKernelGGL((norm_columns_kernel<4>), dim3((quads + 3) / 4), dim3(kColumnThreads), 0, s, a.part, dweight, dbias, d, blocks);
  return hipGetLastError();
}

}  // namespace hk
