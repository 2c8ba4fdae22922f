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

// `e` elements `step` apart, as stored; the others stay.
__device__ __forceinline__ void load_each(const void* base, int64_t at, int step, int e, bool fp32, uint32_t* v) {
  if (fp32) {
    const uint32_t* p = static_cast<const uint32_t*>(base) + at;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < e) v[i] = p[i * step];
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(base) + at;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < e) v[i] = p[i * step];
  }
}

// Eight elements of a row, as loaded, `step` apart, of which `e` exist (with 16-byte access: neighbours, and all).
template <int T>
struct Piece {
  Raw8<T> raw;
  __device__ __forceinline__ void zero() { raw.zero(); }
  __device__ __forceinline__ void load(const void* base, int64_t at, int, int, bool) { raw.template load<true>(base, at); }
  __device__ __forceinline__ void floats(float* v) const { raw.floats(v); }
};
template <>
struct Piece<kAny> {
  uint32_t v[8];  // as stored: a conversion beside the loads would wait for each
  bool wide;
  __device__ __forceinline__ void zero() {
    wide = true;
#pragma unroll
    for (uint32_t& x : v) x = 0u;
  }
  __device__ __forceinline__ void load(const void* base, int64_t at, int step, int e, bool fp32) {
    wide = fp32;
    load_each(base, at, step, e, fp32, v);
  }
  __device__ __forceinline__ void floats(float* o) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = __uint_as_float(wide ? v[i] : v[i] << 16);
  }
};

// PAST: not kept in the caches.
template <int T, bool PAST>
__device__ __forceinline__ void put(void* base, int64_t at, int step, int e, bool fp32, const float* v) {
  if constexpr (T == kAny) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i >= e) continue;
      if (fp32) store1<kRowsFP32>(base, at + i * step, v[i]);
      else store1<kRowsBF16>(base, at + i * step, v[i]);
    }
  } else {
    store8<T, PAST>(base, at, v);
  }
}

template <bool PAST>
__device__ __forceinline__ void put_codes(uint8_t* to, const u32x2& c) {
  if constexpr (PAST) __builtin_nontemporal_store(c, reinterpret_cast<u32x2*>(to));
  else *reinterpret_cast<u32x2*>(to) = c;
}

// Eight elements of a weight or bias from element `at`, `step` apart, of which `e` exist, or `other` without one.  WHOLE: neighbours,
// 16-byte aligned; loaded first and read later, so that loads of several are under way together.
template <bool WHOLE>
struct Parameters {
  u32x4 w[2];
  __device__ __forceinline__ void load(const void* p, bool fp32, int at, int step, int e) {
    w[0] = w[1] = u32x4{0u, 0u, 0u, 0u};
    if (!p || e == 0) return;
    if constexpr (WHOLE) {
      const char* c = static_cast<const char*>(p) + (int64_t)at * (fp32 ? 4 : 2);
      w[0] = *reinterpret_cast<const u32x4*>(c);
      if (fp32) w[1] = *reinterpret_cast<const u32x4*>(c + 16);
    } else {
      uint32_t v[8] = {};
      load_each(p, at, step, e, fp32, v);
      w[0] = u32x4{v[0], v[1], v[2], v[3]};
      w[1] = u32x4{v[4], v[5], v[6], v[7]};
    }
  }
  __device__ __forceinline__ void floats(const void* p, bool fp32, float other, float* v) const {
    if (!p) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = other;
    } else if (WHOLE && !fp32) {
      unpack_bf16(w[0], v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(fp32 ? w[i >> 2][i & 3] : w[i >> 2][i & 3] << 16);
    }
  }
};

// The sum over groups of 1 << log_p neighbouring lanes (at most 64), in each of them: halves, then rows of 16, halves of
// rows (mirrored) and quads by lane permutations inside the vector instruction.
template <int CTRL>
__device__ __forceinline__ float add_dpp(float x) {
  return x + __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), CTRL, 0xf, 0xf, true));
}
// With the lane 16 or 32 lanes away.
__device__ __forceinline__ float add_16(float x) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}
__device__ __forceinline__ float add_32(float x) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}
template <int N>
__device__ __forceinline__ void lanes_add(float (&x)[N], int log_p) {
  auto each = [&](auto step) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = step(x[i]);
  };
  switch (log_p) {
    default: each(add_32); [[fallthrough]];
    case 5: each(add_16); [[fallthrough]];
    case 4: each(add_dpp<0x140>); [[fallthrough]];
    case 3: each(add_dpp<0x141>); [[fallthrough]];
    case 2: each(add_dpp<0x4e>); [[fallthrough]];
    case 1: each(add_dpp<0xb1>); [[fallthrough]];
    case 0: break;
  }
}

// The sum over the lanes of a wave whose numbers agree modulo 1 << log_p, in each of them (rows of 16 are rotated).
__device__ __forceinline__ void rows_add(float (&x)[8], int log_p) {
  auto each = [&](auto step) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = step(x[i]);
  };
  switch (log_p) {
    case 0: each(add_dpp<0xb1>); [[fallthrough]];
    case 1: each(add_dpp<0x4e>); [[fallthrough]];
    case 2: each(add_dpp<0x124>); [[fallthrough]];
    case 3: each(add_dpp<0x128>); [[fallthrough]];
    case 4: each(add_16); [[fallthrough]];
    case 5: each(add_32); [[fallthrough]];
    default: break;
  }
}

__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6); }

// Joins what the waves of a row hold (P > 64 threads a row).  One barrier: steps take two arrays by turns, as waves still in
// the last step read the other.  The forward takes its wave's number as a scalar, whose addresses take no registers of the loop.
template <typename V, typename Join>
__device__ __forceinline__ V join_waves(V* part, int wave, int P, V v, Join join) {
  const int waves = P / kWave, w0 = wave & ~(waves - 1);
  if (lane_id() == 0) part[wave] = v;
  __syncthreads();
  v = part[w0];
  for (int w = 1; w < waves; ++w) v = join(v, part[w0 + w]);
  return v;
}

// Waits for the loads under way.  Stores count like loads, and the compiler would wait for a row's at the end of its
// round, where the next row's elements change registers; called before them, it waits only for the last round's.
__device__ __forceinline__ void loads_done() { __builtin_amdgcn_s_waitcnt(0x0f70); }  // vmcnt(0)

// 1 / sqrt(v) within 2^-23; the instruction takes subnormal arguments as 0.
__device__ __forceinline__ float inverse_root(float v) {
  const bool low = v < 0x1p-96f;
  return __builtin_amdgcn_rsqf(low ? v * 0x1p96f : v) * (low ? 0x1p48f : 1.0f);
}

// A thread's elements of a piece of P threads: eight neighbours or, where rows are accessed one element at a time and their width is no
// multiple of eight, every P-th, so that neighbouring threads access neighbours (sums then add up in another order).
struct Spread {
  int first, step, log_step;
  __device__ __forceinline__ Spread(bool any, int d, int lane, int log_p) {
    const bool apart = any && d % 8 != 0;
    log_step = apart ? log_p : 0;
    step = 1 << log_step;
    first = apart ? lane : 8 * lane;
  }
  // How many exist of a row that is `left` elements long from the piece's first on.
  __device__ __forceinline__ int count(int left) const { return min(max((left - first + step - 1) >> log_step, 0), 8); }
};

// A thread's place in rows `ts` and `hs` apart: of the row's elements from `e` on, `step` further each round where
// rows are one axis (one head).
struct Walk {
  int64_t at, step;
  __device__ __forceinline__ Walk(unsigned row, int heads, int64_t ts, int64_t hs, int rows, int e) : step(rows * ts) {
    at = place(row, heads, ts, hs) + e;
  }
  __device__ __forceinline__ void next(unsigned row, int heads, int64_t ts, int64_t hs, int e) {
    at = heads == 1 ? at + step : place(row, heads, ts, hs) + e;
  }
  static __device__ __forceinline__ int64_t place(unsigned row, int heads, int64_t ts, int64_t hs) {
    if (heads == 1) return row * ts;
    const unsigned t = row / (unsigned)heads;
    return t * ts + (row - t * (unsigned)heads) * hs;
  }
};

}  // namespace

// How rows lie on threads: P = 1 << log_p threads take a row in K pieces of eight elements each, piece k of
// thread t being the (t + k P)-th.
struct NormGrid {
  uint32_t d : 14;      // at most 8,192
  uint32_t log_p : 4;
  uint32_t rounds : 11;  // times threads / P rows of a workgroup
  uint32_t fp32 : 1;     // weight and bias
  uint32_t x32 : 1;      // x, y (rows accessed one element at a time)
  uint32_t y32 : 1;
};
static_assert(sizeof(NormArgs) + sizeof(NormGrid) <= 112, "launches");

namespace {

// y = (x - mean) / sqrt(var + eps) * weight + bias of each row.  A row is read once and stays in registers: a
// first sum gives m0, the mean but for that sum's rounding; the sums of x - m0 and its square then give the rest of
// the mean and the variance about m0, less that rest's square, so neither an offset of the row nor its sum's
// rounding reaches the deviations.  Where the row's first element is as near the mean as roundings leave m0, it is m0: the deviations
// of a constant row are 0 then, whatever its size (of a row of 1e9 m0 is off by 64, whose square's rounding is far above eps; past
// 1e25 the square itself passes fp32).  SAVE: the row is also quantised as a cache row of its own, from the same read.
// Bound by memory: bf16 131,072 x 128 11.5 us (5.8 TB/s), 8,192 x 4,096 23.3 (5.8), 5,003 x 7,168 27.8 (5.2); with an FP8
// checkpoint 18.1, 32.1 and 39.3 us (narrow rows by the instructions of the quotients, 4.6 TB/s), with MXFP8 14.2, 29.2 and 32.7.  The
// next row's elements are under way while one is worked on; places along the rows are kept, not formed again
// (131,072 x 128 14.6 us with 64-bit products a row, against 12.2 of the kernel as it was then).
template <int IN, int OUT, int SAVE, int K, bool PAST>
__global__ void __launch_bounds__(kNormThreads) layer_norm_kernel(NormArgs a, NormGrid g) {
#pragma clang fp contract(off)  // every path (alignment, types, checkpoint) gives the same bits
  __shared__ float2 red[2][kNormThreads / kWave];
  __shared__ float4 red4[kNormThreads / kWave];
  const int d = g.d, P = 1 << g.log_p, RB = kNormThreads >> g.log_p;
  const int lr = threadIdx.x & (P - 1), rl = threadIdx.x >> g.log_p;
  const float inv_d = 1.0f / (float)d;
  const Spread spread(IN == kAny, d, lr, g.log_p);
  const int e0 = spread.first, es = spread.step, last = spread.count(d - (K - 1) * P * 8);
  auto count = [&](int k) { return k < K - 1 ? 8 : last; };  // all but the last pieces are whole
  const unsigned rows = a.rows;
  unsigned row = blockIdx.x * (RB * g.rounds) + rl;
  Walk from(row, a.heads, a.xts, a.xhs, RB, e0), to(row, a.heads, a.yts, a.yhs, RB, e0);
  Piece<IN> raw[K];  // the next row's elements, under way while this one is worked on
  auto fetch = [&](unsigned at_row) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      raw[k].zero();
      if (at_row < rows && count(k) > 0) raw[k].load(a.x, from.at + 8 * k * P, es, count(k), g.x32);
    }
  };
  fetch(row);
  float w[K][8], b[K][8];
  {
    Parameters<IN != kAny> pw[K], pb[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      pw[k].load(a.weight, g.fp32, e0 + 8 * k * P, es, count(k));
      pb[k].load(a.bias, g.fp32, e0 + 8 * k * P, es, count(k));
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      pw[k].floats(a.weight, g.fp32, 1.0f, w[k]);
      pb[k].floats(a.bias, g.fp32, 0.0f, b[k]);
    }
  }
  // `left` rows of this round's first row on, the same in the whole workgroup
  int left = (int)(rows - (row - rl));
  for (int r = 0; r < (int)g.rounds && left > 0; ++r, left -= RB) {
    float v[K][8];
#pragma unroll
    for (int k = 0; k < K; ++k) raw[k].floats(v[k]);
    const unsigned now = row;
    row += RB;
    if (r + 1 < (int)g.rounds) {
      from.next(row, a.heads, a.xts, a.xhs, e0);
      fetch(row);
    }

    float sum[1] = {0.0f}, top = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      sum[0] += ((v[k][0] + v[k][1]) + (v[k][2] + v[k][3])) + ((v[k][4] + v[k][5]) + (v[k][6] + v[k][7]));
      if constexpr (SAVE == kFP8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(v[k][i]));
      }
    }
    lanes_add(sum, g.log_p);
    if constexpr (SAVE == kFP8) top = lanes_max(top, P);
    float first;
    if (P > kWave) {
      if constexpr (SAVE == kFP8) {
        const float4 s = join_waves(red4, wave_id(), P, make_float4(sum[0], v[0][0], top, 0.0f),
                                    [](float4 x, float4 y) { return make_float4(x.x + y.x, x.y, fmaxf(x.z, y.z), 0.0f); });
        sum[0] = s.x;
        first = s.y;
        top = s.z;
      } else {
        const float2 s = join_waves(red[0], wave_id(), P, make_float2(sum[0], v[0][0]),
                                    [](float2 x, float2 y) { return make_float2(x.x + y.x, x.y); });
        sum[0] = s.x;
        first = s.y;
      }
    } else {
      first = __shfl(v[0][0], lane_id() & -P);
    }
    float m0 = sum[0] * inv_d;
    // 17 roundings at most lie between a constant row's m0 and its value
    if (fabsf(first - m0) < fabsf(m0) * 0x1p-19f) m0 = first;
    const int64_t code0 = (int64_t)now * d + 8 * lr;
    if constexpr (SAVE == kFP8) {
      const Reciprocal by(e4m3_scale(top));
      if (now < rows && lr == 0) static_cast<float*>(a.scale)[now] = by.scale;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (now >= rows || count(k) == 0) continue;
        const u32x2 c = {e4m3x4_quotient(v[k], by), e4m3x4_quotient(v[k] + 4, by)};
        put_codes<PAST>(a.codes + code0 + 8 * k * P, c);
      }
    } else if constexpr (SAVE == kMXFP8) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[k][i]));
        const int e = mx_exponent<kMXFP8>(quad_max(m));  // the four lanes of a block
        if (now >= rows || count(k) == 0) continue;
        const int64_t at = code0 + 8 * k * P;
        if ((lr & 3) == 0) static_cast<uint8_t*>(a.scale)[at >> 5] = (uint8_t)(e + 127);
        put_codes<PAST>(a.codes + at, mx_e4m3x8(v[k], e));
      }
    }

    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      // elements that do not exist were read as 0 and keep it
      const float m = count(k) > 0 ? m0 : 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[k][i] -= IN == kAny && i >= count(k) ? 0.0f : m;
        s[0] += v[k][i];
        s[1] = fmaf(v[k][i], v[k][i], s[1]);
      }
    }
    lanes_add(s, g.log_p);
    if (P > kWave) {
      const float2 j = join_waves(red[1], wave_id(), P, make_float2(s[0], s[1]),
                                  [](float2 x, float2 y) { return make_float2(x.x + y.x, x.y + y.y); });
      s[0] = j.x;
      s[1] = j.y;
    }
    const float rest = s[0] * inv_d, var = fmaf(-rest, rest, s[1] * inv_d);
    const float rstd = inverse_root(fmaxf(var, 0.0f) + a.eps), off = -rest * rstd;
    loads_done();
    if (now < rows) {
      if (a.stats && lr == 0) a.stats[now] = make_float2(m0 + rest, rstd);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (count(k) == 0) continue;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[k][i] = fmaf(fmaf(v[k][i], rstd, off), w[k][i], b[k][i]);
        put<OUT, PAST>(a.y, to.at + 8 * k * P, es, count(k), g.y32, v[k]);
      }
    }
    if (r + 1 < (int)g.rounds) to.next(row, a.heads, a.yts, a.yhs, e0);
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

// Results larger than the chip's L2 caches (32 MiB) go past them: the forward of 8,192 x 4,096 23.8 us against 28.8, the
// backward of 131,072 x 128 21.3 against 25.2.  Rows off 16 bytes do not.
bool past_caches(int64_t rows, int d, int dtype) { return rows * d * rows_bytes(dtype) >= int64_t(32) << 20; }

template <int IN, int OUT, int SAVE, bool PAST>
hipError_t layer_norm_past(const NormArgs& a, NormGrid g, int k, hipStream_t s) {
  const int64_t rb = kNormThreads >> g.log_p, sets = (a.rows + rb - 1) / rb;
  // About 2,048 workgroups, of at most eight rounds (131,072 x 128 by 1,024, 2,048 and 4,096 of them 12.2, 11.5 and 11.9 us, 5,003 x 7,168
  // 28.9, 28.2 and 28.6), and no more than a launch holds.
  const int64_t rounds = std::max(std::min<int64_t>((sets + 2047) / 2048, 8), (sets + kMostBlocks - 1) / kMostBlocks);
  g.rounds = (uint32_t)rounds;
  const dim3 grid((unsigned)((sets + rounds - 1) / rounds)), block(kNormThreads);
  switch (k) {
    case 1: hipLaunchKernelGGL((layer_norm_kernel<IN, OUT, SAVE, 1, PAST>), grid, block, 0, s, a, g); break;
    case 2: hipLaunchKernelGGL((layer_norm_kernel<IN, OUT, SAVE, 2, PAST>), grid, block, 0, s, a, g); break;
    case 3: hipLaunchKernelGGL((layer_norm_kernel<IN, OUT, SAVE, 3, PAST>), grid, block, 0, s, a, g); break;
    case 4: hipLaunchKernelGGL((layer_norm_kernel<IN, OUT, SAVE, 4, PAST>), grid, block, 0, s, a, g); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

template <int IN, int OUT, int SAVE>
hipError_t layer_norm_k(const NormArgs& a, const NormGrid& g, int k, hipStream_t s) {
  if constexpr (OUT != kAny) {
    if (past_caches(a.rows, (int)g.d, OUT)) return layer_norm_past<IN, OUT, SAVE, true>(a, g, k, s);
  }
  return layer_norm_past<IN, OUT, SAVE, false>(a, g, k, s);
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
  // of equals two pieces a thread for rows of several waves (with one and two 20.8 and 19.1 us of 8,192 x 2,048 with an FP8 checkpoint,
  // 20.0 and 17.6 of 16,384 x 1,024; without one 12.4 and 12.9, 12.7 and 12.6; with four and two 25.6 and 23.7 of 8,192 x 4,096)
  const RowShape shape = row_shape(d, 8, 4, d > 2048 ? 8 : d > 1024 ? 7 : 6);
  NormGrid g{};
  g.d = (uint32_t)d;
  g.log_p = (uint32_t)shape.log_p;
  g.fp32 = weight32;
  g.x32 = in_dtype == kRowsFP32;
  g.y32 = out_dtype == kRowsFP32;
  const int64_t xhs = a.heads == 1 ? 0 : a.xhs, yhs = a.heads == 1 ? 0 : a.yhs;
  const int64_t xts = a.rows == a.heads ? 0 : a.xts, yts = a.rows == a.heads ? 0 : a.yts;  // one token: no stride
  auto whole = [](const void* p) { return aligned16(p, 0, 0, kRowsBF16); };
  if (d % 8 || !aligned16(a.x, xts, xhs, in_dtype) || !aligned16(a.y, yts, yhs, out_dtype) || !whole(a.weight) || !whole(a.bias))
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
  uint32_t fp32 : 1;  // weight
  uint32_t x32 : 1;   // rows accessed one element at a time
  uint32_t dy32 : 1;
  uint32_t dx32 : 1;
  uint32_t blocks : 10;  // workgroups, at most 512
  // One workgroup writes the results itself: `part` is dweight and dbias lies so many floats behind it, or one of them alone.
  int32_t behind;
};
constexpr int32_t kParts = INT32_MIN, kWeightAlone = INT32_MIN + 1, kBiasAlone = INT32_MIN + 2;
static_assert(sizeof(NormBackArgs) + sizeof(NormBackGrid) <= 112, "launches");

namespace {

template <int X>
struct XPiece {
  Piece<X> raw;
  __device__ __forceinline__ void zero() { raw.zero(); }
  __device__ __forceinline__ void load(const NormBackArgs& a, int64_t, int64_t at, int step, int e, bool fp32) {
    raw.load(a.x, at, step, e, fp32);
  }
  __device__ __forceinline__ void floats(float* v) const { raw.floats(v); }
};
template <int FMT>
struct CodePiece {
  Stored8<FMT> raw;
  __device__ __forceinline__ void zero() { raw = Stored8<FMT>{}; }
  __device__ __forceinline__ void load(const NormBackArgs& a, int64_t row, int64_t at, int, int, bool) {
    raw.load(static_cast<const uint8_t*>(a.x), a.scale, row, at);
  }
  __device__ __forceinline__ void floats(float* v) const { raw.decode(v); }
};
template <>
struct XPiece<kCodesFP8> : CodePiece<kFP8> {};
template <>
struct XPiece<kCodesMXFP8> : CodePiece<kMXFP8> {};

// dx = rstd (g - mean(g) - h mean(g h)) with g = dy weight and h = (x - mean) rstd of each row, and this
// workgroup's sums over its rows of dy h and dy, [2][dp] behind those of the ones before it.  Statistics are the
// forward's, so both of a row's sums are formed at once; each row is read once and stays in registers, and a thread keeps the sums
// of its columns over all its rows: as few workgroups as fill the chip (512 with one piece a thread, else 256, of 512
// threads) keep what is written of them small (1,024 workgroups of 256 threads: 8,192 x 5,120 87 us against 62 then).
// Bound by memory: bf16 131,072 x 128 21.3 us with the sums, 16.1 without (6.2 TB/s), 8,192 x 5,120 52 (4.8 TB/s); from an FP8
// checkpoint with fp32 gradients 23.5 against 27.5 from bf16 rows.
template <int X, int DY, int DX, int K, bool PAST>
__global__ void __launch_bounds__(kBackThreads) layer_norm_backward_kernel(NormBackArgs a, NormBackGrid g) {
#pragma clang fp contract(off)  // as forward
  __shared__ float2 red[2][kBackThreads / kWave];
  __shared__ __attribute__((aligned(16))) float cols[kBackThreads * K * 16];  // [groups][2][K P 8]
  const int d = g.d, P = 1 << g.log_p, RB = kBackThreads >> g.log_p;
  const int lr = threadIdx.x & (P - 1), rl = threadIdx.x >> g.log_p;
  const float inv_d = 1.0f / (float)d;
  const Spread spread(X == kAny, d, lr, g.log_p);
  const int e0 = spread.first, es = spread.step, last = spread.count(d - (K - 1) * P * 8);
  auto count = [&](int k) { return k < K - 1 ? 8 : last; };
  float w[K][8], dw[K][8], db[K][8];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[k][i] = db[k][i] = 0.0f;
  const unsigned rows = a.rows;
  const int step = (int)g.blocks * RB;
  unsigned row = blockIdx.x * RB + rl;
  const bool coded = X >= kCodesFP8;
  // a checkpoint's rows are one axis
  const int xheads = coded ? 1 : a.heads;
  const int64_t xts = coded ? d : a.xts, xhs = coded ? 0 : a.xhs;
  Walk from(row, xheads, xts, xhs, step, e0), up(row, a.heads, a.dyts, a.dyhs, step, e0);
  Walk to(row, a.heads, a.dxts, a.dxhs, step, e0);
  XPiece<X> xr[K];  // the next row's elements and statistics, under way while this one is worked on
  Piece<DY> yr[K];
  float2 stats;
  auto fetch = [&](unsigned at_row) {
    const bool have = at_row < rows;
    // dy and x by turns, or one behind the other where both are fp32 (8,192 x 5,120 to bf16 80.5 us against 82.6 by turns; from an
    // FP8 checkpoint 8,192 x 8,192 by turns 97.7 against 107)
    constexpr bool kTurns = !(X == kRowsFP32 && DY == kRowsFP32);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      yr[k].zero();
      if constexpr (kTurns) xr[k].zero();
      if (have && count(k) > 0) {
        yr[k].load(a.dy, up.at + 8 * k * P, es, count(k), g.dy32);
        if constexpr (kTurns) xr[k].load(a, at_row, from.at + 8 * k * P, es, count(k), g.x32);
      }
    }
    if constexpr (!kTurns) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        xr[k].zero();
        if (have && count(k) > 0) xr[k].load(a, at_row, from.at + 8 * k * P, es, count(k), g.x32);
      }
    }
    stats = have ? a.stats[at_row] : make_float2(0.0f, 0.0f);
  };
  fetch(row);
  {
    Parameters<DY != kAny> pw[K];
#pragma unroll
    for (int k = 0; k < K; ++k) pw[k].load(a.weight, g.fp32, e0 + 8 * k * P, es, count(k));
#pragma unroll
    for (int k = 0; k < K; ++k) pw[k].floats(a.weight, g.fp32, 1.0f, w[k]);
  }
  int flip = 0;
  // rows from this round's first one on, the same in the whole workgroup
  for (int64_t left = (int64_t)rows - (row - rl); left > 0; left -= step) {
    float h[K][8], dy[K][8];
    const float mean = stats.x, rstd = stats.y;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      xr[k].floats(h[k]);
      yr[k].floats(dy[k]);
    }
    const unsigned now = row;
    row += step;  // below 2^31 + 2^18
    from.next(row, xheads, xts, xhs, e0);
    up.next(row, a.heads, a.dyts, a.dyhs, e0);
    fetch(row);
    // Elements that do not exist were read as 0, of x and of dy: their h has to be finite, no more.  Where mean rstd is not they
    // are given the mean (8,000 x 4,099 in bf16 73.2 us; 74.8 with these elements left out of every row).
    if (__any(!(fabsf(mean) * rstd <= 0x1.fffffep127f))) {
      int here = last;
      asm volatile("" : "+v"(here));  // compared here and not before the loop, where the results would take registers
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i >= here) h[K - 1][i] = mean;
    }
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        h[k][i] = (h[k][i] - mean) * rstd;
        dw[k][i] = fmaf(dy[k][i], h[k][i], dw[k][i]);
        db[k][i] += dy[k][i];
        dy[k][i] *= w[k][i];
        s[0] += dy[k][i];
        s[1] = fmaf(dy[k][i], h[k][i], s[1]);
      }
    if (!a.dx) continue;
    lanes_add(s, g.log_p);
    if (P > kWave) {
      const float2 j = join_waves(red[flip], threadIdx.x >> 6, P, make_float2(s[0], s[1]),
                                  [](float2 x, float2 y) { return make_float2(x.x + y.x, x.y + y.y); });
      flip ^= 1;
      s[0] = j.x;
      s[1] = j.y;
    }
    const float c1 = -(s[0] * inv_d) * rstd, c2 = -(s[1] * inv_d) * rstd;
    if (now < rows) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (count(k) == 0) continue;
#pragma unroll
        for (int i = 0; i < 8; ++i) dy[k][i] = fmaf(dy[k][i], rstd, fmaf(h[k][i], c2, c1));
        put<DX, PAST>(a.dx, to.at + 8 * k * P, es, count(k), g.dx32, dy[k]);
      }
    }
    to.next(row, a.heads, a.dxts, a.dxhs, e0);
  }
  if (!a.part) return;
  // The columns' sums over the workgroup's rows: over a wave's lanes, then (P < 64) over the waves or over the row groups, whose
  // sums meet in LDS.
  const int dp = norm_columns(d), width = K * P * 8, groups = min(RB, kBackThreads / kWave);
  const int group = P < kWave ? (int)threadIdx.x >> 6 : rl;
#pragma unroll
  for (int side = 0; side < 2; ++side)
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float (&c)[8] = side ? db[k] : dw[k];
      rows_add(c, g.log_p);
      if (P < kWave && lane_id() >= P) continue;
      float* to = cols + (group * 2 + side) * width + e0 + 8 * k * P;
      if (X != kAny || es == 1) {
        reinterpret_cast<f32x4*>(to)[0] = f32x4{c[0], c[1], c[2], c[3]};
        reinterpret_cast<f32x4*>(to)[1] = f32x4{c[4], c[5], c[6], c[7]};
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) to[i * es] = c[i];
      }
    }
  __syncthreads();
  for (int q = threadIdx.x; q < dp / 2; q += kBackThreads) {  // four columns
    const int side = q >= dp / 4, e0 = 4 * (q - side * (dp / 4));
    f32x4 v = *reinterpret_cast<const f32x4*>(cols + side * width + e0);
    for (int i = 1; i < groups; ++i) v += *reinterpret_cast<const f32x4*>(cols + (i * 2 + side) * width + e0);
    if (g.behind == kParts) {
      *reinterpret_cast<f32x4*>(a.part + ((int64_t)blockIdx.x * 2 + side) * dp + e0) = v;
    } else if (g.behind != (side ? kWeightAlone : kBiasAlone)) {
      float* to = a.part + (side && g.behind != kBiasAlone ? g.behind : 0) + e0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (e0 + i < d) to[i] = v[i];
    }
  }
}

// The sums of the workgroups' columns, [blocks][2][dp], in a fixed order: Q threads of a workgroup take four columns each,
// its other threads further rows, so that all loads of a thread are under way together (512 x 2 x 128 3.9 us, 256 x 2 x 5,120 4.7:
// the launch and three dependent steps; 16 threads a column one load after the other took 21).
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

template <int X, int DY, int DX, bool PAST>
hipError_t backward_past(const NormBackArgs& a, const NormBackGrid& g, int k, hipStream_t s) {
  const dim3 grid(g.blocks), block(kBackThreads);
  switch (k) {
    case 1: hipLaunchKernelGGL((layer_norm_backward_kernel<X, DY, DX, 1, PAST>), grid, block, 0, s, a, g); break;
    case 2: hipLaunchKernelGGL((layer_norm_backward_kernel<X, DY, DX, 2, PAST>), grid, block, 0, s, a, g); break;
    case 3: hipLaunchKernelGGL((layer_norm_backward_kernel<X, DY, DX, 3, PAST>), grid, block, 0, s, a, g); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

template <int X, int DY, int DX>
hipError_t backward_k(const NormBackArgs& a, const NormBackGrid& g, int k, hipStream_t s) {
  if constexpr (DX != kAny) {
    if (past_caches(a.rows, (int)g.d, DX)) return backward_past<X, DY, DX, true>(a, g, k, s);
  }
  return backward_past<X, DY, DX, false>(a, g, k, s);
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

// Of equals the most threads, whose sums of columns are fewer each (little lies between them: 8,192 x 2,048 on 256 x 1 and 128 x 2
// threads 23.1 and 22.2 us, 16,384 x 1,024 on 128 x 1 and 64 x 2 21.9 and 21.8).
RowShape back_shape(int d) { return row_shape(d, 9, 3, 9); }

}  // namespace

int norm_backward_blocks(int64_t rows, int d) {
  const RowShape shape = back_shape(d);
  const int64_t rb = kBackThreads >> shape.log_p, sets = (rows + rb - 1) / rb;
  // Few rows take one workgroup and one launch (through the binding, one against two: 128 x 128 10.0 and 12.7 us, 384 x 128 10.6 and
  // 12.6, 512 x 128 12.9 and 12.6; 32 x 201 9.9 and 12.7, 64 x 201 10.0 and 12.7, 96 x 201 12.7 both; 8 x 2,048 10.0 and 12.8, 16 x 2,048
  // 10.7 and 12.8; 2 x 8,192 10.0 and 12.9, 4 x 8,192 12.0 and 12.8).  The limits lie at a quarter to a half of where two become as fast.
  if (sets <= (d % 8 || d > 2048 ? 2 : 4)) return 1;
  // As many as the chip holds at once: sixteen waves a CU with one piece a thread, else eight (131,072 x 128 on 256, 512 and 1,020
  // workgroups 22.3, 21.5 and 23.7 us, 8,192 x 5,120 on 256 and 512 52.0 and 58.3).
  return (int)std::min<int64_t>(sets, shape.k == 1 ? 512 : 256);
}

hipError_t launch_layer_norm_backward(const NormBackArgs& args, int d, bool weight32, int x_dtype, int codes, int dy_dtype,
                                      int dx_dtype, float* dweight, float* dbias, hipStream_t s) {
  if (d <= 0 || d > kMaxNorm) return hipErrorInvalidValue;
  NormBackArgs a = args;
  if (a.rows <= 0) a.dx = nullptr;
  const bool sums = dweight || dbias;
  if (!a.dx && !sums) return hipSuccess;
  const bool rows = codes == kBF16;  // else a checkpoint's
  // rows that lie evenly over tokens and heads are one axis
  if (a.heads > 1 && a.dyts == a.heads * a.dyhs && (!rows || a.xts == a.heads * a.xhs) &&
      (!a.dx || a.dxts == a.heads * a.dxhs)) {
    a.heads = 1;
    a.dyts = a.dyhs;
    if (rows) a.xts = a.xhs;
    a.dxts = a.dxhs;
  }
  const RowShape shape = back_shape(d);
  const int blocks = norm_backward_blocks(a.rows, d);
  NormBackGrid g{};
  g.d = (uint32_t)d;
  g.log_p = (uint32_t)shape.log_p;
  g.fp32 = weight32;
  g.x32 = x_dtype == kRowsFP32;
  g.dy32 = dy_dtype == kRowsFP32;
  g.dx32 = dx_dtype == kRowsFP32;
  g.blocks = (uint32_t)blocks;
  g.behind = kParts;
  auto ok = [&](const void* p, int64_t ts, int64_t hs, int dtype) {
    return aligned16(p, a.rows == a.heads ? 0 : ts, a.heads == 1 ? 0 : hs, dtype);
  };
  const bool vec = d % 8 == 0 && aligned16(a.weight, 0, 0, kRowsBF16) && ok(a.dy, a.dyts, a.dyhs, dy_dtype) &&
                   (!rows || ok(a.x, a.xts, a.xhs, x_dtype)) && (!a.dx || ok(a.dx, a.dxts, a.dxhs, dx_dtype));
  auto launch = [&](const NormBackArgs& b) {
    if (!vec) {
      return rows ? backward_k<kAny, kAny, kAny>(b, g, shape.k, s)
                  : codes == kFP8 ? backward_k<kCodesFP8, kAny, kAny>(b, g, shape.k, s)
                                  : backward_k<kCodesMXFP8, kAny, kAny>(b, g, shape.k, s);
    }
    if (codes == kFP8) return backward_io<kCodesFP8>(b, g, shape.k, dy_dtype, dx_dtype, s);
    if (codes == kMXFP8) return backward_io<kCodesMXFP8>(b, g, shape.k, dy_dtype, dx_dtype, s);
    return x_dtype == kRowsBF16 ? backward_io<kRowsBF16>(b, g, shape.k, dy_dtype, dx_dtype, s)
                                : backward_io<kRowsFP32>(b, g, shape.k, dy_dtype, dx_dtype, s);
  };
  if (sums && blocks == 1) {  // the one workgroup writes them itself
    const int64_t behind = (int64_t)(reinterpret_cast<intptr_t>(dbias) - reinterpret_cast<intptr_t>(dweight)) / 4;
    if (dweight && dbias && (behind <= kBiasAlone || behind > INT32_MAX)) {  // too far apart: by themselves, dy's rows before dx may replace them
      NormBackArgs bias = a;
      bias.dx = nullptr;
      bias.part = dbias;
      g.behind = kBiasAlone;
      const hipError_t e = launch(bias);
      if (e != hipSuccess) return e;
      dbias = nullptr;
    }
    a.part = dweight ? dweight : dbias;
    g.behind = !dbias ? kWeightAlone : !dweight ? kBiasAlone : (int32_t)behind;
    return launch(a);
  }
  hipError_t e = launch(a);
  if (e != hipSuccess || !sums) return e;
  // 256 contiguous bytes a row where that leaves 32 workgroups or more, else 64
  const int quads = norm_columns(d) / 2;
  if (quads >= 512)
    hipLaunchKernelGGL((norm_columns_kernel<16>), dim3((quads + 15) / 16), dim3(kColumnThreads), 0, s, a.part, dweight, dbias, d, blocks);
  else
    hipLaunchKernelGGL((norm_columns_kernel<4>), dim3((quads + 3) / 4), dim3(kColumnThreads), 0, s, a.part, dweight, dbias, d, blocks);
  return hipGetLastError();
}

}  // namespace hk
