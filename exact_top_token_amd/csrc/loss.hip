// The indexer's training target and loss: the attention's probability mass at
// the selected entries (MFMA over gathered key rows), and the divergence of
// the selection's softmax from it with its gradient.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "common.h"
#include "launch.h"
#include "tile.h"

namespace hk {

namespace {

static_assert(sizeof(MassArgs) + 2 * sizeof(int) <= 112, "launches");

constexpr int kMassThreads = 256;
constexpr int kMassWaves = kMassThreads / kWave;
constexpr int kWideSteps = 16;     // k-steps of a row from which on a wave holds two blocks and no second buffer
constexpr int kItemTiles = 8;      // head tiles whose softmax statistics a wave keeps in registers
constexpr float kNoMax = -3.0e38f;  // maximum of nothing: finite, so that differences stay defined
constexpr float kLazy = 8.0f;      // a maximum moves when exceeded by 2^8: sums stay below 2^19

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// (max, sum) of two parts of a softmax sum in base 2.
__device__ __forceinline__ float2 join(float2 a, float2 b) {
  const float m = fmaxf(a.x, b.x);
  return make_float2(m, a.y * exp2_fast(a.x - m) + b.y * exp2_fast(b.x - m));
}

// lse log2(e) as a rounded reference m and the factor 2^-(what the rounding left).
__device__ __forceinline__ void lse_reference(float l, float& m, float& rl) {
  constexpr float kHi = 1.44269502162933349609375f, kLo = 1.925963033500011e-8f;
  m = l * kHi;
  rl = fabsf(m) < 3.0e38f ? exp2_fast(-fmaf(l, kLo, fmaf(l, kHi, -m))) : 1.0f;
}

// The sum over the four rows of 16 lanes, in each of them.
__device__ __forceinline__ float add_rows(float x) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// (max, sum) of a row over the splits' parts ([nsplit][rows], from the row's first one), by the four
// lanes of a quad together.
__device__ __forceinline__ float2 join_parts(const float2* part, int nsplit, int rows) {
  const int sub = lane_id() & 3;
  float2 p = make_float2(kNoMax, 0.0f);
#pragma unroll 4
  for (int sp = sub; sp < nsplit; sp += 4) p = join(p, part[(int64_t)sp * rows]);
  p = join(p, make_float2(__shfl_xor(p.x, 1), __shfl_xor(p.y, 1)));
  return join(p, make_float2(__shfl_xor(p.x, 2), __shfl_xor(p.y, 2)));
}

// How the heads of a query lie on 16-row tiles: each key head's heads padded to
// whole tiles.
struct HeadTiles {
  int per_group;  // heads of a key head
  int tiles;      // tiles of a key head
  __host__ __device__ HeadTiles(int heads, int groups)
      : per_group(heads / groups), tiles((heads / groups + 15) / 16) {}
  // head of row r of tile t, or -1
  __device__ __forceinline__ int head(int t, int r) const {
    const int g = t / tiles, h = (t - g * tiles) * 16 + r;
    return h < per_group ? g * per_group + h : -1;
  }
};

// LDS of a workgroup that gathers its keys into registers: per row of q the row itself,
// (max, 1 / sum) for the mass and the waves' (max, sum) for the statistics; per entry its
// index and, where there are several passes, its sum.
constexpr int kLdsBytes = 160 * 1024;
constexpr int kMassLongest = 2048;        // entries of a split, at most
constexpr int kMassLdsSmall = 40 * 1024;  // enough passes to keep this where key heads allow it
constexpr int mass_row_bytes(int d, int mode, int waves) {
  return 2 * d + (mode != 0 ? 8 : 0) + (mode != 1 ? 8 * waves : 0);
}

// Tiles of a pass over a query's heads: whole key heads within kMassLdsSmall (their
// keys differ, so passes cost nothing), or else as much of one key head
// as the LDS holds (more than one pass then gathers its keys again).
int mass_pass_tiles(int heads, int groups, int row_bytes) {
  const HeadTiles ht(heads, groups);
  const int tile = 16 * row_bytes;
  if (groups == 1 && ht.tiles * tile <= kLdsBytes - 4 * kMassLongest) return ht.tiles;
  const int fit = (kLdsBytes - 8 * kMassLongest) / tile;
  const int small = kMassLdsSmall / tile / ht.tiles * ht.tiles;
  return std::min(groups * ht.tiles, std::max(small, std::min(ht.tiles, fit)));
}

// MODE 0: (max, sum) of a split; 1: mass, from lse or from the splits' parts; 2: both at once
// (one workgroup a query).
//
// A workgroup of W waves holds one query, its heads in passes of `pass` tiles: their q
// rows lie in LDS in MFMA operand order (lane l of tile t, k-step s reads the 16
// bytes at ((t * NK + s) * 64 + l) * 16), and each wave takes every W-th step of KB blocks
// of 16 entries, whose key rows it gathers from memory straight into operand
// registers, one step ahead with two buffers (BUF).  A key row is read once a pass for all
// heads of its key head.
//   statistics: D = K Q^T, so that a lane holds four keys of one head and
//     keeps one (max, sum) per tile;
//   mass: D = Q K^T, so that a lane holds four heads of one key and adds
//     their exponentials into one number.
// The two gather the keys twice: the logits of a query (heads x k in fp32)
// are as large as a CU's whole register file, and written out they
// would be as many bytes as the key rows.
//
// Rows of 1 KB and more fill a wave's registers with one block; there the reads of q from
// LDS bound the kernel, so two blocks share each of them, without a second buffer, and
// eight waves overlap gathers with products (2,048 queries x 128 heads of 576 x 1,024 entries with
// lse: 453 us, one block with a second buffer and four waves 653).
template <int NK, int MODE, int W, int KB, int BUF>
__global__ void __launch_bounds__(W * kWave) mass_kernel(MassArgs a, int pass) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  constexpr int D = NK * 32, THREADS = W * kWave;
  const HeadTiles ht(a.heads, a.groups);
  const int T = a.groups * ht.tiles, cap = pass * 16;
  uint8_t* qs = lds;
  float* ms = reinterpret_cast<float*>(qs + (size_t)cap * D * 2);           // [cap] reference exponent
  float* rs = ms + (MODE != 0 ? cap : 0);                                   // [cap] 1 / sum
  float2* red = reinterpret_cast<float2*>(rs + (MODE != 0 ? cap : 0));      // [waves][cap]
  int* ids = reinterpret_cast<int*>(red + (MODE != 1 ? W * cap : 0));       // [split_len]
  float* sums = reinterpret_cast<float*>(ids + a.split_len);                // [split_len], several passes only

  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int col = lane & 15, grp = lane >> 4;
  // Workgroups go to the 8 XCDs in turn; each XCD takes a contiguous run of
  // queries, whose selections overlap, so that their keys meet in its L2.
  const int q = [&] {
    const int nx = 8, b = blockIdx.x, x = b % nx;
    const int base = a.n / nx, extra = a.n % nx;
    return x * base + min(x, extra) + b / nx;
  }();
  const int split = blockIdx.y;
  const int j0 = split * a.split_len, nj = min(a.split_len, a.topk - j0);
  for (int j = tid; j < a.split_len; j += THREADS) {
    const int id = j < nj ? a.idx[(int64_t)q * a.topk + j0 + j] : -1;
    ids[j] = (unsigned)id < (unsigned)a.L ? id : -1;
  }
  const int nstep = (nj + 16 * KB - 1) / (16 * KB);
  const int mine = wave < nstep ? (nstep - wave + W - 1) / W : 0;  // wave-uniform
  const int row_elems = a.groups * D;
  // the wave's i-th step, key head g; id: the lane's entries (split_len covers every whole step)
  auto gather = [&](int i, int g, bf16x8 (*f)[NK], int* id) {
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      id[kb] = i < mine ? ids[((wave + i * W) * KB + kb) * 16 + col] : -1;
      const uint16_t* p = a.k + (int64_t)max(id[kb], 0) * row_elems + g * D + grp * 8;
      if (id[kb] >= 0) {
#pragma unroll
        for (int s = 0; s < NK; ++s) f[kb][s] = *reinterpret_cast<const bf16x8*>(p + s * 32);
      } else {
#pragma unroll
        for (int s = 0; s < NK; ++s) f[kb][s] = bf16x8{};
      }
    }
  };
  auto qfrag = [&](int t, int s) {  // t: tile of the pass
    return *reinterpret_cast<const bf16x8*>(qs + ((t * NK + s) * 64 + lane) * 16);
  };

  for (int c0 = 0; c0 < T; c0 += pass) {
    const int c1 = min(T, c0 + pass), rows = (c1 - c0) * 16;
    if (c0) __syncthreads();  // the last pass is through with the LDS
    const u32x4 zero = {0u, 0u, 0u, 0u};
    for (int e = tid; e < rows * NK * 4; e += THREADS) {
      const int r = e / (NK * 4), c = e - r * (NK * 4);
      const int h = ht.head(c0 + (r >> 4), r & 15);
      u32x4 v = zero;
      if (h >= 0)
        v = *reinterpret_cast<const u32x4*>(a.q + ((int64_t)q * a.heads + h) * D + c * 8);
      const int slot = ((r >> 4) * NK + (c >> 2)) * 64 + (c & 3) * 16 + (r & 15);
      *reinterpret_cast<u32x4*>(qs + slot * 16) = v;
    }
    if constexpr (MODE == 1) {
      for (int e = tid; e < rows * 4; e += THREADS) {  // a quad per row
        const int r = e >> 2, h = ht.head(c0 + (r >> 4), r & 15);
        float m = 0.0f, rl = 0.0f;
        if (h >= 0 && a.lse) {
          lse_reference(a.lse[(int64_t)q * a.heads + h], m, rl);
        } else if (h >= 0) {
          const float2 p = join_parts(a.part + (int64_t)q * a.nsplit * (T * 16) + c0 * 16 + r, a.nsplit, T * 16);
          m = p.x;
          rl = p.y == 0.0f ? 0.0f : 1.0f / p.y;
        }
        if ((e & 3) == 0) {
          ms[r] = m;
          rs[r] = rl;
        }
      }
    }
    __syncthreads();

    if constexpr (MODE != 1) {
      // Items: up to kItemTiles tiles of one key head.
      for (int t0 = c0; t0 < c1;) {
        const int g = t0 / ht.tiles;
        const int nt = min(min(kItemTiles, (g + 1) * ht.tiles - t0), c1 - t0);
        float m[kItemTiles], l[kItemTiles];
#pragma unroll
        for (int t = 0; t < kItemTiles; ++t) { m[t] = kNoMax; l[t] = 0.0f; }
        bf16x8 f[BUF][KB][NK];
        int id[BUF][KB];
        if constexpr (BUF == 2) gather(0, g, f[0], id[0]);
        for (int i0 = 0; i0 < mine; i0 += BUF) {
#pragma unroll
          for (int u = 0; u < BUF; ++u) {
            if (i0 + u >= mine) break;  // wave-uniform
            if constexpr (BUF == 2) gather(i0 + u + 1, g, f[1 - u], id[1 - u]);
            else gather(i0, g, f[0], id[0]);
            unsigned live[KB];
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
              live[kb] = (unsigned)(__ballot(id[u][kb] >= 0) & 0xffffu) >> (4 * grp);
#pragma unroll
            for (int t = 0; t < kItemTiles; ++t) {
              if (t >= nt) break;  // uniform
              f32x4 acc[KB];
#pragma unroll
              for (int kb = 0; kb < KB; ++kb) acc[kb] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
              for (int s = 0; s < NK; ++s) {
                const bf16x8 qf = qfrag(t0 - c0 + t, s);
#pragma unroll
                for (int kb = 0; kb < KB; ++kb)
                  acc[kb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f[u][kb][s], qf, acc[kb], 0, 0, 0);
              }
#pragma unroll
              for (int kb = 0; kb < KB; ++kb) {
                float x[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  x[e] = (live[kb] >> e) & 1u ? acc[kb][e] * a.scale2 : -__builtin_inff();
                const float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
                if (top > m[t] + kLazy) {
                  l[t] *= exp2_fast(m[t] - top);
                  m[t] = top;
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) l[t] += exp2_fast(x[e] - m[t]);
              }
            }
          }
        }
#pragma unroll
        for (int t = 0; t < kItemTiles; ++t) {
          if (t >= nt) break;
          float2 p = make_float2(m[t], l[t]);
          p = join(p, make_float2(__shfl_xor(p.x, 16), __shfl_xor(p.y, 16)));
          p = join(p, make_float2(__shfl_xor(p.x, 32), __shfl_xor(p.y, 32)));
          if (grp == 0) red[wave * cap + (t0 - c0 + t) * 16 + col] = p;
        }
        t0 += nt;
      }
      __syncthreads();
      for (int r = tid; r < rows; r += THREADS) {
        float2 p = red[r];
#pragma unroll
        for (int w = 1; w < W; ++w) p = join(p, red[w * cap + r]);
        if constexpr (MODE == 0) {
          a.part[((int64_t)q * a.nsplit + split) * (T * 16) + c0 * 16 + r] = p;
        } else {
          ms[r] = p.x;
          rs[r] = ht.head(c0 + (r >> 4), r & 15) < 0 || p.y == 0.0f ? 0.0f : 1.0f / p.y;
        }
      }
      if constexpr (MODE == 2) __syncthreads();
    }

    if constexpr (MODE != 0) {
      // Steps of (KB blocks, key head of the pass), the key head innermost.
      const int g0 = c0 / ht.tiles, g1 = (c1 + ht.tiles - 1) / ht.tiles;
      const int steps = mine * (g1 - g0);
      bf16x8 f[BUF][KB][NK];
      int id[KB];
      float o[KB];
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) o[kb] = 0.0f;
      int step = 0, g = g0;  // at hand
      int nb = 0, ng = g0;   // being gathered
      auto next = [&](bf16x8 (*dst)[NK]) {
        gather(nb, ng, dst, id);
        if (++ng == g1) { ng = g0; ++nb; }
      };
      if constexpr (BUF == 2) next(f[0]);
      for (int i0 = 0; i0 < steps; i0 += BUF) {
#pragma unroll
        for (int u = 0; u < BUF; ++u) {
          if (i0 + u >= steps) break;  // wave-uniform
          if constexpr (BUF == 2) next(f[1 - u]);
          else next(f[0]);
          const int ta = max(c0, g * ht.tiles) - c0, tb = min(c1, (g + 1) * ht.tiles) - c0;
          for (int t = ta; t < tb; ++t) {
            f32x4 acc[KB];
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) acc[kb] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int s = 0; s < NK; ++s) {
              const bf16x8 qf = qfrag(t, s);
#pragma unroll
              for (int kb = 0; kb < KB; ++kb)
                acc[kb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(qf, f[u][kb][s], acc[kb], 0, 0, 0);
            }
            const f32x4 m = *reinterpret_cast<const f32x4*>(ms + t * 16 + 4 * grp);
            const f32x4 r = *reinterpret_cast<const f32x4*>(rs + t * 16 + 4 * grp);
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                o[kb] = fmaf(exp2_fast(fmaf(acc[kb][e], a.scale2, -m[e])), r[e], o[kb]);
          }
          if (++g == g1) {
            g = g0;
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
              float sum = add_rows(o[kb]);
              const int j = ((wave + step * W) * KB + kb) * 16 + col;
              if (grp == 0) {  // the wave's own entries: no other wave reads or writes them
                if (c0) sum += sums[j];
                if (c1 < T) sums[j] = sum;
                else if (j < nj) a.mass[(int64_t)q * a.topk + j0 + j] = ids[j] >= 0 ? sum * a.inv_heads : 0.0f;
              }
              o[kb] = 0.0f;
            }
            ++step;
          }
        }
      }
    }
  }
}

template <int NK, int MODE>
hipError_t mass_launch(const MassArgs& a, hipStream_t s) {
  constexpr bool wide = NK >= kWideSteps;
  constexpr int W = wide ? 8 : 4, KB = wide ? 2 : 1, BUF = wide ? 1 : 2;
  static LdsLimit lim;
  constexpr int row = mass_row_bytes(NK * 32, MODE, W);
  const int pass = mass_pass_tiles(a.heads, a.groups, row);
  const bool several = pass < mass_rows(a.heads, a.groups) / 16;
  const int lds = pass * 16 * row + a.split_len * (several ? 8 : 4);
  hipError_t e = raise_dynamic_lds((const void*)mass_kernel<NK, MODE, W, KB, BUF>, lds, lim);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((mass_kernel<NK, MODE, W, KB, BUF>), dim3((unsigned)a.n, (unsigned)a.nsplit),
                     dim3(W * kWave), (size_t)lds, s, a, pass);
  return hipGetLastError();
}

template <int NK>
hipError_t mass_d(const MassArgs& a, hipStream_t s) {
  if (a.lse) return mass_launch<NK, 1>(a, s);
  if constexpr (NK < kWideSteps) {
    if (a.nsplit == 1) return mass_launch<NK, 2>(a, s);
  }
  hipError_t e = mass_launch<NK, 0>(a, s);
  return e != hipSuccess ? e : mass_launch<NK, 1>(a, s);
}

constexpr int kBuckets = 64;

// Inclusive sum over the wave's lanes up to each: within rows of 16, then over the rows.
__device__ __forceinline__ int wave_prefix_incl(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false);  // from 1, 2, 4, 8 lanes below
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);  // a row's last lane to the next row
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);  // lane 31 to the upper half
  return x;
}

constexpr int kWaveWords = kMassLongest / kMassThreads;  // runs of 64 entries of a wave, at most

// Orders a workgroup's entries by bucket, stably.  A wave holds `runs` runs of 64 of them, wave after
// wave: key[c], or -1 for padding.  An entry goes to bucket key >> shift (below 63), padding to the last one;
// place[c] is where it comes.  Returns the live entries.  Every wave counts its own entries, in its
// own row of count [wave][bucket] (256 ints of LDS); one barrier, and every wave sums what precedes its part of
// each bucket, a bucket a lane.
__device__ __forceinline__ int order_entries(const int* key, int runs, int shift, int* count, int* place) {
  static_assert(kBuckets == kWave, "a lane per bucket");
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  count[wave * kBuckets + lane] = 0;
  auto bucket = [&](int c) { return key[c] >= 0 ? key[c] >> shift : kBuckets - 1; };
#pragma unroll
  for (int c = 0; c < kWaveWords; ++c) {
    if (c >= runs) break;  // wave-uniform
    const int b = bucket(c);
    uint64_t same = ~0ull;  // lanes of the same bucket
#pragma unroll
    for (int bit = 0; bit < 6; ++bit) {
      const uint64_t set = __ballot((b >> bit) & 1);
      same &= (b >> bit) & 1 ? set : ~set;
    }
    const int rank = __builtin_amdgcn_mbcnt_hi((unsigned)(same >> 32), __builtin_amdgcn_mbcnt_lo((unsigned)same, 0u));
    int* to = &count[wave * kBuckets + b];
    place[c] = *to + rank;
    if (rank == 0) *to = place[c] + __builtin_popcountll(same);
  }
  __syncthreads();
  int all = 0, lower = 0;  // of the lane's bucket; of the waves below
#pragma unroll
  for (int w = 0; w < kMassWaves; ++w) {
    const int n = count[w * kBuckets + lane];
    all += n;
    lower += w < wave ? n : 0;
  }
  const int before = wave_prefix_incl(all) - all, mine = before + lower;
#pragma unroll
  for (int c = 0; c < kWaveWords; ++c) {
    if (c < runs) place[c] += __shfl(mine, bucket(c));
  }
  return __builtin_amdgcn_readlane(before, kBuckets - 1);
}

// The same with the key rows staged through LDS, for rows of 128 or 256 bytes.
// A direct-to-LDS load fetches rows whole, where gathering the operand layout gives
// every lane its own 16 bytes of another row (from a cache that holds the keys the
// one reaches 25 TB/s on this chip and the other 9.5).  Each wave owns two stages of 16 rows
// and waits for its own loads by count; the q rows of a pass (PT tiles of one
// key head) stay in registers.  With the statistics and the mass in one workgroup
// (MODE 2) the mass walks the wave's blocks from the last to the first, so that the
// rows still in LDS and in the caches are used again.
//
// gw waves (1, 2 or 4) take key heads side by side, the others the blocks: with short splits of
// several key heads the passes over them, each a few dependent loads long, run at once.
//
// What bounds it is the rate of instructions of a SIMD (per block of 16 entries and 64 heads of 128:
// 16 MFMAs, 16 exponentials, 32 fused multiplies) and, where the keys come from the
// memory-side cache, its 8.2 TB/s.  So waves count for more than loads in flight or
// gathered bytes: two stages and three waves per SIMD measured 278 us (2,048 queries x 64
// heads x 2,048 entries of 131,072 keys), three stages and two waves 300; eight waves a workgroup
// that kept five of sixteen blocks' logits in registers and four stages in LDS,
// for 44% fewer bytes, 301.  Rows of 128 bytes: four stages 15.8 us against 14.8 (301 queries x 32
// heads on 4 key heads x 500 entries of 131,072 keys, with lse).
//
// With ORDER the entries are walked by key: 63 buckets of 2^order
// keys, in the given order within one, padding last.  The workgroups of an XCD, which run side by
// side, then pass over the same part of the keys at the same time and meet in its L2: 2,048 x 64 heads
// of 128 x 2,048 of 131,072 keys 238 us against 264, with lse 135 against 150.  Blocks behind
// the last live entry are left out.
template <int NK, int PT, int MODE, bool ORDER>
__global__ void __launch_bounds__(kMassThreads, PT > 4 ? 2 : 3) mass_staged_kernel(MassArgs a, int gw, int order) {
  constexpr int D = NK * 32, RB = D * 2, NCH = RB / 16, OPS = 16 * RB / 1024;
  constexpr int KPI = 1024 / RB;  // rows of a load
  constexpr int W = kMassWaves;
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
  const HeadTiles ht(a.heads, a.groups);
  const int T = a.groups * ht.tiles;
  uint8_t* ring = lds;                                                // [2][waves][16 rows]
  float* ms = reinterpret_cast<float*>(ring + 2 * W * 16 * RB);       // [gw][PT * 16]
  float* rs = ms + gw * PT * 16;                                      // [gw][PT * 16]
  float2* red = reinterpret_cast<float2*>(rs + gw * PT * 16);         // [waves][PT * 16]
  uint64_t* live64 = reinterpret_cast<uint64_t*>(red + W * PT * 16);  // [split_len / 64] live entries
  // [split_len] where an entry's key row begins, in 16-byte pieces (padding fetches row 0, and live64 leaves it out)
  uint32_t* rows_at = reinterpret_cast<uint32_t*>(live64 + a.split_len / 64);
  // [gw][split_len] fp32 bits; with one pass each sum takes the place of its row, which is through by then
  uint32_t* sums = rows_at + (T > PT ? a.split_len : 0);
  // [split_len] with ORDER: the entries' places in the row
  uint16_t* place = reinterpret_cast<uint16_t*>(sums + gw * a.split_len);

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, grp = lane >> 4;
  const int gi = wave & (gw - 1), bi = wave / gw, bw = W / gw;
  ms += gi * PT * 16;
  rs += gi * PT * 16;
  const int q = [&] {  // a contiguous run of queries per XCD
    const int nx = 8, b = blockIdx.x, x = b % nx;
    const int base = a.n / nx, extra = a.n % nx;
    return x * base + min(x, extra) + b / nx;
  }();
  const int split = blockIdx.y;
  const int j0 = split * a.split_len, nj = min(a.split_len, a.topk - j0);
  uint32_t* const all_sums = sums;
  sums += gi * a.split_len;
  const int words = a.split_len / 64;  // split_len is a multiple of 64
  // blocks of this wave, bi + i * bw, up to the last live entry
  auto blocks = [&] {
    const uint64_t w = lane < words ? live64[lane] : 0, any = __ballot(w != 0);
    if (!any) return 0;
    const int top = 63 - __builtin_clzll(any);
    const int nblk = top * 4 + (63 - __builtin_clzll(live64[top])) / 16 + 1;
    return __builtin_amdgcn_readfirstlane(bi < nblk ? (nblk - bi + bw - 1) / bw : 0);
  };
  uint8_t* const ring0 = ring + wave * 16 * RB;  // stage s: + s * SLOT
  constexpr int SLOT = W * 16 * RB;
  int dsw[OPS];  // load p fetches this chunk of its row (the stage's swizzle)
#pragma unroll
  for (int p = 0; p < OPS; ++p) dsw[p] = 16 * ((lane % NCH) ^ key_swz<NCH>(p * KPI + lane / NCH));
  typedef uint16_t __attribute__((may_alias)) live_bits;
  const live_bits* live16 = reinterpret_cast<const live_bits*>(live64);
  const uint32_t* my_rows = rows_at + bi * 16 + lane / NCH;
  // the wave's i-th block, from kg (the key head's first byte), into its stage i % 2
  auto issue = [&](int i, const uint8_t* kg) {
    uint8_t* to = ring0 + (i & 1) * SLOT;
    uint32_t at[OPS];  // read together, ahead of the loads
#pragma unroll
    for (int p = 0; p < OPS; ++p) at[p] = my_rows[i * bw * 16 + p * KPI];
#pragma unroll
    for (int p = 0; p < OPS; ++p) lds_dma16(kg + dsw[p] + ((uint64_t)at[p] << 4), to + p * 1024);
  };
  const uint32_t ring_at = lds_addr(ring0);
  uint32_t chunk_at[NK];
#pragma unroll
  for (int s = 0; s < NK; ++s) chunk_at[s] = ring_at + col * RB + (((4 * s + grp) ^ key_swz<NCH>(col)) * 16);
  auto frags = [&](int i, bf16x8* f) {
    uint32_t ad[NK];
    u32x4 r[NK];
#pragma unroll
    for (int s = 0; s < NK; ++s) ad[s] = chunk_at[s] + (i & 1) * SLOT;
    lds_read_chunks<NK>(ad, r);
#pragma unroll
    for (int s = 0; s < NK; ++s) f[s] = __builtin_bit_cast(bf16x8, r[s]);
  };

  // The q rows of a pass, tiles ta on of key head gp + gi, and (MODE 1) their softmax statistics.
  bf16x8 qf[PT][NK];
  auto take = [&](int gp, int ta) {
    const int g = gp + gi, c0 = g * ht.tiles + ta, nt = g < a.groups ? min(PT, ht.tiles - ta) : 0;
#pragma unroll
    for (int t = 0; t < PT; ++t) {
      const int h = t < nt ? ht.head(c0 + t, col) : -1;
      const uint16_t* p = a.q + ((int64_t)q * a.heads + max(h, 0)) * D + grp * 8;
#pragma unroll
      for (int s = 0; s < NK; ++s) qf[t][s] = *reinterpret_cast<const bf16x8*>(p + s * 32);
    }
    if (nt < PT || ht.per_group % 16) {  // rows of no head; apart, so that all loads are under way at once
#pragma unroll
      for (int t = 0; t < PT; ++t) {
        if (t < nt && ht.head(c0 + t, col) >= 0) continue;
#pragma unroll
        for (int s = 0; s < NK; ++s) qf[t][s] = bf16x8{};
      }
    }
    if constexpr (MODE == 1) {
      for (int e = bi * kWave + lane; e < PT * 64; e += bw * kWave) {  // a quad per row, by this key head's waves
        const int r = e >> 2, h = (r >> 4) < nt ? ht.head(c0 + (r >> 4), r & 15) : -1;
        float m = 0.0f, rl = 0.0f;
        if (h >= 0 && a.lse) {
          lse_reference(a.lse[(int64_t)q * a.heads + h], m, rl);
        } else if (h >= 0) {
          const float2 p = join_parts(a.part + (int64_t)q * a.nsplit * (T * 16) + c0 * 16 + r, a.nsplit, T * 16);
          m = p.x;
          rl = p.y == 0.0f ? 0.0f : 1.0f / p.y;
        }
        if ((e & 3) == 0) {
          ms[r] = m;
          rs[r] = rl;
        }
      }
    }
  };
  // The entries into LDS.
  const int* idx = a.idx + (int64_t)q * a.topk + j0;
  auto row_of = [&](int key) { return key >= 0 ? (uint32_t)key * (uint32_t)(a.groups * NCH) : 0u; };
  const int w0 = wave * words / W, runs = (wave + 1) * words / W - w0;  // the wave's: 64 w0 on
  int key[kWaveWords];
#pragma unroll
  for (int c = 0; c < kWaveWords; ++c) key[c] = idx[min((w0 + c) * 64 + lane, nj - 1)];  // all under way at once
  take(0, 0);
#pragma unroll
  for (int c = 0; c < kWaveWords; ++c) {
    const bool on = (w0 + c) * 64 + lane < nj && (unsigned)key[c] < (unsigned)a.L;
    key[c] = on ? key[c] : -1;
  }
  if constexpr (ORDER) {
    int to[kWaveWords];
    const int live = order_entries(key, runs, order, reinterpret_cast<int*>(ring), to);
    const int left = live - tid * 64;
    if (tid < words) live64[tid] = left >= 64 ? ~0ull : left > 0 ? (1ull << left) - 1 : 0;
#pragma unroll
    for (int c = 0; c < kWaveWords; ++c) {
      if (c >= runs) break;  // wave-uniform
      rows_at[to[c]] = row_of(key[c]);
      place[to[c]] = (uint16_t)((w0 + c) * 64 + lane);
    }
  } else {
#pragma unroll
    for (int c = 0; c < kWaveWords; ++c) {
      if (c >= runs) break;  // wave-uniform
      const uint64_t live = __ballot(key[c] >= 0);
      rows_at[(w0 + c) * 64 + lane] = row_of(key[c]);
      if (lane == 0) live64[w0 + c] = live;
    }
  }
  if (T > PT && MODE != 0) {  // what no block reaches
    for (int j = tid; j < gw * a.split_len; j += kMassThreads) all_sums[j] = 0u;
  }
  __syncthreads();
  const int have = blocks();

  for (int gp = 0, ta = 0;;) {
    // tiles of this pass: ta .. ta + nt - 1 of key head g, c0 on of the query
    const int g = gp + gi, c0 = g * ht.tiles + ta;
    const bool in = g < a.groups, first = gp == 0 && ta == 0;
    const int nt = in ? min(PT, ht.tiles - ta) : 0, mine = in ? have : 0;
    const bool last = gp + gw >= a.groups && ta + PT >= ht.tiles;
    const uint8_t* kg = reinterpret_cast<const uint8_t*>(a.k) + g * RB;

    if constexpr (MODE != 1) {
      float m[PT], l[PT];
#pragma unroll
      for (int t = 0; t < PT; ++t) { m[t] = kNoMax; l[t] = 0.0f; }
      HK_WAIT_VM(0);  // from here on the wave counts its stages' loads alone
      if (mine) issue(0, kg);
      for (int i = 0; i < mine; ++i) {
        if (i + 1 < mine) {
          issue(i + 1, kg);
          HK_WAIT_VM(OPS);
        } else {
          HK_WAIT_VM(0);
        }
        bf16x8 f[NK];
        frags(i, f);
        // lane: keys 4 grp .. + 3 of the block, head col of each tile
        const unsigned all = __builtin_amdgcn_readfirstlane(live16[bi + i * bw]), live = all >> (4 * grp);
        // Tiles in pairs whose products are under way together, one branch a pair for a maximum that moves
        // and a copy of it all for blocks with padding (a branch a tile for each: 96 heads of 128 298 us against
        // 272, 64 heads 232 against 228).
        constexpr int TG = PT % 2 ? PT : 2;
        auto add = [&](auto padded) {
#pragma unroll
          for (int t0 = 0; t0 < PT; t0 += TG) {
            f32x4 acc[TG];
#pragma unroll
            for (int u = 0; u < TG; ++u) acc[u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int s = 0; s < NK; ++s)
#pragma unroll
              for (int u = 0; u < TG; ++u)
                acc[u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f[s], qf[t0 + u][s], acc[u], 0, 0, 0);
            // padding takes no part, whatever its row holds
            auto value = [&](int u, int e) {
              const float y = fmaf(acc[u][e], a.scale2, -m[t0 + u]);
              return !padded.value || ((live >> e) & 1u) ? y : -__builtin_inff();
            };
            float over = -__builtin_inff();
#pragma unroll
            for (int u = 0; u < TG; ++u)
#pragma unroll
              for (int e = 0; e < 4; ++e) over = fmaxf(over, value(u, e));
            if (__any(over > kLazy)) {
#pragma unroll
              for (int u = 0; u < TG; ++u) {
                float top = -__builtin_inff();
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  top = !padded.value || ((live >> e) & 1u) ? fmaxf(top, acc[u][e] * a.scale2) : top;
                if (top > m[t0 + u] + kLazy) {
                  l[t0 + u] *= exp2_fast(m[t0 + u] - top);
                  m[t0 + u] = top;
                }
              }
            }
#pragma unroll
            for (int u = 0; u < TG; ++u)
              l[t0 + u] += (exp2_fast(value(u, 0)) + exp2_fast(value(u, 1))) + (exp2_fast(value(u, 2)) + exp2_fast(value(u, 3)));
          }
        };
        if (all == 0xffffu) add(std::false_type{});
        else add(std::true_type{});
      }
#pragma unroll
      for (int t = 0; t < PT; ++t) {
        float2 p = make_float2(m[t], l[t]);
        p = join(p, make_float2(__shfl_xor(p.x, 16), __shfl_xor(p.y, 16)));
        p = join(p, make_float2(__shfl_xor(p.x, 32), __shfl_xor(p.y, 32)));
        if (grp == 0) red[wave * PT * 16 + t * 16 + col] = p;
      }
      __syncthreads();
      for (int r = bi * kWave + lane; r < PT * 16; r += bw * kWave) {
        float2 p = red[gi * PT * 16 + r];
        for (int w = 1; w < bw; ++w) p = join(p, red[(gi + w * gw) * PT * 16 + r]);
        if constexpr (MODE == 0) {
          if (r < nt * 16) a.part[((int64_t)q * a.nsplit + split) * (T * 16) + c0 * 16 + r] = p;
        } else {
          const bool head = (r >> 4) < nt && ht.head(c0 + (r >> 4), r & 15) >= 0;
          ms[r] = p.x;
          rs[r] = !head || p.y == 0.0f ? 0.0f : 1.0f / p.y;
        }
      }
      __syncthreads();
    }

    if constexpr (MODE != 0) {
      HK_WAIT_VM(0);
      // Blocks from the last to the first, block i in stage i % 2; after the statistics of
      // the same pass the last two still lie there.
      if constexpr (MODE == 1) {
        if (mine) issue(mine - 1, kg);
      }
      for (int i = mine - 1; i >= 0; --i) {
        if constexpr (MODE == 1) {
          if (i > 0) {
            issue(i - 1, kg);
            HK_WAIT_VM(OPS);
          } else {
            HK_WAIT_VM(0);
          }
        } else if (i < mine - 2) {  // fetched since: one younger block at most
          if (i > 0) HK_WAIT_VM(OPS);
          else HK_WAIT_VM(0);
        }
        bf16x8 f[NK];
        frags(i, f);
        if constexpr (MODE == 2) {
          if (i >= 2) issue(i - 2, kg);  // into the stage that has just been read
        }
        float o = 0.0f;  // lane: heads 4 grp .. + 3 of each tile, key col
#pragma unroll
        for (int t = 0; t < PT; ++t) {
          f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int s = 0; s < NK; ++s)
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(qf[t][s], f[s], acc, 0, 0, 0);
          const f32x4 m = *reinterpret_cast<const f32x4*>(ms + t * 16 + 4 * grp);
          const f32x4 r = *reinterpret_cast<const f32x4*>(rs + t * 16 + 4 * grp);
#pragma unroll
          for (int e = 0; e < 4; ++e) o = fmaf(exp2_fast(fmaf(acc[e], a.scale2, -m[e])), r[e], o);
        }
        o = add_rows(o);
        if (grp == 0) {  // the wave's own entries: no other wave reads or writes them
          const int blk = bi + i * bw, j = blk * 16 + col;
          const bool on = (live16[blk] >> col) & 1;
          sums[j] = on ? __float_as_uint(first ? o : __uint_as_float(sums[j]) + o) : 0u;
        }
      }
      if (last) {
        __syncthreads();
        auto total = [&](int j) {
          float o = __uint_as_float(all_sums[j]);
          for (int k = 1; k < gw; ++k) o += __uint_as_float(all_sums[k * a.split_len + j]);
          return o * a.inv_heads;
        };
        if constexpr (ORDER) {  // back to their places, within the LDS
          float o[kWaveWords];
          int to[kWaveWords];
#pragma unroll
          for (int c = 0; c < kWaveWords; ++c) {
            const int j = tid + c * kMassThreads;
            o[c] = j < a.split_len ? total(j) : 0.0f;
            to[c] = j < a.split_len ? place[j] : -1;
          }
          __syncthreads();
#pragma unroll
          for (int c = 0; c < kWaveWords; ++c)
            if (to[c] >= 0) all_sums[to[c]] = __float_as_uint(o[c]);
          __syncthreads();
          for (int j = tid; j < nj; j += kMassThreads)
            a.mass[(int64_t)q * a.topk + j0 + j] = __uint_as_float(all_sums[j]);
        } else {
          for (int j = tid; j < nj; j += kMassThreads) a.mass[(int64_t)q * a.topk + j0 + j] = total(j);
        }
      }
    }
    ta += PT;
    if (ta >= ht.tiles) { ta = 0; gp += gw; }
    if (last) break;
    __syncthreads();
    take(gp, ta);
    __syncthreads();
  }
}

// Entries by key (in buckets of 2^order keys, 63 at most) where that saves more than it takes: queries
// that fill the chip, long rows, keys beyond two L2s (8 MiB).  Given order against by key, 64 heads of
// 128 on one key head, without lse: 2,048 queries x 2,048 entries of 131,072 keys 264 us, 238; x 1,024 135,
// 128; x 512 70, 72; x 2,048 of 65,536 keys 231, 202; of 32,768 (8 MiB) 197, 199; 600 x 2,048 92, 83;
// 301 x 2,048 54, 58; 8 key heads, 2,048 x 2,048 of 65,536 1,976, 1,328.  Passes of more than four
// tiles run two waves per SIMD: 128 heads with lse 185, 187.
template <int NK>
int mass_order(const MassArgs& a) {
  if (a.n <= 512 || a.topk < 1024 || (int64_t)a.L * a.groups * NK * 64 <= int64_t(8) << 20) return -1;
  int order = 0;
  while ((a.L - 1) >> order >= kBuckets - 1) ++order;
  return order;
}

template <int NK, int PT, int MODE, bool ORDER>
hipError_t mass_staged_launch(const MassArgs& a, int order, hipStream_t s) {
  static LdsLimit lim;
  // Key heads side by side where queries are few and their sums take no more LDS than one row of
  // 2,048 (without lse, 301 queries x 4 key heads x 500 entries: 26 us against 32; 2,048 queries: 146
  // against 127, for they fill the chip without).
  int gw = 1;
  while (a.n <= 512 && gw < kMassWaves && 2 * gw <= a.groups && 2 * gw * a.split_len <= 2048) gw *= 2;
  const bool apart = mass_rows(a.heads, a.groups) > PT * 16;  // sums beside the rows
  const int lds = 2 * kMassWaves * 16 * NK * 64 + PT * 16 * 8 * (gw + kMassWaves) + a.split_len / 8 +
                  a.split_len * 4 * (apart ? 1 + gw : 1) + (ORDER ? a.split_len * 2 : 0);
  hipError_t e = raise_dynamic_lds((const void*)mass_staged_kernel<NK, PT, MODE, ORDER>, lds, lim);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((mass_staged_kernel<NK, PT, MODE, ORDER>), dim3((unsigned)a.n, (unsigned)a.nsplit),
                     dim3(kMassThreads), (size_t)lds, s, a, gw, order);
  return hipGetLastError();
}

template <int NK, int PT, int MODE>
hipError_t mass_staged_mode(const MassArgs& a, hipStream_t s) {
  if constexpr (PT <= 4 && MODE != 0) {
    const int order = mass_order<NK>(a);
    if (order >= 0) return mass_staged_launch<NK, PT, MODE, true>(a, order, s);
  }
  return mass_staged_launch<NK, PT, MODE, false>(a, -1, s);
}

template <int NK, int PT>
hipError_t mass_staged_pt(const MassArgs& a, hipStream_t s) {
  if (a.lse) return mass_staged_mode<NK, PT, 1>(a, s);
  if (a.nsplit == 1) return mass_staged_mode<NK, PT, 2>(a, s);
  hipError_t e = mass_staged_mode<NK, PT, 0>(a, s);
  return e != hipSuccess ? e : mass_staged_mode<NK, PT, 1>(a, s);
}

// Tiles of a pass: those of a key head, up to eight (q rows in 4 NK registers a tile).  From five on
// a SIMD holds two waves instead of three, which costs less than gathering the keys once more for
// every four tiles: 128 heads of 128 with lse 232 us against 283, without 384 against 523, 96 heads
// 176 against 277 (2,048 queries, 2,048 of 131,072 keys).
template <int NK>
hipError_t mass_staged(const MassArgs& a, hipStream_t s) {
  const int tiles = HeadTiles(a.heads, a.groups).tiles;
  if (tiles == 1) return mass_staged_pt<NK, 1>(a, s);
  if (tiles == 2) return mass_staged_pt<NK, 2>(a, s);
  if (tiles == 3) return mass_staged_pt<NK, 3>(a, s);
  if (tiles == 4) return mass_staged_pt<NK, 4>(a, s);
  if (tiles <= 6) return mass_staged_pt<NK, 6>(a, s);
  return mass_staged_pt<NK, 8>(a, s);
}

}  // namespace

int64_t mass_rows(int heads, int groups) { return (int64_t)groups * HeadTiles(heads, groups).tiles * 16; }

// Splits of a query's entries so that few queries still fill the chip, each with a block of 16
// entries for every wave: about 256 workgroups where one fills a CU (wide heads), 1,024 of the
// narrowest rows, 512 else.  64 queries x 64 heads of 128 x 2,048 with lse: 256, 512, 768, 1,024
// workgroups 10.1, 9.9, 11.4, 14.5 us; 100 x 128 heads of 576 x 1,024: 34.6, 46.4, 57.8, 68.1;
// 301 x 32 heads of 64 on 4 key heads x 500 of 4,096 keys: 512, 768, 1,024, 2,048 workgroups
// 15.4, 10.8, 9.8, 9.7, and 301 x 64 heads on one key head x 2,000 of 131,072: 26.3, 19.7, 18.2,
// 20.0.
void mass_splits(int64_t n, int topk, int d, int& nsplit, int& split_len) {
  const int most = (topk + 63) / 64;
  const int64_t workgroups = d / 32 >= kWideSteps ? 256 : d <= 64 ? 1024 : 512;
  const int64_t want = std::max<int64_t>(1, std::min<int64_t>(most, workgroups / std::max<int64_t>(1, n)));
  split_len = (int)(((topk + want - 1) / want + 63) / 64 * 64);
  nsplit = (topk + split_len - 1) / split_len;
}

bool mass_keeps_parts(int d, int nsplit) { return nsplit > 1 || d / 32 >= kWideSteps; }

bool mass_supports(int d) {
  return d == 64 || d == 96 || d == 128 || d == 192 || d == 256 || d == 512 || d == 576;
}

int64_t mass_most_queries(int d) { return int64_t(1) << (d / 32 >= kWideSteps ? 23 : 24); }

hipError_t launch_attention_mass(const MassArgs& a, int d, hipStream_t s) {
  if (a.n <= 0) return hipSuccess;
  // the staged kernels count key rows in 16-byte pieces of 32 bits: tables below 64 GiB
  const bool pieces = (int64_t)a.L * a.groups * (d / 8) < int64_t(1) << 32;
  switch (d) {
    case 64: return pieces ? mass_staged<2>(a, s) : mass_d<2>(a, s);
    case 96: return mass_d<3>(a, s);
    case 128: return pieces ? mass_staged<4>(a, s) : mass_d<4>(a, s);
    case 192: return mass_d<6>(a, s);
    case 256: return mass_d<8>(a, s);
    case 512: return mass_d<16>(a, s);
    case 576: return mass_d<18>(a, s);
    default: return hipErrorInvalidValue;
  }
}

// ------------------------------------------------------------ index loss

namespace {

constexpr int kLossThreads = 256;
constexpr int64_t kMostLossBlocks = int64_t(1) << 22;  // workgroups walk the rest in steps of so many

__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) x += __shfl_xor(x, off);
  return x;
}
__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) x = fmaxf(x, __shfl_xor(x, off));
  return x;
}

// One wave a row, the row's N entries per lane in registers, so that scores
// and mass are read once and the gradient is written once.  With p = softmax
// and t = mass / sum, each term t (ln t - ln p) - t + p is non-negative and
// their sum is the loss (both t and p sum to 1): no cancellation between large terms.
template <int N, bool VEC, bool PAST>
__global__ void __launch_bounds__(kLossThreads, 4) index_loss_kernel(LossArgs a) {
  const int lane = threadIdx.x & 63;
  constexpr int W = kLossThreads / kWave;
  for (int64_t i = (int64_t)blockIdx.x * W + (threadIdx.x >> 6); i < a.n; i += kMostLossBlocks * W) {
    const int64_t at = i * a.k;
    float s[N], t[N];
    // entry j of this lane: pieces of four (VEC), or every 64th
    auto entry = [&](int e) { return VEC ? (e >> 2) * 256 + lane * 4 + (e & 3) : e * 64 + lane; };
    if constexpr (VEC) {
#pragma unroll
      for (int c = 0; c < N / 4; ++c) {
        const int j = c * 256 + lane * 4;
        const bool in = j < a.k;  // k is a multiple of four
        const f32x4 sv = in ? *reinterpret_cast<const f32x4*>(a.score + at + j) : f32x4{};
        const f32x4 tv = in ? *reinterpret_cast<const f32x4*>(a.mass + at + j) : f32x4{};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[4 * c + e] = in ? sv[e] : -__builtin_inff();
          t[4 * c + e] = tv[e];
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const int j = entry(e);
        s[e] = j < a.k ? a.score[at + j] : -__builtin_inff();
        t[e] = j < a.k ? a.mass[at + j] : 0.0f;
      }
    }
    float top = -__builtin_inff(), total = 0.0f;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const bool live = !(s[e] == -__builtin_inff());
      t[e] = live ? t[e] : 0.0f;  // dead entries hold anything
      top = fmaxf(top, s[e]);
      total += t[e];
    }
    top = wave_max(top);
    total = wave_sum(total);
    const bool none = total == 0.0f;  // also a row without a live entry
    const float ref = top == -__builtin_inff() ? 0.0f : top;
    // Powers and logarithms in base 2 (one instruction each).  The score's part of ln p is taken as it is: at the
    // type's lowest value it is finite, and times log2(e) it would not be (that product once more, for p, and the masses' factor
    // below cost 2%: 8,192 x 2,048 40.9 us against 40.1).
    constexpr float kLog2e = 1.44269504088896341f;
    float sum = 0.0f;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      s[e] -= ref;
      sum += exp2_fast(s[e] * kLog2e);
    }
    sum = wave_sum(sum);
    // Sums far from 1, infinity among them, are taken again of scaled masses, so that total and 1 / total stay within
    // fp32's normal range.
    float up = 1.0f;
    if (!(total >= 0x1p-100f && total <= 0x1p100f)) {
      up = total < 1.0f ? 0x1p100f : 0x1p-40f;
      total = 0.0f;
#pragma unroll
      for (int e = 0; e < N; ++e) total = fmaf(t[e], up, total);
      total = wave_sum(total);
    }
    const float lsum = __builtin_amdgcn_logf(sum), rsum = 1.0f / sum, rtotal = 1.0f / total;
    const float w = a.weight ? a.weight[i] : 1.0f;
    float loss = 0.0f;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float p = exp2_fast(s[e] * kLog2e) * rsum, q = t[e] * up * rtotal;
      // the logarithm instruction takes no subnormals; their term is nothing
      const float lq = __builtin_amdgcn_logf(fmaxf(q, 0x1p-126f));
      const float kl = q == 0.0f ? 0.0f : q * fmaf(lq + lsum, 0.693147180559945309f, -s[e]);
      loss += kl - q + p;
      t[e] = w * (p - q);
    }
    loss = wave_sum(loss);
    if (a.loss && lane == 0) a.loss[i] = none ? 0.0f : w * loss;
    if (a.dscore) {
      if constexpr (VEC) {
#pragma unroll
        for (int c = 0; c < N / 4; ++c) {
          const int j = c * 256 + lane * 4;
          if (j >= a.k) continue;
          f32x4 v;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = none ? 0.0f : t[4 * c + e];
          f32x4* to = reinterpret_cast<f32x4*>(a.dscore + at + j);
          if constexpr (PAST) __builtin_nontemporal_store(v, to);
          else *to = v;
        }
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const int j = entry(e);
          if (j < a.k) a.dscore[at + j] = none ? 0.0f : t[e];
        }
      }
    }
  }
}

template <bool VEC, bool PAST>
hipError_t index_loss_vec(const LossArgs& a, hipStream_t s) {
  const int64_t w = kLossThreads / kWave;
  const dim3 grid((unsigned)std::min<int64_t>((a.n + w - 1) / w, kMostLossBlocks)), block(kLossThreads);
  if (a.k <= 256) hipLaunchKernelGGL((index_loss_kernel<4, VEC, PAST>), grid, block, 0, s, a);
  else if (a.k <= 512) hipLaunchKernelGGL((index_loss_kernel<8, VEC, PAST>), grid, block, 0, s, a);
  else if (a.k <= 1024) hipLaunchKernelGGL((index_loss_kernel<16, VEC, PAST>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((index_loss_kernel<32, VEC, PAST>), grid, block, 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_index_loss(const LossArgs& a, hipStream_t s) {
  if (a.n <= 0) return hipSuccess;
  auto off = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 != 0; };
  const bool vec = a.k % 4 == 0 && !off(a.score) && !off(a.mass) && !off(a.dscore);
  if (!vec) return index_loss_vec<false, false>(a, s);
  // a gradient larger than the chip's L2 caches (32 MiB) goes past them: 8,192 x 2,048 (64 MiB)
  // 40.9 us against 44.4; a smaller one stays for the backward that reads it
  const bool past = a.dscore && (int64_t)a.n * a.k * 4 >= int64_t(32) << 20;
  return past ? index_loss_vec<true, true>(a, s) : index_loss_vec<true, false>(a, s);
}

}  // namespace hk
