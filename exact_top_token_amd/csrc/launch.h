// Internal host-side launch interface between the C ABI (api.hip) and the
// kernel translation units.  Every launcher enqueues on `s` and returns the
// hipError_t of the launch.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <mutex>

namespace hk {

// Per-device record of the dynamic-LDS limit a kernel was given.
struct LdsLimit {
  static constexpr int kDevices = 64;
  std::atomic<int> bytes[kDevices];
  std::mutex mu;  // orders the raises, so the recorded limit is the one in force
};

// Raises `fn`'s dynamic-LDS limit to at least `bytes` on the current device,
// once: later launches that fit the limit make no runtime call (so a launch
// recorded in a stream capture after a first call outside it makes none).
// Raises never lower the limit, also when threads race.
inline hipError_t raise_dynamic_lds(const void* fn, int bytes, LdsLimit& lim) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  if (dev < 0 || dev >= LdsLimit::kDevices)
    return hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (lim.bytes[dev].load(std::memory_order_acquire) >= bytes) return hipSuccess;
  std::lock_guard<std::mutex> g(lim.mu);
  const int want = std::max(bytes, lim.bytes[dev].load(std::memory_order_relaxed));
  e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, want);
  if (e != hipSuccess) return e;
  lim.bytes[dev].store(want, std::memory_order_release);
  return hipSuccess;
}

// Device-side row count of a row-path pass enqueued without a host
// synchronisation (recovery in hytopk_select_async): the pass covers list
// entries base .. base + nq - 1 of a list whose length the device holds in
// *count; entries at or beyond that length do nothing, and a length above
// max_count (too many failures for recovery) makes the whole pass empty.
// count == null: every entry of the pass is live.
struct RowGate {
  const int* count;
  int max_count;
  int base;
  __device__ __forceinline__ int live(int nq) const {
    if (!count) return nq;
    const int c = *count;
    if (c > max_count) return 0;
    const int r = c - base;
    return r < 0 ? 0 : (r < nq ? r : nq);
  }
};

// Fused indexer scoring over causal key ranges.
//   COMPACT (rows == nullptr): keys with score >= tau[q] go to the candidate
//     buffer cand[q][0..cap) as {position, fp32 bits}; cnt[q] counts every
//     passing key, including those beyond cap.
//   ROWS (rows != nullptr): the score of every causal key is written to
//     rows[e * row_stride + key] for launch entry e.
// Launch entry e scores query qlist[e] (or q_offset + e when qlist is null).
struct ScoreArgs {
  const uint8_t* q;
  const uint8_t* k;
  const float* w;
  const void* q_scale;   // fp32 [n] (FP8) or E8M0 [n][H][d/32] (MX)
  const void* k_scale;   // fp32 [L] (FP8) or E8M0 [L][d/32] (MX)
  const float* tau;
  int* cnt;
  uint2* cand;
  float* rows;
  const int* qlist;
  const int* qpos;     // [n] query positions, or null (q_start + i)
  const int* qfirst;   // [n] first key of each query's context, or null (0)
  int64_t row_stride;
  int L;
  int q_start;
  int q_offset;
  int nq;
  int H;
  int cap;
  int nsplit;
  int split_len;
  int reverse;         // 1: walk each launch entry's key tiles from last to first
  RowGate gate;        // ROWS: device-side count of live entries (count null: all nq)
};

hipError_t launch_score(const ScoreArgs& a, int d, int fmt, hipStream_t s);
int score_group_queries(int fmt);  // queries per workgroup of the score kernel

// Per-query sampled threshold: tau[q] = the r-th largest of the M_q sample
// scores at positions floor(j * ctx / M_q).
struct SampleArgs {
  const uint8_t* q;
  const uint8_t* k;
  const float* w;
  const void* q_scale;   // fp32 [n] (FP8) or E8M0 [n][H][d/32] (MX)
  const void* k_scale;   // fp32 [L] (FP8) or E8M0 [L][d/32] (MX)
  float* tau;
  const int* qpos;
  const int* qfirst;
  int L;
  int q_start;
  int n;
  int H;
  int topk;
  int M;
  int oversample;
};

hipError_t launch_sample_tau(const SampleArgs& a, int d, int fmt, hipStream_t s);

// Replay: out[q][j] = I(q_start + q, idx[q][j]) (-inf where idx is outside [0, L)).
struct ReplayArgs {
  const uint8_t* q;
  const uint8_t* k;
  const float* w;
  const void* q_scale;   // fp32 [n] (FP8) or E8M0 [n][H][d/32] (MX)
  const void* k_scale;   // fp32 [L] (FP8) or E8M0 [L][d/32] (MX)
  const int* idx;
  float* out;
  int L;
  int n;
  int H;
  int topk;
};

hipError_t launch_replay(const ReplayArgs& a, int d, int fmt, hipStream_t s);

// Device counters of one selection call.
struct DevStats {
  int n_overflow;
  int n_underk;
  int n_failed;
  int cand_max;
  unsigned long long cand_total;
  int pad[2];
};

hipError_t launch_zero(int* cnt, int n, DevStats* st, hipStream_t s);

// The device status words of hytopk_select_async (HYTOPK_ASYNC_STATUS_WORDS
// int32): [0] 1 when more than max_recover queries failed (their rows were
// not recovered), [1] failures, [2] overflows, [3] under-k queries, [4] the
// largest candidate count, [5], [6] the candidate total (low, high 32 bits),
// [7] 0.
hipError_t launch_async_status(const DevStats* st, int max_recover, int32_t* out, hipStream_t s);

// Check: flags queries whose candidate count is above cap or below
// min(k, ctx) and appends them to `failed`.
hipError_t launch_check(const int* cnt, int n, const int* qpos, const int* qfirst, int q_start,
                        int L, int topk, int cap, DevStats* st, int* failed, hipStream_t s);

// Exact top-k of each passing query's candidates (failed queries are skipped).
hipError_t launch_cand_select(const int* cnt, const uint2* cand, int n, const int* qpos,
                              const int* qfirst, int q_start, int topk, int cap, int L,
                              int* out_idx, float* out_score, hipStream_t s);

// Exact top-k of score rows: entry e is row rows[e * row_stride] of query
// qlist[e] (or q_offset + e).
hipError_t launch_row_topk(const float* rows, int64_t row_stride, const int* qlist, int q_offset,
                           int nq, const int* qpos, const int* qfirst, int q_start, int topk, int L,
                           int* out_idx, float* out_score, RowGate gate, hipStream_t s);

// Exact top-k of a few long score rows, each row split over `nchunk`
// workgroups of `chunk_len` entries (recovery and the full rescore): three
// radix passes over the rows find each row's k-th largest key, an emission
// pass keeps the entries above it and the lowest-position entries equal to
// it, and one workgroup per row sorts the kept entries.  Same result as
// launch_row_topk.
struct RowSelArgs {
  const float* rows;
  int64_t row_stride;
  const int* qlist;    // entry e is query qlist[e] (or q_offset + e)
  int q_offset;
  int nq;
  const int* qpos;
  const int* qfirst;
  int q_start;
  int topk;
  int L;
  int nchunk;          // workgroups per row
  int chunk_len;       // entries per workgroup (a multiple of 1024)
  void* scratch;       // row_select_scratch_bytes(nq, nchunk, topk) bytes, 256-byte aligned
  int* out_idx;
  float* out_score;
  RowGate gate;        // device-side count of live entries (count null: all nq)
};

hipError_t launch_row_select_split(const RowSelArgs& a, hipStream_t s);
size_t row_select_scratch_bytes(int nrows, int nchunk, int topk);
int row_select_max_chunks(int64_t L);
// Chunking of rows of up to maxctx entries for nq rows (nchunk <= row_select_max_chunks(L)).
void row_select_chunks(int nq, int64_t maxctx, int64_t L, int& nchunk, int& chunk_len);
constexpr int kRowSplitMaxRows = 128;  // more rows than this fill the GPU one workgroup per row

// LDS bytes cand_select needs for this cap / k (the host checks the limit).
size_t cand_select_lds_bytes(int cap, int topk);


// Indexer backward at the replayed entries (backward.hip).
struct BwdArgs {
  const uint16_t* q;   // bf16 bits [n][H][d]
  const uint16_t* k;   // bf16 bits [L][d]
  const float* w;      // [n][H]
  const int* idx;      // [n][topk]
  const float* dsc;    // [n][topk] upstream gradient of each replayed score
  float* dq;           // [n][H][d] or null
  float* dw;           // [n][H] or null
  float* u;            // [nq * bwd_padded_k(topk)][d] dk rows of the chunk's entries, or null
  const float* q_scale;  // [n] per-token FP8 scales of q and k (q, k then hold the codes
  const float* k_scale;  // [L] as bf16), or null for bf16 / dequantized MX inputs
  int L;
  int H;
  int topk;
  int q0;              // first query of the chunk
  int nq;              // queries in the chunk
};

hipError_t launch_bwd_query(const BwdArgs& a, int d, hipStream_t s);
// Scaled-format q or k ([rows][d] elements) as bf16 bits for the backward.
hipError_t launch_bwd_dequant(const void* x, const void* scale, int64_t rows, int d, int fmt,
                              uint16_t* out, hipStream_t s);

struct DkArgs {
  const int* idx;      // the chunk's [nq][topk] indices (entry e = row-major position)
  int L;
  int N;               // entries in the chunk (nq * topk)
  int topk;
  uint32_t* k0;        // [N] sort ping-pong buffers
  uint32_t* v0;
  uint32_t* k1;
  uint32_t* v1;
  uint32_t* hist;      // [bwd_sort_hist_count(N)]: per-tile digit counts, digit totals
};

// Groups the chunk's entries by key: stable sort of (key position, u row)
// by key (padding last); returns the sorted keys and rows.
hipError_t launch_bwd_sort(const DkArgs& a, const uint32_t** sorted_keys,
                           const uint32_t** sorted_rows, hipStream_t s);
// dk[s] = (or +=) the sum of the u rows of key s's run, in sorted order.
hipError_t launch_bwd_segments(const uint32_t* sorted_keys, const uint32_t* sorted_rows, int N,
                               int L, const float* u, float* dk, bool accumulate, int d,
                               hipStream_t s);
int bwd_padded_k(int topk);  // key slots per query in the u buffer
hipError_t launch_fill_zero(float* p, int64_t n, hipStream_t s);
size_t bwd_sort_hist_count(int64_t N);

// ---- rotary positions, the quantised cache (rows.hip)

constexpr int kRowsBF16 = 0, kRowsFP32 = 1;            // hytopk_rows_dtype
constexpr int kRotHalf = 0, kRotInterleaved = 1;       // hytopk_rotary_layout

// What a launch takes on the host grows from 2.8 to 3.6 us where a kernel's arguments pass 112 bytes,
// the grid's and block's sizes (gridDim, blockDim: about 70 bytes) among them.  The kernels of rows.hip,
// norm.hip and loss.hip are often shorter than that, so their arguments stay within it and they read neither.

// A rotation (freq == null: none) and the tokens' positions.
struct RotArgs {
  const double* freq;  // [dim/2] radians a position; with several axes, behind them int [dim/2]: each pair's
  const int* pos;      // [n][axes] positions, or null (pos0 + i on every axis)
  union {
    int pos0;          // without positions
    int axes;          // with them; at least 1
  };
  float gain;          // factor on the cosines
  float turn;          // factor on the sines: gain, or -gain for the transposed rotation
  int dim;
};

struct RotaryArgs {
  const void* x;
  void* y;
  int64_t xts, xhs, yts, yhs;  // token and head strides in elements
  RotArgs rot;
  int n, heads, d, first;      // first: where the rotated part begins
};

hipError_t launch_rotary(const RotaryArgs& a, int layout, int in_dtype, int out_dtype, hipStream_t s);

struct CacheWriteArgs {
  const void* x;
  int64_t ts, hs;
  uint8_t* codes;
  void* scale;
  const int* slots;    // [n] cache rows, or null (start + i)
  int* claim;          // [L] last row naming each slot, or null (each row looks for a later one)
  RotArgs rot;
  int n, L, start, first;
};

// Rows up to this many look for a later row of the same slot by themselves; more take
// `claim`.  FP8 rows of 128 on the GPU: 512, 1,024, 2,048 rows 6.8, 9.6, 15.5 us looking and
// 8.0 claiming, whose two more launches take the host another 5 us.
constexpr int kClaimRows = 1024;
hipError_t launch_cache_write(const CacheWriteArgs& a, int heads, int d, int layout, int in_dtype, int fmt,
                              hipStream_t s);

struct CacheReadArgs {
  const uint8_t* codes;
  const void* scale;
  const int* slots;
  void* out;
  int L, start, n;
  int row;             // elements of a row (heads * d)
};

hipError_t launch_cache_read(const CacheReadArgs& a, int out_dtype, int fmt, hipStream_t s);

// ---- layer norm and its 8-bit checkpoints (norm.hip)

constexpr int kMaxNorm = 8192;  // elements of a row

struct NormArgs {
  const void* x;
  void* y;
  int64_t xts, xhs, yts, yhs;  // token and head strides in elements
  const void* weight;  // [d], or null (1)
  const void* bias;    // [d], or null (0)
  float2* stats;       // [rows] mean and reciprocal deviation, or null
  uint8_t* codes;      // the checkpoint's [rows][d] and its scales
  void* scale;
  int rows, heads;     // rows = tokens * heads
  float eps;
};

// save: kFP8, kMXFP8, or kBF16 for no checkpoint.
hipError_t launch_layer_norm(const NormArgs& a, int d, bool weight32, int in_dtype, int out_dtype, int save,
                             hipStream_t s);

struct NormBackArgs {
  const void* x;       // rows, or a checkpoint's codes
  const void* dy;
  void* dx;            // or null
  union {
    struct { int64_t xts, xhs; };
    const void* scale;  // of a checkpoint
  };
  int64_t dyts, dyhs, dxts, dxhs;
  const void* weight;  // [d], or null (1)
  const float2* stats;  // [rows]
  float* part;         // [norm_backward_blocks][2][norm_columns(d)] of more than one workgroup, or null: no sums
  int rows, heads;
};

// codes: kFP8 or kMXFP8 for a checkpoint, kBF16 for rows of x_dtype.
hipError_t launch_layer_norm_backward(const NormBackArgs& a, int d, bool weight32, int x_dtype, int codes, int dy_dtype,
                                      int dx_dtype, float* dweight, float* dbias, hipStream_t s);
int norm_backward_blocks(int64_t rows, int d);
// Columns of a workgroup's sums: d rounded up to whole 16 bytes.
__host__ __device__ constexpr int norm_columns(int d) { return (d + 3) / 4 * 4; }

// ---- attention mass at the selected entries, index loss (loss.hip)

struct MassArgs {
  const uint16_t* q;   // bf16 [n][heads][d]
  const uint16_t* k;   // bf16 [L][groups][d]
  const int* idx;      // [n][topk]
  const float* lse;    // [n][heads] natural, or null
  float2* part;        // [n][nsplit][rows]: (max, sum) of each split (mass_keeps_parts, without lse)
  float* mass;         // [n][topk]
  int L, n, heads, groups, topk;
  float scale2;        // softmax scale * log2(e)
  float inv_heads;
  int nsplit;          // workgroups of a query
  int split_len;       // entries of a split, a multiple of 64
};

// Rows of q as the kernel holds them: the heads of a key head padded to 16.
int64_t mass_rows(int heads, int groups);
void mass_splits(int64_t n, int topk, int d, int& nsplit, int& split_len);
bool mass_supports(int d);
int64_t mass_most_queries(int d);  // a call has fewer
bool mass_keeps_parts(int d, int nsplit);  // whether the statistics go through `part`
hipError_t launch_attention_mass(const MassArgs& a, int d, hipStream_t s);

struct LossArgs {
  const float* score;
  const float* mass;
  const float* weight;  // or null (1)
  float* loss;          // or null
  float* dscore;        // or null
  int n, k;
};

hipError_t launch_index_loss(const LossArgs& a, hipStream_t s);

}  // namespace hk
