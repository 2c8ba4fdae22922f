// C ABI of the selection library: argument validation, workspace layout and
// the launch sequence of hytopk_select / hytopk_replay /
// hytopk_baseline_select (declared in include/hytopk.h).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <mutex>
#include <string>
#include <vector>

#include "hytopk.h"
#include "launch.h"

constexpr size_t kNoAllocBytes = size_t(64) << 20;
static_assert(kNoAllocBytes == HYTOPK_NOALLOC_SCRATCH_BYTES, "header and library disagree");
// The workspace of hytopk_select_noalloc (see scratch_address below).
static __device__ __align__(256) uint8_t scratch[kNoAllocBytes];

namespace {

thread_local std::string g_err;

int fail(int code, const char* msg) {
  g_err = msg;
  return code;
}

int hip_fail(hipError_t e, const char* where) {
  g_err = std::string(where) + ": " + hipGetErrorString(e);
  return HYTOPK_EHIP;
}

#define HK_HIP(expr, where)                     \
  do {                                          \
    hipError_t e_ = (expr);                     \
    if (e_ != hipSuccess) return hip_fail(e_, where); \
  } while (0)

// ------------------------------------------------------------------ tracing

struct TraceRec {
  std::string name;
  hipEvent_t a, b;
};

struct Tracer {
  std::mutex mu;
  bool on = false;
  std::vector<TraceRec> pending;
  std::vector<hipEvent_t> pool;
  std::map<std::string, std::pair<int, double>> acc;
};

Tracer& tracer() {
  static Tracer t;
  return t;
}

hipEvent_t take_event(Tracer& t) {
  if (!t.pool.empty()) {
    hipEvent_t e = t.pool.back();
    t.pool.pop_back();
    return e;
  }
  hipEvent_t e = nullptr;
  if (hipEventCreate(&e) != hipSuccess) return nullptr;
  return e;
}

// Brackets one launch with events when tracing is on.
struct Span {
  const char* name;
  hipStream_t s;
  hipEvent_t a = nullptr;
  Span(const char* nm, hipStream_t st) : name(nm), s(st) {
    Tracer& t = tracer();
    std::lock_guard<std::mutex> g(t.mu);
    if (!t.on) return;
    a = take_event(t);
    if (a && hipEventRecord(a, s) != hipSuccess) {  // no timing for this span
      (void)hipGetLastError();  // handled here; keep it from the next launch check
      t.pool.push_back(a);
      a = nullptr;
    }
  }
  ~Span() {
    if (!a) return;
    Tracer& t = tracer();
    std::lock_guard<std::mutex> g(t.mu);
    hipEvent_t b = take_event(t);
    if (b && hipEventRecord(b, s) == hipSuccess) {
      t.pending.push_back(TraceRec{name, a, b});
      return;
    }
    if (b) (void)hipGetLastError();  // handled here; keep it from the next launch check
    t.pool.push_back(a);  // the span is dropped; both events go back to the pool
    if (b) t.pool.push_back(b);
  }
};

constexpr size_t kAlign = 256;
constexpr int kMaxK = 2048;
constexpr int kMaxCap = 16384;
constexpr int kMaxM = 16384;
constexpr size_t kLdsLimit = 160 * 1024 - 10 * 1024;  // gfx950 LDS minus static scratch

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

struct Params {
  int m_min, m_max, m_div, oversample, cap, max_recover, force_path, rows_chunk;
};

int check_problem(const hytopk_problem* p) {
  if (!p) return fail(HYTOPK_EINVAL, "problem is NULL");
  if (p->L <= 0 || p->n <= 0 || p->q_start < 0) return fail(HYTOPK_EINVAL, "L, n must be > 0 and q_start >= 0");
  if (!p->q_pos && p->q_start + p->n > p->L) return fail(HYTOPK_EINVAL, "q_start + n > L");
  if (p->L >= (int64_t(1) << 31)) return fail(HYTOPK_EUNSUPPORTED, "L >= 2^31");
  if (p->n >= (int64_t(1) << 31)) return fail(HYTOPK_EUNSUPPORTED, "n >= 2^31");
  if (p->q_start >= (int64_t(1) << 31)) return fail(HYTOPK_EUNSUPPORTED, "q_start >= 2^31");
  if (p->k <= 0) return fail(HYTOPK_EINVAL, "k must be > 0");
  if (p->k > kMaxK) return fail(HYTOPK_EUNSUPPORTED, "k > 2048");
  if (p->H <= 0 || p->d <= 0) return fail(HYTOPK_EINVAL, "H, d must be > 0");
  if (p->H > 64) return fail(HYTOPK_EUNSUPPORTED, "H > 64");
  if (p->dtype == HYTOPK_BF16) {
    if (p->d != 64 && p->d != 128) return fail(HYTOPK_EUNSUPPORTED, "bf16 needs d in {64, 128}");
  } else if (p->dtype == HYTOPK_FP8_E4M3 || p->dtype == HYTOPK_MXFP8_E4M3 ||
             p->dtype == HYTOPK_MXFP4_E2M1) {
    if (p->d != 128) return fail(HYTOPK_EUNSUPPORTED, "fp8 and MX formats need d = 128");
  } else {
    return fail(HYTOPK_EINVAL, "unknown dtype");
  }
  return HYTOPK_OK;
}

Params resolve(const hytopk_problem* p, const hytopk_params* prm) {
  Params r{};
  r.m_min = (prm && prm->m_min) ? prm->m_min : 4096;
  r.m_max = (prm && prm->m_max) ? prm->m_max : 8192;
  r.m_div = (prm && prm->m_div) ? prm->m_div : 128;
  r.oversample = (prm && prm->oversample) ? prm->oversample : 3;
  r.cap = (prm && prm->cap) ? prm->cap : 6 * p->k;
  r.max_recover = (prm && prm->max_recover) ? prm->max_recover : 64;
  r.force_path = prm ? prm->force_path : HYTOPK_PATH_AUTO;
  // rows buffer: max_recover rows by default (one recovery pass)
  const int64_t dflt = std::min<int64_t>(p->n, std::max(1, r.max_recover));
  r.rows_chunk = (prm && prm->rows_chunk) ? prm->rows_chunk : (int)dflt;
  return r;
}

int check_params(const hytopk_problem* p, const Params& r) {
  if (r.m_min < 1 || r.m_max < r.m_min || r.m_div < 1 || r.oversample < 1 || r.cap < 1 ||
      r.max_recover < 0 || r.rows_chunk < 1)
    return fail(HYTOPK_EINVAL, "invalid threshold parameters");
  if (r.force_path != HYTOPK_PATH_AUTO && r.force_path != HYTOPK_PATH_ROWS_ALL)
    return fail(HYTOPK_EINVAL, "unknown force_path");
  // the rows buffer (rows_chunk x L fp32) must stay far from size_t overflow
  if (std::min<int64_t>(r.rows_chunk, p->n) * p->L > (int64_t(1) << 40))
    return fail(HYTOPK_EUNSUPPORTED, "rows_chunk * L > 2^40");
  if (r.m_max > kMaxM) return fail(HYTOPK_EUNSUPPORTED, "m_max > 16384");
  if (r.cap > kMaxCap) return fail(HYTOPK_EUNSUPPORTED, "cap > 16384");
  if (hk::cand_select_lds_bytes(r.cap, p->k) > kLdsLimit)
    return fail(HYTOPK_EUNSUPPORTED, "cap and k exceed the LDS of one workgroup");
  return HYTOPK_OK;
}

int sample_count(const hytopk_problem* p, const Params& r) {
  int64_t m = std::max<int64_t>(r.m_min, p->L / r.m_div);
  return (int)std::min<int64_t>(m, r.m_max);
}

struct Layout {
  size_t tau, cnt, failed, stats, cand, rows, split, total;
  int rows_n;
};

// Scratch of the split row top-k for up to `rows` rows (0 when that many rows
// fill the GPU one workgroup per row).
size_t split_bytes(const hytopk_problem* p, int rows) {
  if (rows > hk::kRowSplitMaxRows) return 0;
  return hk::row_select_scratch_bytes(rows, hk::row_select_max_chunks(p->L), p->k);
}

Layout layout(const hytopk_problem* p, const Params& r) {
  Layout l{};
  size_t off = 0;
  const size_t n = (size_t)p->n;
  l.tau = off; off = align_up(off + n * 4);
  l.cnt = off; off = align_up(off + n * 4);
  l.failed = off; off = align_up(off + n * 4);
  l.stats = off; off = align_up(off + sizeof(hk::DevStats));
  l.cand = off; off = align_up(off + n * (size_t)r.cap * 8);
  l.rows_n = (int)std::min<int64_t>(r.rows_chunk, p->n);
  l.rows = off; off = align_up(off + (size_t)l.rows_n * (size_t)p->L * 4);
  l.split = off; off = align_up(off + split_bytes(p, l.rows_n));
  l.total = off;
  return l;
}

int check_ws(void* ws, size_t bytes, size_t need) {
  if (!ws) return fail(HYTOPK_EWORKSPACE, "workspace is NULL");
  if (reinterpret_cast<uintptr_t>(ws) % kAlign) return fail(HYTOPK_EWORKSPACE, "workspace not 256-byte aligned");
  if (bytes < need) return fail(HYTOPK_EWORKSPACE, "workspace too small");
  return HYTOPK_OK;
}

int check_inputs(const hytopk_problem* p, const void* q, const void* qs, const void* k,
                 const void* ks, const float* w) {
  if (!q || !k || !w) return fail(HYTOPK_EINVAL, "q, k and w must be non-NULL");
  if (p->dtype != HYTOPK_BF16 && (!qs || !ks))
    return fail(HYTOPK_EINVAL, "fp8 and MX formats need q_scale and k_scale");
  auto off = [](const void* x, uintptr_t a) { return reinterpret_cast<uintptr_t>(x) % a != 0; };
  if (off(q, 16) || off(k, 16)) return fail(HYTOPK_EINVAL, "q and k must be 16-byte aligned");
  if (off(w, 4) || off(qs, 4) || off(ks, 4))
    return fail(HYTOPK_EINVAL, "w, q_scale and k_scale must be 4-byte aligned");
  return HYTOPK_OK;
}

// Splits of the key range so that the score launch has enough workgroups.
void splits(int64_t nq, int64_t maxctx, int fmt, int& nsplit, int& split_len) {
  const int64_t gq = hk::score_group_queries(fmt);
  const int64_t groups = (nq + gq - 1) / gq;
  int64_t want = (512 + groups - 1) / groups;
  const int64_t most = std::max<int64_t>(1, (maxctx + 4095) / 4096);
  want = std::max<int64_t>(1, std::min(want, most));
  int64_t len = (maxctx + want - 1) / want;
  len = (len + 127) / 128 * 128;  // whole key tiles
  nsplit = (int)((maxctx + len - 1) / len);
  split_len = (int)len;
}

// Backward workspace: u rows of one chunk of queries, then the sort buffers.
constexpr int64_t kBwdChunkBytes = int64_t(1) << 33;

struct BwdLayout {
  int64_t chunk;
  size_t u, k0, v0, k1, v1, hist, qb, kb, total;
};

BwdLayout bwd_layout(const hytopk_problem* p) {
  BwdLayout l{};
  const int64_t kp = hk::bwd_padded_k(p->k);
  const int64_t row = kp * p->d * 4;  // u bytes per query
  l.chunk = std::max<int64_t>(1, std::min<int64_t>(p->n, kBwdChunkBytes / row));
  const int64_t N = l.chunk * p->k;
  size_t off = 0;
  l.u = off; off = align_up(off + (size_t)(l.chunk * kp) * p->d * 4);
  l.k0 = off; off = align_up(off + (size_t)N * 4);
  l.v0 = off; off = align_up(off + (size_t)N * 4);
  l.k1 = off; off = align_up(off + (size_t)N * 4);
  l.v1 = off; off = align_up(off + (size_t)N * 4);
  l.hist = off; off = align_up(off + hk::bwd_sort_hist_count(N) * 4);
  if (p->dtype != HYTOPK_BF16) {  // q and k as bf16 for the gradient products
    l.qb = off; off = align_up(off + (size_t)p->n * p->H * p->d * 2);
    l.kb = off; off = align_up(off + (size_t)p->L * p->d * 2);
  }
  l.total = off;
  return l;
}

hk::ScoreArgs score_args(const hytopk_problem* p, const void* q, const void* qs, const void* k,
                         const void* ks, const float* w) {
  hk::ScoreArgs a{};
  a.q = static_cast<const uint8_t*>(q);
  a.k = static_cast<const uint8_t*>(k);
  a.w = w;
  a.q_scale = qs;
  a.k_scale = ks;
  a.L = (int)p->L;
  a.q_start = (int)p->q_start;
  a.qpos = p->q_pos;
  a.qfirst = p->q_first;
  a.H = p->H;
  // Debug knob (determinism check): HYTOPK_REVERSE_KEY_WALK=1 makes the
  // scoring kernels walk key tiles from last to first; results must not change.
  const char* rev = std::getenv("HYTOPK_REVERSE_KEY_WALK");
  a.reverse = (rev && rev[0] == '1') ? 1 : 0;
  return a;
}

// Upper bound on the key range queries first..last-1 can see.
int64_t ctx_bound(const hytopk_problem* p, int64_t last) {
  return p->q_pos ? p->L : p->q_start + last;
}

// Score `nq` queries (qlist or q_offset..) into rows, then row top-k: split
// over many workgroups per row when the rows are few and `split` scratch is
// given, else one workgroup per row.
int rows_path(const hytopk_problem* p, const hk::ScoreArgs& base, const int* qlist, int q_offset,
              int nq, int64_t maxctx, float* rows, int32_t* out_idx, float* out_score,
              void* split, hipStream_t s, hk::RowGate gate = hk::RowGate{nullptr, 0, 0}) {
  hk::ScoreArgs a = base;
  a.rows = rows;
  a.row_stride = p->L;
  a.qlist = qlist;
  a.q_offset = q_offset;
  a.nq = nq;
  a.gate = gate;
  splits(nq, maxctx, p->dtype, a.nsplit, a.split_len);
  {
    Span sp("score_rows", s);
    HK_HIP(hk::launch_score(a, p->d, p->dtype, s), "score rows launch");
  }
  Span sp("row_topk", s);
  if (split && nq <= hk::kRowSplitMaxRows) {
    hk::RowSelArgs r{};
    r.rows = rows;
    r.row_stride = p->L;
    r.qlist = qlist;
    r.q_offset = q_offset;
    r.nq = nq;
    r.qpos = p->q_pos;
    r.qfirst = p->q_first;
    r.q_start = (int)p->q_start;
    r.topk = p->k;
    r.L = (int)p->L;
    hk::row_select_chunks(nq, maxctx, p->L, r.nchunk, r.chunk_len);
    r.scratch = split;
    r.out_idx = out_idx;
    r.out_score = out_score;
    r.gate = gate;
    HK_HIP(hk::launch_row_select_split(r, s), "split row top-k launch");
  } else {
    HK_HIP(hk::launch_row_topk(rows, p->L, qlist, q_offset, nq, p->q_pos, p->q_first,
                               (int)p->q_start, p->k, (int)p->L, out_idx, out_score, gate, s),
           "row top-k launch");
  }
  return HYTOPK_OK;
}

// Library-owned workspace of hytopk_select_noalloc: one copy per GPU the
// library runs on, held until the process ends.  Host code never passes the
// array's name to a kernel or a copy (on the host it is a stand-in, not a
// device address); it uses the per-device address hipGetSymbolAddress gives.
std::mutex g_scratch_mu;
std::map<int, void*> g_scratch_ptr;  // device ordinal -> device address of `scratch`

// Device address of this device's `scratch`, looked up on the first call on
// each device (with that device current).
int scratch_address(void** out) {
  int dev = 0;
  HK_HIP(hipGetDevice(&dev), "hipGetDevice");
  std::lock_guard<std::mutex> g(g_scratch_mu);
  auto it = g_scratch_ptr.find(dev);
  if (it != g_scratch_ptr.end()) {
    *out = it->second;
    return HYTOPK_OK;
  }
  void* ptr = nullptr;
  HK_HIP(hipGetSymbolAddress(&ptr, HIP_SYMBOL(scratch)), "hipGetSymbolAddress(scratch)");
  if (!ptr || reinterpret_cast<uintptr_t>(ptr) % kAlign)
    return fail(HYTOPK_EHIP, "static scratch has no usable device address");
  g_scratch_ptr[dev] = ptr;
  *out = ptr;
  return HYTOPK_OK;
}

}  // namespace

extern "C" {

const char* hytopk_status_string(int status) {
  switch (status) {
    case HYTOPK_OK: return "ok";
    case HYTOPK_EINVAL: return "invalid argument";
    case HYTOPK_EUNSUPPORTED: return "unsupported problem";
    case HYTOPK_EWORKSPACE: return "bad workspace";
    case HYTOPK_EHIP: return "HIP runtime error";
    default: return "unknown status";
  }
}

const char* hytopk_last_error(void) { return g_err.c_str(); }

int hytopk_trace_enable(int on) {
  Tracer& t = tracer();
  std::lock_guard<std::mutex> g(t.mu);
  const int prev = t.on ? 1 : 0;
  t.on = on != 0;
  if (t.on) t.acc.clear();
  return prev;
}

int hytopk_trace_read(hytopk_trace_entry* out, int max) {
  Tracer& t = tracer();
  std::lock_guard<std::mutex> g(t.mu);
  for (TraceRec& r : t.pending) {
    hipError_t e = hipEventSynchronize(r.b);
    if (e != hipSuccess) return hip_fail(e, "trace event sync");
    float ms = 0.f;
    e = hipEventElapsedTime(&ms, r.a, r.b);
    if (e != hipSuccess) return hip_fail(e, "trace elapsed time");
    auto& slot = t.acc[r.name];
    slot.first += 1;
    slot.second += ms;
    t.pool.push_back(r.a);
    t.pool.push_back(r.b);
  }
  t.pending.clear();
  int i = 0;
  for (const auto& kv : t.acc) {
    if (out && i < max) {
      std::memset(out[i].name, 0, sizeof(out[i].name));
      std::strncpy(out[i].name, kv.first.c_str(), sizeof(out[i].name) - 1);
      out[i].launches = kv.second.first;
      out[i].total_ms = kv.second.second;
    }
    ++i;
  }
  return i;
}

size_t hytopk_select_workspace(const hytopk_problem* p, const hytopk_params* prm) {
  if (check_problem(p) != HYTOPK_OK) return 0;
  Params r = resolve(p, prm);
  if (check_params(p, r) != HYTOPK_OK) return 0;
  return layout(p, r).total;
}

size_t hytopk_baseline_workspace(const hytopk_problem* p) {
  if (check_problem(p) != HYTOPK_OK) return 0;
  return (size_t)p->n * (size_t)p->L * 4;
}

}  // extern "C"

namespace {

// The selection.  status == null: the recovery path is chosen on the host
// after one synchronisation (hytopk_select).  status != null: nothing
// synchronises; recovery passes for up to max_recover failures are enqueued
// with device-side row counts, and the device status words tell whether the
// failures exceeded max_recover (hytopk_select_async).
int select_impl(const hytopk_problem* p, const hytopk_params* prm, const void* q,
                const void* q_scale, const void* k, const void* k_scale, const float* w,
                int32_t* out_idx, float* out_score, void* workspace, size_t workspace_bytes,
                void* stream, hytopk_stats* stats, int32_t* status) {
  int rc = check_problem(p);
  if (rc) return rc;
  Params r = resolve(p, prm);
  if ((rc = check_params(p, r))) return rc;
  if ((rc = check_inputs(p, q, q_scale, k, k_scale, w))) return rc;
  if (!out_idx) return fail(HYTOPK_EINVAL, "out_idx is NULL");
  const Layout l = layout(p, r);
  if ((rc = check_ws(workspace, workspace_bytes, l.total))) return rc;

  hipStream_t s = static_cast<hipStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  float* tau = reinterpret_cast<float*>(ws + l.tau);
  int* cnt = reinterpret_cast<int*>(ws + l.cnt);
  int* failed = reinterpret_cast<int*>(ws + l.failed);
  hk::DevStats* dst = reinterpret_cast<hk::DevStats*>(ws + l.stats);
  uint2* cand = reinterpret_cast<uint2*>(ws + l.cand);
  float* rows = reinterpret_cast<float*>(ws + l.rows);
  void* split = split_bytes(p, l.rows_n) ? static_cast<void*>(ws + l.split) : nullptr;
  const int fmt = p->dtype;
  const int n = (int)p->n;
  const int64_t maxctx = ctx_bound(p, p->n);
  const hk::ScoreArgs base = score_args(p, q, q_scale, k, k_scale, w);

  const bool async = status != nullptr;
  hk::DevStats hs{};
  int path = 0;
  if (r.force_path != HYTOPK_PATH_ROWS_ALL || async) {
    HK_HIP(hk::launch_zero(cnt, n, dst, s), "zero launch");
  }
  if (r.force_path != HYTOPK_PATH_ROWS_ALL) {
    hk::SampleArgs sa{};
    sa.q = base.q; sa.k = base.k; sa.w = w; sa.q_scale = q_scale; sa.k_scale = k_scale;
    sa.tau = tau; sa.L = (int)p->L; sa.q_start = (int)p->q_start; sa.n = n; sa.H = p->H;
    sa.qpos = p->q_pos; sa.qfirst = p->q_first;
    sa.topk = p->k; sa.M = sample_count(p, r); sa.oversample = r.oversample;
    {
      Span sp("sample_tau", s);
      HK_HIP(hk::launch_sample_tau(sa, p->d, fmt, s), "sample/threshold launch");
    }

    hk::ScoreArgs a = base;
    a.tau = tau;
    a.cnt = cnt;
    a.cand = cand;
    a.cap = r.cap;
    a.nq = n;
    splits(n, maxctx, p->dtype, a.nsplit, a.split_len);
    {
      Span sp("score_compact", s);
      HK_HIP(hk::launch_score(a, p->d, fmt, s), "fused score launch");
    }
    {
      Span sp("check", s);
      HK_HIP(hk::launch_check(cnt, n, p->q_pos, p->q_first, (int)p->q_start, (int)p->L, p->k,
                              r.cap, dst, failed, s),
             "check launch");
    }
    if (async) {
      path = 3;
    } else {
      HK_HIP(hipMemcpyAsync(&hs, dst, sizeof(hs), hipMemcpyDeviceToHost, s), "stats copy");
      HK_HIP(hipStreamSynchronize(s), "stream sync");
      path = hs.n_failed > r.max_recover ? 1 : 0;
    }
  } else {
    path = 2;
  }

  if (path == 3) {
    // No synchronisation: the candidate select skips the failed queries by
    // itself, and each recovery pass reads the failure count on the device.
    {
      Span sp("cand_select", s);
      HK_HIP(hk::launch_cand_select(cnt, cand, n, p->q_pos, p->q_first, (int)p->q_start, p->k,
                                    r.cap, (int)p->L, out_idx, out_score, s),
             "candidate select launch");
    }
    const int most = std::min(r.max_recover, n);
    for (int f0 = 0; f0 < most; f0 += l.rows_n) {
      const int nf = std::min(l.rows_n, most - f0);
      rc = rows_path(p, base, failed + f0, 0, nf, maxctx, rows, out_idx, out_score, split, s,
                     hk::RowGate{&dst->n_failed, r.max_recover, f0});
      if (rc) return rc;
    }
  } else if (path == 0) {
    {
      Span sp("cand_select", s);
      HK_HIP(hk::launch_cand_select(cnt, cand, n, p->q_pos, p->q_first, (int)p->q_start, p->k,
                                    r.cap, (int)p->L, out_idx, out_score, s),
             "candidate select launch");
    }
    // Recovery: full score rows for the flagged queries only, then row top-k.
    for (int f0 = 0; f0 < hs.n_failed; f0 += l.rows_n) {
      const int nf = std::min(l.rows_n, hs.n_failed - f0);
      rc = rows_path(p, base, failed + f0, 0, nf, maxctx, rows, out_idx, out_score, split, s);
      if (rc) return rc;
    }
  } else {
    // Full rescore: every query through the row path, in chunks of rows_n.
    for (int c0 = 0; c0 < n; c0 += l.rows_n) {
      const int nc = std::min(l.rows_n, n - c0);
      rc = rows_path(p, base, nullptr, c0, nc, ctx_bound(p, c0 + nc), rows, out_idx, out_score,
                     split, s);
      if (rc) return rc;
    }
  }
  if (stats && stats->failed_queries && stats->failed_capacity > 0 && hs.n_failed > 0) {
    const int m = std::min(hs.n_failed, stats->failed_capacity);
    HK_HIP(hipMemcpyAsync(stats->failed_queries, failed, (size_t)m * sizeof(int32_t),
                          hipMemcpyDeviceToHost, s),
           "failed list copy");
    HK_HIP(hipStreamSynchronize(s), "stream sync");
    std::sort(stats->failed_queries, stats->failed_queries + m);
  }
  if (stats) {
    stats->n_overflow = hs.n_overflow;
    stats->n_underk = hs.n_underk;
    stats->n_failed = hs.n_failed;
    stats->full_rescore = path != 0;
    stats->cand_total = (int64_t)hs.cand_total;
    stats->cand_max = hs.cand_max;
    stats->path = path;
  }
  if (async) HK_HIP(hk::launch_async_status(dst, r.max_recover, status, s), "status launch");
  return HYTOPK_OK;
}

}  // namespace

extern "C" {

int hytopk_select(const hytopk_problem* p, const hytopk_params* prm, const void* q,
                  const void* q_scale, const void* k, const void* k_scale, const float* w,
                  int32_t* out_idx, float* out_score, void* workspace, size_t workspace_bytes,
                  void* stream, hytopk_stats* stats) {
  g_err.clear();
  return select_impl(p, prm, q, q_scale, k, k_scale, w, out_idx, out_score, workspace,
                     workspace_bytes, stream, stats, nullptr);
}

int hytopk_select_async(const hytopk_problem* p, const hytopk_params* prm, const void* q,
                        const void* q_scale, const void* k, const void* k_scale, const float* w,
                        int32_t* out_idx, float* out_score, void* workspace,
                        size_t workspace_bytes, void* stream, int32_t* status) {
  g_err.clear();
  if (!status) return fail(HYTOPK_EINVAL, "status is NULL");
  if (reinterpret_cast<uintptr_t>(status) % 4) return fail(HYTOPK_EINVAL, "status must be 4-byte aligned");
  return select_impl(p, prm, q, q_scale, k, k_scale, w, out_idx, out_score, workspace,
                     workspace_bytes, stream, nullptr, status);
}

int hytopk_select_noalloc(const hytopk_problem* p, const hytopk_params* prm, const void* q,
                          const void* q_scale, const void* k, const void* k_scale, const float* w,
                          int32_t* out_idx, float* out_score, void* stream, hytopk_stats* stats) {
  g_err.clear();
  int rc = check_problem(p);
  if (rc) return rc;
  Params r = resolve(p, prm);
  if ((rc = check_params(p, r))) return rc;
  const size_t need = layout(p, r).total;
  if (need > kNoAllocBytes) {
    char msg[160];
    std::snprintf(msg, sizeof msg,
                  "problem needs %zu bytes of workspace, more than the %zu-byte static scratch "
                  "(use hytopk_select with a workspace, or a smaller rows_chunk / cap)",
                  need, kNoAllocBytes);
    return fail(HYTOPK_EWORKSPACE, msg);
  }
  void* ws = nullptr;
  if ((rc = scratch_address(&ws))) return rc;
  return hytopk_select(p, prm, q, q_scale, k, k_scale, w, out_idx, out_score, ws, kNoAllocBytes,
                       stream, stats);
}

int hytopk_replay(const hytopk_problem* p, const void* q, const void* q_scale, const void* k,
                  const void* k_scale, const float* w, const int32_t* idx, float* out_score,
                  void* stream) {
  g_err.clear();
  int rc = check_problem(p);
  if (rc) return rc;
  if ((rc = check_inputs(p, q, q_scale, k, k_scale, w))) return rc;
  if (!idx || !out_score) return fail(HYTOPK_EINVAL, "idx and out_score must be non-NULL");
  hk::ReplayArgs a{};
  a.q = static_cast<const uint8_t*>(q);
  a.k = static_cast<const uint8_t*>(k);
  a.w = w;
  a.q_scale = q_scale;
  a.k_scale = k_scale;
  a.idx = idx;
  a.out = out_score;
  a.L = (int)p->L;
  a.n = (int)p->n;
  a.H = p->H;
  a.topk = p->k;
  hipStream_t s = static_cast<hipStream_t>(stream);
  Span sp("replay", s);
  HK_HIP(hk::launch_replay(a, p->d, p->dtype, s), "replay launch");
  return HYTOPK_OK;
}

int hytopk_baseline_select(const hytopk_problem* p, const void* q, const void* q_scale,
                           const void* k, const void* k_scale, const float* w, int32_t* out_idx,
                           float* out_score, void* workspace, size_t workspace_bytes,
                           void* stream) {
  g_err.clear();
  int rc = check_problem(p);
  if (rc) return rc;
  if ((rc = check_inputs(p, q, q_scale, k, k_scale, w))) return rc;
  if (!out_idx) return fail(HYTOPK_EINVAL, "out_idx is NULL");
  if ((rc = check_ws(workspace, workspace_bytes, hytopk_baseline_workspace(p)))) return rc;
  const hk::ScoreArgs base = score_args(p, q, q_scale, k, k_scale, w);
  return rows_path(p, base, nullptr, 0, (int)p->n, ctx_bound(p, p->n),
                   static_cast<float*>(workspace), out_idx, out_score, nullptr,
                   static_cast<hipStream_t>(stream));
}


size_t hytopk_backward_workspace(const hytopk_problem* p) {
  if (check_problem(p) != HYTOPK_OK) return 0;
  return bwd_layout(p).total;
}

int hytopk_backward(const hytopk_problem* p, const void* q, const void* q_scale, const void* k,
                    const void* k_scale, const float* w, const int32_t* idx,
                    const float* d_score, float* dq, float* dw, float* dk, void* workspace,
                    size_t workspace_bytes, void* stream) {
  g_err.clear();
  int rc = check_problem(p);
  if (rc) return rc;
  if ((rc = check_inputs(p, q, q_scale, k, k_scale, w))) return rc;
  if (!idx || !d_score) return fail(HYTOPK_EINVAL, "idx and d_score must be non-NULL");
  const BwdLayout l = bwd_layout(p);
  const bool scaled = p->dtype != HYTOPK_BF16;
  if ((dk || scaled) && (rc = check_ws(workspace, workspace_bytes, l.total))) return rc;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int K = p->k, D = p->d;
  char* ws = static_cast<char*>(workspace);
  // Scaled formats: q and k as bf16 (decoded MX values, or FP8 codes whose
  // per-token scales the query kernel applies).
  const uint16_t* qb = static_cast<const uint16_t*>(q);
  const uint16_t* kb = static_cast<const uint16_t*>(k);
  const bool tok = p->dtype == HYTOPK_FP8_E4M3;
  if (scaled) {
    Span sp("bwd_query", s);
    uint16_t* qd = reinterpret_cast<uint16_t*>(ws + l.qb);
    uint16_t* kd = reinterpret_cast<uint16_t*>(ws + l.kb);
    HK_HIP(hk::launch_bwd_dequant(q, tok ? nullptr : q_scale, p->n * p->H, D, p->dtype, qd, s),
           "backward q decode launch");
    HK_HIP(hk::launch_bwd_dequant(k, tok ? nullptr : k_scale, p->L, D, p->dtype, kd, s),
           "backward k decode launch");
    qb = qd;
    kb = kd;
  }
  float* u = dk ? reinterpret_cast<float*>(ws + l.u) : nullptr;
  if (dk) {
    Span sp("bwd_dk", s);
    HK_HIP(hk::launch_fill_zero(dk, p->L * (int64_t)D, s), "dk clear");
  }
  for (int64_t q0 = 0; q0 < p->n; q0 += l.chunk) {
    const int nq = (int)std::min<int64_t>(l.chunk, p->n - q0);
    const uint32_t *sorted_keys = nullptr, *sorted_rows = nullptr;
    if (dk) {
      hk::DkArgs b{};
      b.idx = idx + q0 * K;
      b.L = (int)p->L;
      b.N = nq * K;
      b.topk = K;
      b.k0 = reinterpret_cast<uint32_t*>(ws + l.k0);
      b.v0 = reinterpret_cast<uint32_t*>(ws + l.v0);
      b.k1 = reinterpret_cast<uint32_t*>(ws + l.k1);
      b.v1 = reinterpret_cast<uint32_t*>(ws + l.v1);
      b.hist = reinterpret_cast<uint32_t*>(ws + l.hist);
      Span sp("bwd_dk", s);
      HK_HIP(hk::launch_bwd_sort(b, &sorted_keys, &sorted_rows, s), "backward key sort launch");
    }
    hk::BwdArgs a{};
    a.q = qb;
    a.k = kb;
    a.w = w;
    a.q_scale = tok ? static_cast<const float*>(q_scale) : nullptr;
    a.k_scale = tok ? static_cast<const float*>(k_scale) : nullptr;
    a.idx = idx;
    a.dsc = d_score;
    a.dq = dq;
    a.dw = dw;
    a.u = u;
    a.L = (int)p->L;
    a.H = p->H;
    a.topk = K;
    a.q0 = (int)q0;
    a.nq = nq;
    {
      Span sp("bwd_query", s);
      HK_HIP(hk::launch_bwd_query(a, D, s), "backward query launch");
    }
    if (dk) {
      Span sp("bwd_dk", s);
      HK_HIP(hk::launch_bwd_segments(sorted_keys, sorted_rows, nq * K, (int)p->L, u, dk, q0 > 0,
                                     D, s),
             "backward dk launch");
    }
  }
  return HYTOPK_OK;
}

}  // extern "C"

// ------------------------------------- rotary, cache, attention mass, loss

namespace {

// Runs an entry point's body; what it throws (host memory running out) comes
// back as a status.
template <typename F>
int guarded(F body) noexcept {
  try {
    g_err.clear();
    return body();
  } catch (...) {
    return HYTOPK_EHIP;
  }
}

constexpr int64_t kMaxRows = int64_t(1) << 31;
constexpr int kMaxRotary = 1024;
constexpr int kMaxRowElems = 8192;
constexpr int kMaxAxes = 16;

bool misaligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

int rows_elem(const hytopk_rows* r) { return r->dtype == HYTOPK_ROWS_BF16 ? 2 : 4; }

int check_rows(const hytopk_rows* r, int64_t n, int32_t heads, int32_t d) {
  if (!r) return fail(HYTOPK_EINVAL, "rows are NULL");
  if (r->dtype != HYTOPK_ROWS_BF16 && r->dtype != HYTOPK_ROWS_FP32)
    return fail(HYTOPK_EINVAL, "unknown rows dtype");
  if (r->token_stride < 0 || r->head_stride < 0) return fail(HYTOPK_EINVAL, "strides must be >= 0");
  if (n == 0) return HYTOPK_OK;
  if (!r->data) return fail(HYTOPK_EINVAL, "rows data is NULL");
  if (misaligned(r->data, (uintptr_t)rows_elem(r)))
    return fail(HYTOPK_EINVAL, "rows must be aligned to their element");
  const __int128 span = (__int128)(n - 1) * r->token_stride + (__int128)(heads - 1) * r->head_stride + d;
  if (span > ((__int128)1 << 60)) return fail(HYTOPK_EINVAL, "rows span more memory than exists");
  return HYTOPK_OK;
}

int check_tokens(int64_t n, int32_t heads, int32_t d) {
  if (n < 0 || heads <= 0 || d <= 0) return fail(HYTOPK_EINVAL, "n must be >= 0 and heads, d > 0");
  if (n >= kMaxRows) return fail(HYTOPK_EUNSUPPORTED, "n >= 2^31");
  if ((int64_t)heads * d >= kMaxRows) return fail(HYTOPK_EUNSUPPORTED, "heads * d >= 2^31");
  return HYTOPK_OK;
}

// Whether no two rows share an element: one axis' rows lie apart and the other axis steps over
// all of them.
bool rows_apart(const hytopk_rows* r, int64_t n, int32_t heads, int32_t d) {
  const __int128 t = r->token_stride, h = r->head_stride;
  if (heads == 1) return n == 1 || t >= d;
  if (n == 1) return h >= d;
  return (h >= d && t >= (heads - 1) * h + d) || (t >= d && h >= (n - 1) * t + d);
}

struct Extent {
  uintptr_t lo, hi;
};

Extent extent(const hytopk_rows* r, int64_t n, int32_t heads, int32_t d) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(r->data);
  const int64_t span = (n - 1) * r->token_stride + (heads - 1) * r->head_stride + d;
  return Extent{lo, lo + (uintptr_t)(span * rows_elem(r))};
}

Extent extent(const void* p, int64_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return Extent{lo, lo + (uintptr_t)bytes};
}

bool overlap(Extent a, Extent b) { return a.lo < b.hi && b.lo < a.hi; }
// The bytes that rows are stored in along one axis: `count` pieces `stride` apart.
struct Axis {
  int64_t count, stride;
};

// Whether pieces of `lx` and `ly` bytes that repeat along the same axes, outermost first, meet, where y's
// begin `off` bytes behind x's.  Each axis steps over all of what lies inside it, so off modulo its stride leaves
// two neighbours of an x piece.
bool pieces_meet(const Axis* axis, int axes, int64_t lx, int64_t ly, int64_t off) {
  int64_t steps = 0;
  for (int i = 0; i < axes; ++i) steps += (axis[i].count - 1) * axis[i].stride;
  if (off >= steps + lx || off + steps + ly <= 0) return false;
  if (axes == 0) return true;
  const int64_t s = axis->stride, r = ((off % s) + s) % s;
  return pieces_meet(axis + 1, axes - 1, lx, ly, r) || pieces_meet(axis + 1, axes - 1, lx, ly, r - s);
}

// Whether rows x and y share memory.  Rows of one geometry (slices of one buffer) may lie between each other's;
// others are taken as whole extents.
bool rows_meet(const hytopk_rows* x, const hytopk_rows* y, int64_t n, int32_t heads, int32_t d) {
  const Extent ex = extent(x, n, heads, d), ey = extent(y, n, heads, d);
  if (!overlap(ex, ey)) return false;
  const int64_t bx = rows_elem(x), by = rows_elem(y);
  Axis axis[2];
  int axes = 0;
  if (n > 1) axis[axes++] = Axis{n, y->token_stride * by};
  if (heads > 1) axis[axes++] = Axis{heads, y->head_stride * by};
  if ((n > 1 && x->token_stride * bx != y->token_stride * by) ||
      (heads > 1 && x->head_stride * bx != y->head_stride * by))
    return true;
  if (axes == 2 && axis[0].stride < axis[1].stride) std::swap(axis[0], axis[1]);
  // an axis steps over what lies inside it
  int64_t span = std::max(bx, by) * d;
  for (int i = axes - 1; i >= 0; --i) {
    if (axis[i].stride < span) return true;
    span += (axis[i].count - 1) * axis[i].stride;
  }
  return pieces_meet(axis, axes, bx * d, by * d, (int64_t)(ey.lo - ex.lo));
}

// Whether `bytes` bytes at p (NULL: none) lie in m.
bool touches(Extent m, const void* p, int64_t bytes) { return p && overlap(m, extent(p, bytes)); }

int check_plan(const hytopk_rotary_plan* p, int32_t d) {
  if (!p) return fail(HYTOPK_EINVAL, "rotary plan is NULL");
  if (p->dim <= 0 || p->dim % 2) return fail(HYTOPK_EINVAL, "the rotary dim must be even and > 0");
  if (p->first < 0 || (int64_t)p->first + p->dim > d)
    return fail(HYTOPK_EINVAL, "the rotated part lies outside the head");
  if (p->dim > kMaxRotary) return fail(HYTOPK_EUNSUPPORTED, "rotary dim > 1024");
  if (p->layout != HYTOPK_ROTARY_HALF && p->layout != HYTOPK_ROTARY_INTERLEAVED)
    return fail(HYTOPK_EINVAL, "unknown rotary layout");
  if (!p->freq) return fail(HYTOPK_EINVAL, "rotary freq is NULL");
  if (misaligned(p->freq, 8)) return fail(HYTOPK_EINVAL, "rotary freq must be 8-byte aligned");
  if (!std::isfinite((float)p->gain)) return fail(HYTOPK_EINVAL, "the rotary gain must be finite in fp32");
  if (p->axes < 0) return fail(HYTOPK_EINVAL, "the rotary axes must be >= 0");
  if (p->axes > kMaxAxes) return fail(HYTOPK_EUNSUPPORTED, "rotary axes > 16");
  return HYTOPK_OK;
}

int check_positions(int64_t n, const int32_t* q_pos, int64_t q_start) {
  if (q_pos) {
    if (misaligned(q_pos, 4)) return fail(HYTOPK_EINVAL, "q_pos must be 4-byte aligned");
  } else if (q_start < 0 || q_start > kMaxRows - n) {
    return fail(HYTOPK_EINVAL, "positions q_start .. q_start + n - 1 must lie in [0, 2^31)");
  }
  return HYTOPK_OK;
}

// Bytes of a plan's frequencies (and the axes behind them), and of the positions of n tokens.
int64_t plan_bytes(const hytopk_rotary_plan* p) { return (p->axes > 1 ? 6 : 4) * (int64_t)p->dim; }
int64_t position_bytes(const hytopk_rotary_plan* p, int64_t n) { return 4 * n * std::max(p->axes, 1); }

hk::RotArgs rot_args(const hytopk_rotary_plan* p, const int32_t* q_pos, int64_t q_start, bool backward) {
  hk::RotArgs r{};
  if (!p) return r;
  r.freq = p->freq;
  r.pos = q_pos;
  if (q_pos) r.axes = std::max(p->axes, 1);
  else r.pos0 = (int)q_start;  // below 2^31
  r.gain = (float)p->gain;
  r.turn = backward ? -r.gain : r.gain;
  r.dim = p->dim;
  return r;
}

// The cache's codes and (none for bf16) scales.
Extent cache_codes(const hytopk_cache* c) {
  const int64_t e = c->L * c->heads * c->d;
  return extent(c->codes, c->dtype == HYTOPK_BF16 ? 2 * e : (c->dtype == HYTOPK_MXFP4_E2M1 ? e / 2 : e));
}
Extent cache_scale(const hytopk_cache* c) {
  if (c->dtype == HYTOPK_BF16) return Extent{0, 0};
  return extent(c->scale, c->dtype == HYTOPK_FP8_E4M3 ? 4 * c->L : c->L * c->heads * c->d / 32);
}
// Whether memory lies in the cache's codes or scales.
bool in_cache(const hytopk_cache* c, Extent m) { return overlap(m, cache_codes(c)) || overlap(m, cache_scale(c)); }
bool in_cache(const hytopk_cache* c, const void* p, int64_t bytes) { return p && in_cache(c, extent(p, bytes)); }

// The geometry alone (what the workspace query knows).
int check_cache_shape(const hytopk_cache* c) {
  if (!c) return fail(HYTOPK_EINVAL, "cache is NULL");
  if (c->L <= 0 || c->heads <= 0 || c->d <= 0) return fail(HYTOPK_EINVAL, "L, heads and d must be > 0");
  if (c->dtype < HYTOPK_BF16 || c->dtype > HYTOPK_MXFP4_E2M1) return fail(HYTOPK_EINVAL, "unknown dtype");
  if (c->L >= kMaxRows) return fail(HYTOPK_EUNSUPPORTED, "L >= 2^31");
  if (c->d % 32) return fail(HYTOPK_EUNSUPPORTED, "cache rows need d in multiples of 32");
  if ((int64_t)c->heads * c->d > kMaxRowElems) return fail(HYTOPK_EUNSUPPORTED, "heads * d > 8192");
  return HYTOPK_OK;
}

int check_cache(const hytopk_cache* c, int64_t n, const int32_t* slots, int64_t start) {
  int rc = check_cache_shape(c);
  if (rc) return rc;
  if (n < 0) return fail(HYTOPK_EINVAL, "n must be >= 0");
  if (n >= kMaxRows) return fail(HYTOPK_EUNSUPPORTED, "n >= 2^31");
  if (!c->codes) return fail(HYTOPK_EINVAL, "cache codes are NULL");
  if (misaligned(c->codes, 16)) return fail(HYTOPK_EINVAL, "cache codes must be 16-byte aligned");
  if (c->dtype != HYTOPK_BF16) {
    if (!c->scale) return fail(HYTOPK_EINVAL, "fp8 and MX caches need scales");
    if (misaligned(c->scale, 4)) return fail(HYTOPK_EINVAL, "cache scales must be 4-byte aligned");
  }
  if (slots) {
    if (misaligned(slots, 4)) return fail(HYTOPK_EINVAL, "slots must be 4-byte aligned");
  } else if (start < 0 || start > c->L - n) {
    return fail(HYTOPK_EINVAL, "rows start .. start + n - 1 lie outside the cache");
  }
  return HYTOPK_OK;
}

bool wants_claim(int64_t n, bool by_slot) { return by_slot && n > hk::kClaimRows; }

int check_norm(const hytopk_norm* p) {
  if (!p) return fail(HYTOPK_EINVAL, "norm is NULL");
  if (p->dtype != HYTOPK_ROWS_BF16 && p->dtype != HYTOPK_ROWS_FP32)
    return fail(HYTOPK_EINVAL, "unknown dtype of the norm's parameters");
  const uintptr_t e = p->dtype == HYTOPK_ROWS_BF16 ? 2 : 4;
  if (misaligned(p->weight, e) || misaligned(p->bias, e))
    return fail(HYTOPK_EINVAL, "weight and bias must be aligned to their element");
  return HYTOPK_OK;
}

int check_norm_rows(int64_t n, int32_t heads, int32_t d) {
  const int rc = check_tokens(n, heads, d);
  if (rc) return rc;
  if (d > hk::kMaxNorm) return fail(HYTOPK_EUNSUPPORTED, "rows of a norm have d <= 8192");
  if (n * heads >= kMaxRows) return fail(HYTOPK_EUNSUPPORTED, "n * heads >= 2^31");
  return HYTOPK_OK;
}

int check_stats(const float* stats) {
  if (misaligned(stats, 8)) return fail(HYTOPK_EINVAL, "stats must be 8-byte aligned");
  return HYTOPK_OK;
}

// A norm's checkpoint: one cache row for each of its rows.
int check_checkpoint(const hytopk_cache* c, int64_t rows, int32_t d) {
  const int rc = check_cache(c, rows, nullptr, 0);
  if (rc) return rc;
  if (c->dtype != HYTOPK_FP8_E4M3 && c->dtype != HYTOPK_MXFP8_E4M3)
    return fail(HYTOPK_EUNSUPPORTED, "checkpoints are FP8 or MXFP8");
  if (c->heads != 1 || c->d != d) return fail(HYTOPK_EINVAL, "a checkpoint's rows are the norm's: heads 1, the same d");
  return HYTOPK_OK;
}

// The bytes of a norm's parameters.
Extent parameter(const hytopk_norm* p, const void* v, int32_t d) {
  return v ? extent(v, (int64_t)d * (p->dtype == HYTOPK_ROWS_BF16 ? 2 : 4)) : Extent{0, 0};
}

// Memory that a call reads or writes, empty where it does not exist.
Extent memory(const void* p, int64_t bytes) { return p ? extent(p, bytes) : Extent{0, 0}; }
Extent memory(const hytopk_rows* r, int64_t n, int32_t heads, int32_t d) { return r ? extent(r, n, heads, d) : Extent{0, 0}; }
bool empty(Extent e) { return e.lo == e.hi; }

// Whether any of `written` overlaps another of them or any of `read`.
template <size_t W, size_t R>
bool written_meets(const Extent (&written)[W], const Extent (&read)[R]) {
  for (size_t i = 0; i < W; ++i) {
    if (empty(written[i])) continue;
    for (size_t j = 0; j < W; ++j)
      if (j != i && !empty(written[j]) && overlap(written[i], written[j])) return true;
    for (size_t j = 0; j < R; ++j)
      if (!empty(read[j]) && overlap(written[i], read[j])) return true;
  }
  return false;
}

bool same_rows(const hytopk_rows* x, const hytopk_rows* y, int64_t n, int32_t heads) {
  return x->data == y->data && x->dtype == y->dtype && (n == 1 || x->token_stride == y->token_stride) &&
         (heads == 1 || x->head_stride == y->head_stride);
}

// The softmax's scale in base 2.
float log2_scale(const hytopk_attention* p) { return (float)((double)p->softmax_scale * 1.4426950408889634074); }

int check_attention(const hytopk_attention* p) {
  if (!p) return fail(HYTOPK_EINVAL, "attention is NULL");
  if (p->L <= 0 || p->n < 0) return fail(HYTOPK_EINVAL, "L must be > 0 and n >= 0");
  if (p->heads <= 0 || p->key_heads <= 0 || p->heads % p->key_heads)
    return fail(HYTOPK_EINVAL, "key_heads must divide heads");
  if (p->k <= 0) return fail(HYTOPK_EINVAL, "k must be > 0");
  if (!std::isfinite(log2_scale(p))) return fail(HYTOPK_EINVAL, "softmax_scale must be finite, in base 2 too");
  if (p->k > kMaxK) return fail(HYTOPK_EUNSUPPORTED, "k > 2048");
  if (p->L >= kMaxRows) return fail(HYTOPK_EUNSUPPORTED, "L >= 2^31");
  // a launch holds fewer than 2^32 threads along the queries
  if (p->n >= hk::mass_most_queries(p->d)) return fail(HYTOPK_EUNSUPPORTED, "n >= 2^24, or 2^23 with d > 256");
  if (!hk::mass_supports(p->d)) return fail(HYTOPK_EUNSUPPORTED, "d must be 64, 96, 128, 192, 256, 512 or 576");
  if (p->heads > 1024) return fail(HYTOPK_EUNSUPPORTED, "heads > 1024");
  return HYTOPK_OK;
}

}  // namespace

extern "C" {

int hytopk_rotary_frequencies(int32_t dim, double base, int32_t scaling, double factor,
                              int64_t original, double* freq, double* gain) {
  return guarded([&]() -> int {
    if (!freq || !gain) return fail(HYTOPK_EINVAL, "freq and gain must be non-NULL");
    if (dim <= 0 || dim % 2) return fail(HYTOPK_EINVAL, "the rotary dim must be even and > 0");
    if (dim > kMaxRotary) return fail(HYTOPK_EUNSUPPORTED, "rotary dim > 1024");
    if (!(base > 1.0) || !std::isfinite(base)) return fail(HYTOPK_EINVAL, "base must be finite and > 1");
    if (scaling < HYTOPK_SCALING_NONE || scaling > HYTOPK_SCALING_YARN)
      return fail(HYTOPK_EINVAL, "unknown rotary scaling");
    if (scaling != HYTOPK_SCALING_NONE && (!(factor >= 1.0) || !std::isfinite(factor)))
      return fail(HYTOPK_EINVAL, "factor must be finite and >= 1");
    if (scaling == HYTOPK_SCALING_YARN && original <= 0)
      return fail(HYTOPK_EINVAL, "yarn needs the original context length");
    double b = base;
    // base^(-(dim - 2)/dim) divided by factor is the slowest frequency of the raised base
    if (scaling == HYTOPK_SCALING_NTK) b *= std::pow(factor, (double)dim / std::max(dim - 2, 1));
    double lo = 0.0, width = 1.0;
    bool slow = false;  // every pair turns once or less
    if (scaling == HYTOPK_SCALING_YARN) {
      // the pair that makes r turns in the original context
      auto pair = [&](double r) {
        return dim * std::log((double)original / (r * 2.0 * M_PI)) / (2.0 * std::log(base));
      };
      lo = std::max(std::floor(pair(32.0)), 0.0);
      const double hi = std::min(std::ceil(pair(1.0)), (double)(dim - 1));
      width = std::max(hi - lo, 1e-3);
      slow = pair(1.0) <= 0.0;
    }
    for (int i = 0; i < dim / 2; ++i) {
      const double f = std::pow(b, -2.0 * i / dim);
      if (scaling == HYTOPK_SCALING_LINEAR) {
        freq[i] = f / factor;
      } else if (scaling == HYTOPK_SCALING_YARN) {
        const double r = slow ? 1.0 : std::min(std::max((i - lo) / width, 0.0), 1.0);
        freq[i] = f * (1.0 - r) + f / factor * r;
      } else {
        freq[i] = f;
      }
    }
    *gain = scaling == HYTOPK_SCALING_YARN ? 0.1 * std::log(factor) + 1.0 : 1.0;
    return HYTOPK_OK;
  });
}

int hytopk_rotary(const hytopk_rotary_plan* plan, int64_t n, int32_t heads, int32_t d,
                  const hytopk_rows* x, const hytopk_rows* y, const int32_t* q_pos,
                  int64_t q_start, int32_t backward, void* stream) {
  return guarded([&]() -> int {
    int rc = check_tokens(n, heads, d);
    if (rc) return rc;
    if ((rc = check_plan(plan, d))) return rc;
    if ((rc = check_rows(x, n, heads, d)) || (rc = check_rows(y, n, heads, d))) return rc;
    if ((rc = check_positions(n, q_pos, q_start))) return rc;
    if (n == 0) return HYTOPK_OK;
    if (!rows_apart(y, n, heads, d)) return fail(HYTOPK_EINVAL, "rows of y overlap each other");
    if (!same_rows(x, y, n, heads) && rows_meet(x, y, n, heads, d))
      return fail(HYTOPK_EINVAL, "x and y overlap (y may be x itself)");
    const Extent out = extent(y, n, heads, d);
    if (touches(out, q_pos, position_bytes(plan, n)) || touches(out, plan->freq, plan_bytes(plan)))
      return fail(HYTOPK_EINVAL, "y overlaps the positions or the plan");
    hk::RotaryArgs a{};
    a.x = x->data;
    a.y = y->data;
    a.xts = x->token_stride; a.xhs = x->head_stride;
    a.yts = y->token_stride; a.yhs = y->head_stride;
    a.n = (int)n;
    a.heads = heads;
    a.d = d;
    a.first = plan->first;
    a.rot = rot_args(plan, q_pos, q_start, backward != 0);
    hipStream_t s = static_cast<hipStream_t>(stream);
    Span sp("rotary", s);
    HK_HIP(hk::launch_rotary(a, plan->layout, x->dtype, y->dtype, s), "rotary launch");
    return HYTOPK_OK;
  });
}

size_t hytopk_cache_write_workspace(const hytopk_cache* c, int64_t n, int32_t by_slot) {
  size_t need = 0;
  guarded([&]() -> int {
    const int rc = check_cache_shape(c);
    if (rc == HYTOPK_OK && wants_claim(n, by_slot != 0)) need = align_up((size_t)c->L * sizeof(int32_t));
    return rc;
  });
  return need;
}

int hytopk_cache_write(const hytopk_cache* c, int64_t n, const hytopk_rows* x,
                       const int32_t* slots, int64_t start, const hytopk_rotary_plan* plan,
                       const int32_t* q_pos, int64_t q_start, void* workspace,
                       size_t workspace_bytes, void* stream) {
  return guarded([&]() -> int {
    int rc = check_cache(c, n, slots, start);
    if (rc) return rc;
    if ((rc = check_rows(x, n, c->heads, c->d))) return rc;
    if (plan && ((rc = check_plan(plan, c->d)) || (rc = check_positions(n, q_pos, q_start)))) return rc;
    if (n == 0) return HYTOPK_OK;
    if (in_cache(c, extent(x, n, c->heads, c->d)))
      return fail(HYTOPK_EINVAL, "x overlaps the cache");
    const bool claim = wants_claim(n, slots != nullptr);
    if (claim && (rc = check_ws(workspace, workspace_bytes, hytopk_cache_write_workspace(c, n, 1)))) return rc;
    if (in_cache(c, slots, 4 * n) || (claim && in_cache(c, workspace, 4 * c->L)) ||
        (plan && (in_cache(c, q_pos, position_bytes(plan, n)) || in_cache(c, plan->freq, plan_bytes(plan)))))
      return fail(HYTOPK_EINVAL, "the slots, the positions, the plan or the workspace overlap the cache");
    if (claim) {  // cleared and written while the others are read
      const Extent w = extent(workspace, 4 * c->L);
      if (touches(w, slots, 4 * n) || overlap(w, extent(x, n, c->heads, c->d)) ||
          (plan && (touches(w, q_pos, position_bytes(plan, n)) || touches(w, plan->freq, plan_bytes(plan)))))
        return fail(HYTOPK_EINVAL, "the workspace overlaps the rows, the slots, the positions or the plan");
    }
    if (overlap(cache_codes(c), cache_scale(c))) return fail(HYTOPK_EINVAL, "the cache's codes and scales overlap");
    hk::CacheWriteArgs a{};
    a.x = x->data;
    a.ts = x->token_stride;
    a.hs = x->head_stride;
    a.n = (int)n;
    a.first = plan ? plan->first : 0;
    a.rot = rot_args(plan, q_pos, q_start, false);
    a.codes = static_cast<uint8_t*>(c->codes);
    a.scale = c->scale;
    a.L = (int)c->L;
    a.slots = slots;
    a.start = (int)start;
    a.claim = claim ? static_cast<int*>(workspace) : nullptr;
    hipStream_t s = static_cast<hipStream_t>(stream);
    Span sp("cache_write", s);
    HK_HIP(hk::launch_cache_write(a, c->heads, c->d, plan ? plan->layout : 0, x->dtype, c->dtype, s), "cache write launch");
    return HYTOPK_OK;
  });
}

int hytopk_cache_read(const hytopk_cache* c, int64_t n, const int32_t* slots, int64_t start,
                      void* out, int32_t out_dtype, void* stream) {
  return guarded([&]() -> int {
    int rc = check_cache(c, n, slots, start);
    if (rc) return rc;
    if (out_dtype != HYTOPK_ROWS_BF16 && out_dtype != HYTOPK_ROWS_FP32)
      return fail(HYTOPK_EINVAL, "unknown rows dtype");
    if (n == 0) return HYTOPK_OK;
    if (!out) return fail(HYTOPK_EINVAL, "out is NULL");
    if (misaligned(out, 16)) return fail(HYTOPK_EINVAL, "out must be 16-byte aligned");
    const int64_t bytes = n * c->heads * c->d * (out_dtype == HYTOPK_ROWS_BF16 ? 2 : 4);
    if (in_cache(c, extent(out, bytes)))
      return fail(HYTOPK_EINVAL, "out overlaps the cache");
    if (touches(extent(out, bytes), slots, 4 * n)) return fail(HYTOPK_EINVAL, "out overlaps the slots");
    hk::CacheReadArgs a{};
    a.codes = static_cast<const uint8_t*>(c->codes);
    a.scale = c->scale;
    a.L = (int)c->L;
    a.slots = slots;
    a.start = (int)start;
    a.n = (int)n;
    a.row = c->heads * c->d;
    a.out = out;
    hipStream_t s = static_cast<hipStream_t>(stream);
    Span sp("cache_read", s);
    HK_HIP(hk::launch_cache_read(a, out_dtype, c->dtype, s), "cache read launch");
    return HYTOPK_OK;
  });
}

int hytopk_layer_norm(const hytopk_norm* norm, int64_t n, int32_t heads, int32_t d, const hytopk_rows* x,
                      const hytopk_rows* y, float* stats, const hytopk_cache* save, void* stream) {
  return guarded([&]() -> int {
    int rc = check_norm_rows(n, heads, d);
    if (rc) return rc;
    if ((rc = check_norm(norm))) return rc;
    if (!(norm->eps >= 0.0f) || !std::isfinite(norm->eps)) return fail(HYTOPK_EINVAL, "eps must be finite and >= 0");
    if ((rc = check_rows(x, n, heads, d)) || (rc = check_rows(y, n, heads, d))) return rc;
    if ((rc = check_stats(stats))) return rc;
    const int64_t rows = n * heads;
    if (save && n > 0) {
      if ((rc = check_checkpoint(save, rows, d))) return rc;
      if (!stats) return fail(HYTOPK_EINVAL, "a checkpoint needs stats");
    }
    if (n == 0) return HYTOPK_OK;
    if (!rows_apart(y, n, heads, d)) return fail(HYTOPK_EINVAL, "rows of y overlap each other");
    if (!same_rows(x, y, n, heads) && rows_meet(x, y, n, heads, d))
      return fail(HYTOPK_EINVAL, "x and y overlap (y may be x itself)");
    const Extent w = parameter(norm, norm->weight, d), b = parameter(norm, norm->bias, d);
    const Extent codes = save ? cache_codes(save) : Extent{0, 0}, scale = save ? cache_scale(save) : Extent{0, 0};
    const Extent st = memory(stats, 8 * rows), ex = extent(x, n, heads, d), ey = extent(y, n, heads, d);
    if (written_meets({ey, st, codes, scale}, {w, b}) || written_meets({st, codes, scale}, {ex}))
      return fail(HYTOPK_EINVAL, "y, the statistics or the checkpoint overlap each other, x or the parameters");
    hk::NormArgs a{};
    a.x = x->data;
    a.y = y->data;
    a.xts = x->token_stride; a.xhs = x->head_stride;
    a.yts = y->token_stride; a.yhs = y->head_stride;
    a.weight = norm->weight;
    a.bias = norm->bias;
    a.stats = reinterpret_cast<float2*>(stats);
    a.codes = save ? static_cast<uint8_t*>(save->codes) : nullptr;
    a.scale = save ? save->scale : nullptr;
    a.rows = (int)rows;
    a.heads = heads;
    a.eps = norm->eps;
    hipStream_t s = static_cast<hipStream_t>(stream);
    Span sp("layer_norm", s);
    HK_HIP(hk::launch_layer_norm(a, d, norm->dtype == HYTOPK_ROWS_FP32, x->dtype, y->dtype,
                                 save ? save->dtype : HYTOPK_BF16, s), "layer norm launch");
    return HYTOPK_OK;
  });
}

size_t hytopk_layer_norm_backward_workspace(int64_t n, int32_t heads, int32_t d) {
  size_t need = 0;
  guarded([&]() -> int {
    const int rc = check_norm_rows(n, heads, d);
    const int blocks = rc == HYTOPK_OK ? hk::norm_backward_blocks(n * heads, d) : 1;
    if (blocks > 1) need = align_up((size_t)blocks * 2 * hk::norm_columns(d) * sizeof(float));
    return rc;
  });
  return need;
}

int hytopk_layer_norm_backward(const hytopk_norm* norm, int64_t n, int32_t heads, int32_t d, const hytopk_rows* dy,
                               const hytopk_rows* x, const hytopk_cache* saved, const float* stats,
                               const hytopk_rows* dx, float* dweight, float* dbias, void* workspace,
                               size_t workspace_bytes, void* stream) {
  return guarded([&]() -> int {
    int rc = check_norm_rows(n, heads, d);
    if (rc) return rc;
    if ((rc = check_norm(norm))) return rc;
    if ((rc = check_rows(dy, n, heads, d))) return rc;
    if ((x != nullptr) == (saved != nullptr)) return fail(HYTOPK_EINVAL, "give the norm's input or its checkpoint");
    const int64_t rows = n * heads;
    if (x ? (rc = check_rows(x, n, heads, d)) : n > 0 && (rc = check_checkpoint(saved, rows, d))) return rc;
    if (dx && (rc = check_rows(dx, n, heads, d))) return rc;
    if ((rc = check_stats(stats))) return rc;
    if (!stats && n > 0) return fail(HYTOPK_EINVAL, "the backward needs the forward's stats");
    if (misaligned(dweight, 4) || misaligned(dbias, 4)) return fail(HYTOPK_EINVAL, "dweight and dbias must be 4-byte aligned");
    const int64_t need = dweight || dbias ? (int64_t)hytopk_layer_norm_backward_workspace(n, heads, d) : 0;
    if (need && (rc = check_ws(workspace, workspace_bytes, (size_t)need))) return rc;
    if (n > 0 && dx) {
      if (!rows_apart(dx, n, heads, d)) return fail(HYTOPK_EINVAL, "rows of dx overlap each other");
      if (!same_rows(dy, dx, n, heads) && rows_meet(dy, dx, n, heads, d))
        return fail(HYTOPK_EINVAL, "dy and dx overlap (dx may be dy itself)");
      if (x && !same_rows(x, dx, n, heads) && rows_meet(x, dx, n, heads, d))
        return fail(HYTOPK_EINVAL, "x and dx overlap (dx may be x itself)");
    }
    const Extent none{0, 0}, w = parameter(norm, norm->weight, d), st = memory(stats, 8 * rows);
    const Extent ws = need ? extent(workspace, need) : none, gw = memory(dweight, 4 * (int64_t)d), gb = memory(dbias, 4 * (int64_t)d);
    const Extent ex = n > 0 ? memory(x, n, heads, d) : none, ey = n > 0 ? extent(dy, n, heads, d) : none;
    const Extent edx = n > 0 ? memory(dx, n, heads, d) : none;
    const Extent codes = saved && n > 0 ? cache_codes(saved) : none, scale = saved && n > 0 ? cache_scale(saved) : none;
    if (written_meets({edx, gw, gb, ws}, {w, st, codes, scale}) || written_meets({gw, gb, ws}, {ex, ey}))
      return fail(HYTOPK_EINVAL, "the gradients or the workspace overlap each other or what is read");
    hk::NormBackArgs a{};
    a.dy = dy->data;
    a.dyts = dy->token_stride; a.dyhs = dy->head_stride;
    if (x) {
      a.x = x->data;
      a.xts = x->token_stride; a.xhs = x->head_stride;
    } else {
      a.x = saved->codes;
      a.scale = saved->scale;
    }
    if (dx) {
      a.dx = dx->data;
      a.dxts = dx->token_stride; a.dxhs = dx->head_stride;
    }
    a.weight = norm->weight;
    a.stats = reinterpret_cast<const float2*>(stats);
    a.part = need ? static_cast<float*>(workspace) : nullptr;
    a.rows = (int)rows;
    a.heads = heads;
    hipStream_t s = static_cast<hipStream_t>(stream);
    Span sp("layer_norm_backward", s);
    HK_HIP(hk::launch_layer_norm_backward(a, d, norm->dtype == HYTOPK_ROWS_FP32, x ? x->dtype : 0,
                                          saved ? saved->dtype : HYTOPK_BF16, dy->dtype, dx ? dx->dtype : dy->dtype,
                                          dweight, dbias, s), "layer norm backward launch");
    return HYTOPK_OK;
  });
}

size_t hytopk_attention_mass_workspace(const hytopk_attention* p) {
  size_t need = 0;
  guarded([&]() -> int {
    const int rc = check_attention(p);
    if (rc) return rc;
    int nsplit = 1, len = 0;
    hk::mass_splits(p->n, p->k, p->d, nsplit, len);
    const size_t parts =
        hk::mass_keeps_parts(p->d, nsplit) ? (size_t)p->n * nsplit * (size_t)hk::mass_rows(p->heads, p->key_heads) : 0;
    need = align_up(std::max<size_t>(parts * sizeof(float2), 1));
    return HYTOPK_OK;
  });
  return need;
}

int hytopk_attention_mass(const hytopk_attention* p, const void* q, const void* k,
                          const int32_t* idx, const float* lse, float* mass, void* workspace,
                          size_t workspace_bytes, void* stream) {
  return guarded([&]() -> int {
    int rc = check_attention(p);
    if (rc) return rc;
    if (p->n == 0) return HYTOPK_OK;
    if (!q || !k || !idx || !mass) return fail(HYTOPK_EINVAL, "q, k, idx and mass must be non-NULL");
    if (misaligned(q, 16) || misaligned(k, 16)) return fail(HYTOPK_EINVAL, "q and k must be 16-byte aligned");
    if (misaligned(idx, 4) || misaligned(lse, 4) || misaligned(mass, 4))
      return fail(HYTOPK_EINVAL, "idx, lse and mass must be 4-byte aligned");
    const size_t ws = lse ? 0 : hytopk_attention_mass_workspace(p);
    if (!lse && (rc = check_ws(workspace, workspace_bytes, ws))) return rc;
    const Extent out = extent(mass, 4 * p->n * p->k), part = extent(workspace, (int64_t)ws);
    const int64_t qb = 2 * p->n * p->heads * p->d, kb = 2 * p->L * p->key_heads * p->d, ib = 4 * p->n * p->k;
    if (touches(out, q, qb) || touches(out, k, kb) || touches(out, idx, ib) ||
        touches(out, lse, 4 * p->n * p->heads) ||
        (ws && (overlap(out, part) || touches(part, q, qb) || touches(part, k, kb) || touches(part, idx, ib))))
      return fail(HYTOPK_EINVAL, "mass and the workspace must not overlap the inputs or each other");
    hk::MassArgs a{};
    a.q = static_cast<const uint16_t*>(q);
    a.k = static_cast<const uint16_t*>(k);
    a.idx = idx;
    a.lse = lse;
    a.part = static_cast<float2*>(workspace);
    a.mass = mass;
    a.L = (int)p->L;
    a.n = (int)p->n;
    a.heads = p->heads;
    a.groups = p->key_heads;
    a.topk = p->k;
    a.scale2 = log2_scale(p);
    a.inv_heads = 1.0f / (float)p->heads;
    hk::mass_splits(p->n, p->k, p->d, a.nsplit, a.split_len);
    hipStream_t s = static_cast<hipStream_t>(stream);
    Span sp("attention_mass", s);
    HK_HIP(hk::launch_attention_mass(a, p->d, s), "attention mass launch");
    return HYTOPK_OK;
  });
}

int hytopk_index_loss(int64_t n, int32_t k, const float* score, const float* mass,
                      const float* weight, float* loss, float* d_score, void* stream) {
  return guarded([&]() -> int {
    if (n < 0 || k <= 0) return fail(HYTOPK_EINVAL, "n must be >= 0 and k > 0");
    if (n >= kMaxRows) return fail(HYTOPK_EUNSUPPORTED, "n >= 2^31");
    if (k > kMaxK) return fail(HYTOPK_EUNSUPPORTED, "k > 2048");
    if (n == 0) return HYTOPK_OK;
    if (!score || !mass) return fail(HYTOPK_EINVAL, "score and mass must be non-NULL");
    if (!loss && !d_score) return fail(HYTOPK_EINVAL, "loss and d_score are both NULL");
    for (const void* x : {(const void*)score, (const void*)mass, (const void*)weight,
                          (const void*)loss, (const void*)d_score})
      if (misaligned(x, 4)) return fail(HYTOPK_EINVAL, "arrays must be 4-byte aligned");
    const int64_t rows = 4 * n, all = rows * k;
    if (d_score && ((d_score != score && touches(extent(d_score, all), score, all)) ||
                    (d_score != mass && touches(extent(d_score, all), mass, all)) ||
                    touches(extent(d_score, all), weight, rows)))
      return fail(HYTOPK_EINVAL, "d_score overlaps an input (it may be score or mass itself)");
    if (loss && (touches(extent(loss, rows), score, all) || touches(extent(loss, rows), mass, all) ||
                 touches(extent(loss, rows), weight, rows) || touches(extent(loss, rows), d_score, all)))
      return fail(HYTOPK_EINVAL, "loss overlaps another array");
    hk::LossArgs a{score, mass, weight, loss, d_score, (int)n, k};
    hipStream_t s = static_cast<hipStream_t>(stream);
    Span sp("index_loss", s);
    HK_HIP(hk::launch_index_loss(a, s), "index loss launch");
    return HYTOPK_OK;
  });
}

}  // extern "C"
