// Host-side exercise of the argument validation of the operators around the selection (rotary positions,
// the cache, the attention mass, the index loss), built like abi_validation.cpp with AddressSanitizer and
// UndefinedBehaviorSanitizer on the host code.  Sizes, strides, positions and pointers at the ends of their
// types; every call is refused (or sized) before any HIP call: where all else is in order, by the
// fault that it looks for last.  Exit status 0 when every expectation holds.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <limits>
#include <vector>

#include "hytopk.h"

static int failures = 0;

static void expect(bool ok, const char* what) {
  if (!ok) {
    std::printf("FAIL: %s (last error: %s)\n", what, hytopk_last_error());
    ++failures;
  }
}

static void refused(int rc, int status, const char* words, const char* what) {
  expect(rc == status && std::strstr(hytopk_last_error(), words) != nullptr, what);
}

template <typename T = void>
static T* at(int i, int64_t off = 0) {
  return reinterpret_cast<T*>((uintptr_t(i + 1) << 34) + (uintptr_t)off);
}

constexpr int64_t kTop = std::numeric_limits<int64_t>::max(), kBottom = std::numeric_limits<int64_t>::min();
constexpr int32_t kTop32 = std::numeric_limits<int32_t>::max(), kBottom32 = std::numeric_limits<int32_t>::min();

static hytopk_rows rows(void* data, int64_t ts, int64_t hs, int32_t dtype = HYTOPK_ROWS_BF16) {
  return hytopk_rows{data, ts, hs, dtype, 0};
}

static void frequencies() {
  std::vector<double> f(512);
  double gain = 0;
  for (int32_t dim : {2, 64, 1024})
    for (int32_t s = 0; s <= 3; ++s)
      for (double factor : {1.0, 40.0, 1e308})
        for (double base : {std::nextafter(1.0, 2.0), 10000.0, 1e308})
          for (int64_t original : {int64_t(1), int64_t(4096), kTop}) {
            expect(hytopk_rotary_frequencies(dim, base, s, factor, original, f.data(), &gain) == HYTOPK_OK, "frequencies");
            expect(f[0] <= 1.0 && f[0] > 0.0 && std::isfinite(gain), "frequencies are finite");
          }
  for (int32_t dim : {kTop32, kTop32 - 1, 0, -2, kBottom32, 1026, 7})
    expect(hytopk_rotary_frequencies(dim, 1e4, 0, 1, 0, f.data(), &gain) != HYTOPK_OK, "bad dim");
  for (int32_t s : {-1, 4, kTop32, kBottom32})
    refused(hytopk_rotary_frequencies(64, 1e4, s, 1, 0, f.data(), &gain), HYTOPK_EINVAL, "scaling", "bad scaling");
  const double inf = std::numeric_limits<double>::infinity(), nan = std::nan("");
  for (double base : {1.0, 0.0, -5.0, inf, nan})
    refused(hytopk_rotary_frequencies(64, base, 0, 1, 0, f.data(), &gain), HYTOPK_EINVAL, "base", "bad base");
  for (double factor : {0.5, -1.0, inf, nan})
    refused(hytopk_rotary_frequencies(64, 1e4, 1, factor, 0, f.data(), &gain), HYTOPK_EINVAL, "factor", "bad factor");
  for (int64_t original : {int64_t(0), int64_t(-1), kBottom})
    refused(hytopk_rotary_frequencies(64, 1e4, 3, 4, original, f.data(), &gain), HYTOPK_EINVAL, "original", "bad context");
  refused(hytopk_rotary_frequencies(64, 1e4, 0, 1, 0, nullptr, &gain), HYTOPK_EINVAL, "non-NULL", "no freq");
  refused(hytopk_rotary_frequencies(64, 1e4, 0, 1, 0, f.data(), nullptr), HYTOPK_EINVAL, "non-NULL", "no gain");
}

static void rotary() {
  const hytopk_rows x = rows(at(0), 192, 64), y = rows(at(1), 192, 64);
  hytopk_rotary_plan p{at<double>(1), 1.0, 32, 0, HYTOPK_ROTARY_HALF, 0};  // over y: looked for last
  auto call = [&](int64_t n, int32_t heads, int32_t d, const hytopk_rows* a, const hytopk_rows* b, const int32_t* pos = nullptr,
                  int64_t start = 0) { return hytopk_rotary(&p, n, heads, d, a, b, pos, start, 0, nullptr); };
  refused(call(4, 3, 64, &x, &y), HYTOPK_EINVAL, "the positions or the plan", "rotary");
  for (int64_t n : {kBottom, int64_t(-1)}) refused(call(n, 3, 64, &x, &y), HYTOPK_EINVAL, "n must be >= 0", "rotary n");
  for (int64_t n : {kTop, int64_t(1) << 31}) refused(call(n, 3, 64, &x, &y), HYTOPK_EUNSUPPORTED, "n >= 2^31", "rotary n");
  refused(call(4, kTop32, kTop32, &x, &y), HYTOPK_EUNSUPPORTED, "heads * d", "rotary heads");
  refused(call(4, kBottom32, 64, &x, &y), HYTOPK_EINVAL, "heads, d > 0", "rotary heads");
  for (int64_t s : {kTop, int64_t(1) << 60}) {
    hytopk_rows a = rows(at(0), s, 64), b = rows(at(0), 192, s);
    refused(call(4, 3, 64, &a, &y), HYTOPK_EINVAL, "more memory", "token stride");
    refused(call(4, 3, 64, &b, &y), HYTOPK_EINVAL, "more memory", "head stride");
    refused(call((int64_t(1) << 31) - 1, 3, 64, &a, &y), HYTOPK_EINVAL, "more memory", "token stride");
    // one token, one head: the stride counts nothing
    hytopk_rows c = rows(at(1), s, s);
    refused(call(1, 1, 64, &x, &c), HYTOPK_EINVAL, "the positions or the plan", "strides of one row");
    refused(call(1, 1, 64, &c, &c), HYTOPK_EINVAL, "the positions or the plan", "one row in place");
    hytopk_rows e = rows(at(1, 64), s, s);
    refused(call(1, 1, 64, &e, &y), HYTOPK_EINVAL, "x and y overlap", "one row over another");
  }
  for (int64_t s : {kBottom, int64_t(-1)}) {
    hytopk_rows a = rows(at(0), s, 64), b = rows(at(0), 192, s);
    refused(call(4, 3, 64, &a, &y), HYTOPK_EINVAL, "strides must be >= 0", "token stride");
    refused(call(4, 3, 64, &b, &y), HYTOPK_EINVAL, "strides must be >= 0", "head stride");
  }
  // slices of one buffer, the largest strides that pass
  for (int32_t type : {HYTOPK_ROWS_BF16, HYTOPK_ROWS_FP32})
    for (int64_t s : {int64_t(1) << 59, (int64_t(1) << 60) - 128, int64_t(1) << 40}) {
      hytopk_rows a = rows(at(0), s, 64, type), b = rows(at(0, 1024), s, 64, type), c = rows(at(0, 32), s, 64, type);
      p.freq = at<double>(0, 1024);
      refused(call(2, 1, 64, &a, &b), HYTOPK_EINVAL, "the positions or the plan", "rows between rows");
      refused(call(2, 1, 64, &b, &a), HYTOPK_EINVAL, "the positions or the plan", "rows between rows");
      refused(call(2, 1, 64, &a, &c), HYTOPK_EINVAL, "x and y overlap", "rows over rows");
      hytopk_rows g = rows(at(0), 64, s, type), h = rows(at(0, 1024), 64, s, type);
      refused(call(2, 2, 64, &g, &h), HYTOPK_EINVAL, "the positions or the plan", "heads before tokens");
    }
  p.freq = at<double>(1);
  const int64_t last = int64_t(1) << 31;
  for (int64_t start : {kBottom, int64_t(-1), last - 3, kTop})
    refused(call(4, 3, 64, &x, &y, nullptr, start), HYTOPK_EINVAL, "positions q_start", "start");
  refused(call(4, 3, 64, &x, &y, nullptr, last - 4), HYTOPK_EINVAL, "the positions or the plan", "the last start");
  for (int32_t v : {kBottom32, -1, kTop32}) {
    hytopk_rotary_plan bad = p;
    bad.first = v;
    refused(hytopk_rotary(&bad, 4, 3, 64, &x, &y, nullptr, 0, 0, nullptr), HYTOPK_EINVAL, "outside the head", "first");
    bad = p;
    bad.layout = v;
    refused(hytopk_rotary(&bad, 4, 3, 64, &x, &y, nullptr, 0, 0, nullptr), HYTOPK_EINVAL, "layout", "layout");
    bad = p;
    bad.dim = v;
    expect(hytopk_rotary(&bad, 4, 3, 64, &x, &y, nullptr, 0, 0, nullptr) == HYTOPK_EINVAL, "dim");
  }
  for (double gain : {std::nan(""), 1e308, -std::numeric_limits<double>::infinity()}) {
    hytopk_rotary_plan bad = p;
    bad.gain = gain;
    refused(hytopk_rotary(&bad, 4, 3, 64, &x, &y, nullptr, 0, 0, nullptr), HYTOPK_EINVAL, "gain", "gain");
  }
  expect(call(4, 3, 64, nullptr, &y) == HYTOPK_EINVAL && call(4, 3, 64, &x, nullptr) == HYTOPK_EINVAL, "no rows");
  expect(hytopk_rotary(nullptr, 4, 3, 64, &x, &y, nullptr, 0, 0, nullptr) == HYTOPK_EINVAL, "no plan");
  const hytopk_rows none = rows(nullptr, 0, 0);
  expect(call(0, 3, 64, &none, &none) == HYTOPK_OK, "no tokens");
}

static void cache() {
  hytopk_cache c{at(0), at(0, 256), 1 << 20, 1, 128, HYTOPK_FP8_E4M3, 0};  // scales over the codes: looked for last
  const hytopk_rows x = rows(at(1), 128, 128);
  const hytopk_rotary_plan p{at<double>(2), 1.0, 64, 0, HYTOPK_ROTARY_HALF, 0};
  auto write = [&](const hytopk_cache& k, int64_t n, const int32_t* slots, int64_t start, int64_t q_start = 0, size_t ws = size_t(1) << 40) {
    return hytopk_cache_write(&k, n, &x, slots, start, &p, nullptr, q_start, at(4), ws, nullptr);
  };
  auto read = [&](const hytopk_cache& k, int64_t n, int64_t start) {
    return hytopk_cache_read(&k, n, nullptr, start, at(0), HYTOPK_ROWS_BF16, nullptr);  // over the codes
  };
  refused(write(c, 4, nullptr, 0), HYTOPK_EINVAL, "codes and scales overlap", "write");
  refused(write(c, 5000, at<int32_t>(5), 0), HYTOPK_EINVAL, "codes and scales overlap", "write by slot");
  refused(read(c, 4, 0), HYTOPK_EINVAL, "out overlaps the cache", "read");
  for (int64_t n : {kBottom, int64_t(-1)}) {
    refused(write(c, n, nullptr, 0), HYTOPK_EINVAL, "n must be >= 0", "write n");
    refused(read(c, n, 0), HYTOPK_EINVAL, "n must be >= 0", "read n");
  }
  for (int64_t n : {kTop, int64_t(1) << 31}) {
    refused(write(c, n, nullptr, 0), HYTOPK_EUNSUPPORTED, "n >= 2^31", "write n");
    refused(read(c, n, 0), HYTOPK_EUNSUPPORTED, "n >= 2^31", "read n");
  }
  for (int64_t start : {kBottom, int64_t(-1), (int64_t(1) << 20) - 3, kTop}) {
    refused(write(c, 4, nullptr, start), HYTOPK_EINVAL, "outside the cache", "write start");
    refused(read(c, 4, start), HYTOPK_EINVAL, "outside the cache", "read start");
  }
  for (int64_t start : {kBottom, (int64_t(1) << 31) - 3, kTop})
    refused(write(c, 4, nullptr, 0, start), HYTOPK_EINVAL, "positions q_start", "positions");
  refused(write(c, 5000, at<int32_t>(5), 0, 0, 0), HYTOPK_EWORKSPACE, "too small", "workspace");
  for (int64_t L : {kBottom, int64_t(0), kTop, int64_t(1) << 31}) {
    hytopk_cache k = c;
    k.L = L;
    expect(write(k, 4, nullptr, 0) != HYTOPK_OK && read(k, 4, 0) != HYTOPK_OK, "L");
    expect(hytopk_cache_write_workspace(&k, kTop, 1) == 0, "no workspace of a bad L");
  }
  for (int32_t v : {kBottom32, 0, kTop32, kTop32 - 31}) {
    hytopk_cache k = c;
    k.heads = v;
    expect(write(k, 4, nullptr, 0) != HYTOPK_OK && read(k, 4, 0) != HYTOPK_OK, "heads");
    k = c;
    k.d = v;
    expect(write(k, 4, nullptr, 0) != HYTOPK_OK && read(k, 4, 0) != HYTOPK_OK, "d");
    k = c;
    k.dtype = v == 0 ? 4 : v;
    refused(write(k, 4, nullptr, 0), HYTOPK_EINVAL, "unknown dtype", "dtype");
  }
  // the largest cache of every format, read and written at its end
  for (int32_t dtype : {HYTOPK_BF16, HYTOPK_FP8_E4M3, HYTOPK_MXFP8_E4M3, HYTOPK_MXFP4_E2M1}) {
    hytopk_cache k{at(0), at(0, 256), (int64_t(1) << 31) - 1, 256, 32, dtype, 0};
    const hytopk_rows w = rows(at(0, -8192), 8192, 32);
    refused(hytopk_cache_write(&k, 1, &w, nullptr, k.L - 1, nullptr, nullptr, 0, nullptr, 0, nullptr), HYTOPK_EINVAL, "x overlaps the cache", "the largest cache");
    refused(read(k, 1, k.L - 1), HYTOPK_EINVAL, "out overlaps the cache", "the largest cache");
    expect(hytopk_cache_write_workspace(&k, kTop, 1) == (size_t(1) << 33), "its workspace");
  }
  expect(hytopk_cache_write_workspace(nullptr, 5000, 1) == 0 && hytopk_cache_write_workspace(&c, kBottom, 1) == 0, "no workspace");
  expect(hytopk_cache_write(nullptr, 4, &x, nullptr, 0, nullptr, nullptr, 0, nullptr, 0, nullptr) == HYTOPK_EINVAL, "no cache");
  expect(hytopk_cache_read(nullptr, 4, nullptr, 0, at(6), 0, nullptr) == HYTOPK_EINVAL, "no cache");
  expect(hytopk_cache_write(&c, 4, nullptr, nullptr, 0, nullptr, nullptr, 0, nullptr, 0, nullptr) == HYTOPK_EINVAL, "no rows");
  for (int32_t t : {kBottom32, -1, 2, kTop32})
    refused(hytopk_cache_read(&c, 4, nullptr, 0, at(6), t, nullptr), HYTOPK_EINVAL, "rows dtype", "type of what is read");
}

static void attention_mass() {
  auto call = [&](const hytopk_attention& a, const float* lse = nullptr, size_t ws = size_t(1) << 50) {
    return hytopk_attention_mass(&a, at(0), at(1), at<int32_t>(2), lse, at<float>(2), at(4), ws, nullptr);  // over the indices
  };
  const hytopk_attention base{1000, 4, 64, 1, 128, 100, 0.1f, 0};
  refused(call(base), HYTOPK_EINVAL, "must not overlap", "mass");
  refused(call(base, at<float>(3)), HYTOPK_EINVAL, "must not overlap", "mass with lse");
  // the largest sizes of every width: the workspace's size and the extents stay within 64 bits
  for (int32_t d : {64, 96, 128, 192, 256, 512, 576}) {
    const int64_t n = (int64_t(1) << (d > 256 ? 23 : 24)) - 1;
    for (int32_t key_heads : {1, 2, 1024}) {
      const hytopk_attention a{(int64_t(1) << 31) - 1, n, 1024, key_heads, d, 2048, 1.0f, 0};
      const size_t ws = hytopk_attention_mass_workspace(&a);
      expect(ws > 0 && ws % 256 == 0 && ws <= size_t(n) * 1024 * 16 * 8 * 32, "workspace of the largest mass");
      refused(call(a), HYTOPK_EINVAL, "must not overlap", "the largest mass");
    }
    const hytopk_attention few{5, 1, 1024, 1024, d, 2048, 1.0f, 0};
    expect(hytopk_attention_mass_workspace(&few) >= size_t(256), "workspace of one query");
    refused(call(few, nullptr, 0), HYTOPK_EWORKSPACE, "too small", "no workspace");
  }
  for (int64_t v : {kBottom, int64_t(-1), kTop, int64_t(1) << 31}) {
    hytopk_attention a = base;
    a.n = v;
    expect(call(a) != HYTOPK_OK && hytopk_attention_mass_workspace(&a) == 0, "n");
    a = base;
    a.L = v;
    expect(call(a) != HYTOPK_OK && hytopk_attention_mass_workspace(&a) == 0, "L");
  }
  for (int32_t v : {kBottom32, -1, 0, kTop32}) {
    hytopk_attention a = base;
    a.heads = v;
    expect(call(a) != HYTOPK_OK && hytopk_attention_mass_workspace(&a) == 0, "heads");
    a = base;
    a.key_heads = v;
    expect(call(a) != HYTOPK_OK && hytopk_attention_mass_workspace(&a) == 0, "key heads");
    a = base;
    a.d = v;
    expect(call(a) != HYTOPK_OK && hytopk_attention_mass_workspace(&a) == 0, "d");
    a = base;
    a.k = v;
    expect(call(a) != HYTOPK_OK && hytopk_attention_mass_workspace(&a) == 0, "k");
  }
  for (float v : {std::numeric_limits<float>::infinity(), -std::numeric_limits<float>::max(), std::nanf("")}) {
    hytopk_attention a = base;
    a.softmax_scale = v;
    refused(call(a), HYTOPK_EINVAL, "softmax_scale", "scale");
  }
  expect(hytopk_attention_mass_workspace(nullptr) == 0, "no attention");
  expect(hytopk_attention_mass(nullptr, at(0), at(1), at<int32_t>(2), nullptr, at<float>(3), at(4), 1, nullptr) == HYTOPK_EINVAL, "no attention");
  hytopk_attention none = base;
  none.n = 0;
  expect(hytopk_attention_mass(&none, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0, nullptr) == HYTOPK_OK, "no queries");
}

static void index_loss() {
  auto call = [&](int64_t n, int32_t k) {
    return hytopk_index_loss(n, k, at<float>(0), at<float>(2000), at<float>(4000), at<float>(4000), at<float>(6000),
                             nullptr);  // 16 TiB and more apart; loss over the weights
  };
  refused(call(4, 100), HYTOPK_EINVAL, "loss overlaps", "loss");
  refused(call((int64_t(1) << 31) - 1, 2048), HYTOPK_EINVAL, "loss overlaps", "the most rows");
  for (int64_t n : {kBottom, int64_t(-1)}) refused(call(n, 5), HYTOPK_EINVAL, "n must be >= 0", "loss n");
  for (int64_t n : {kTop, int64_t(1) << 31}) refused(call(n, 5), HYTOPK_EUNSUPPORTED, "n >= 2^31", "loss n");
  for (int32_t k : {kBottom32, -1, 0}) refused(call(4, k), HYTOPK_EINVAL, "k > 0", "loss k");
  for (int32_t k : {2049, kTop32}) refused(call(4, k), HYTOPK_EUNSUPPORTED, "k > 2048", "loss k");
  expect(hytopk_index_loss(0, 2048, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr) == HYTOPK_OK, "no rows");
}

int main() {
  frequencies();
  rotary();
  cache();
  attention_mass();
  index_loss();
  std::printf("ok: %d failure(s)\n", failures);
  return failures != 0;
}
