// Host-side exercise of the argument validation of the layer norm and of rotary plans of several axes, built like
// operators_validation.cpp with AddressSanitizer and UndefinedBehaviorSanitizer on the host code.  Sizes, strides and
// pointers at the ends of their types; every call is refused (or sized) before any HIP call: where all else is in order,
// by the fault that it looks for last.  Exit status 0 when every expectation holds.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <initializer_list>
#include <limits>

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
  return reinterpret_cast<T*>((uintptr_t(i + 1) << 42) + (uintptr_t)off);
}

constexpr int64_t kTop = std::numeric_limits<int64_t>::max(), kBottom = std::numeric_limits<int64_t>::min();
constexpr int32_t kTop32 = std::numeric_limits<int32_t>::max(), kBottom32 = std::numeric_limits<int32_t>::min();

static hytopk_rows rows(void* data, int64_t ts, int64_t hs, int32_t dtype = HYTOPK_ROWS_BF16) {
  return hytopk_rows{data, ts, hs, dtype, 0};
}

static const char* kForward = "overlap each other, x or the parameters";
static const char* kBackward = "the gradients or the workspace overlap";

static void forward() {
  const hytopk_rows x = rows(at(0), 192, 64), y = rows(at(1), 192, 64);
  const hytopk_norm base{at(2), at(3), HYTOPK_ROWS_FP32, 1e-5f};
  hytopk_cache c{at(4), at(5), 1 << 20, 1, 64, HYTOPK_FP8_E4M3, 0};
  // the statistics lie over the weight: looked for last
  auto call = [&](const hytopk_norm& p, int64_t n, int32_t heads, int32_t d, const hytopk_rows* a, const hytopk_rows* b,
                  const hytopk_cache* save = nullptr) {
    return hytopk_layer_norm(&p, n, heads, d, a, b, at<float>(2), save, nullptr);
  };
  refused(call(base, 4, 3, 64, &x, &y), HYTOPK_EINVAL, kForward, "forward");
  refused(call(base, 4, 3, 64, &x, &x), HYTOPK_EINVAL, kForward, "in place");
  refused(call(base, 4, 3, 64, &x, &y, &c), HYTOPK_EINVAL, kForward, "with a checkpoint");
  const hytopk_rows wide = rows(at(0), 8192, 8192, HYTOPK_ROWS_FP32), far = rows(at(40), 8192, 8192, HYTOPK_ROWS_FP32);
  refused(call(base, (int64_t(1) << 31) - 1, 1, 8192, &wide, &far), HYTOPK_EINVAL, kForward, "the most rows");
  for (int64_t n : {kBottom, int64_t(-1)}) refused(call(base, n, 3, 64, &x, &y), HYTOPK_EINVAL, "n must be >= 0", "n");
  for (int64_t n : {kTop, int64_t(1) << 31}) refused(call(base, n, 3, 64, &x, &y), HYTOPK_EUNSUPPORTED, "n >= 2^31", "n");
  refused(call(base, int64_t(1) << 30, 2, 64, &x, &y), HYTOPK_EUNSUPPORTED, "n * heads", "rows");
  refused(call(base, (int64_t(1) << 31) - 1, kTop32, 1, &x, &y), HYTOPK_EUNSUPPORTED, "heads", "rows and heads");
  refused(call(base, 4, kTop32, kTop32, &x, &y), HYTOPK_EUNSUPPORTED, "heads * d", "heads");
  for (int32_t v : {kBottom32, -1, 0}) {
    refused(call(base, 4, v, 64, &x, &y), HYTOPK_EINVAL, "heads, d > 0", "heads");
    refused(call(base, 4, 3, v, &x, &y), HYTOPK_EINVAL, "heads, d > 0", "d");
  }
  for (int32_t d : {8193, kTop32}) refused(call(base, 4, 1, d, &x, &y), HYTOPK_EUNSUPPORTED, "d <= 8192", "d");
  for (int64_t s : {kTop, int64_t(1) << 60}) {
    const hytopk_rows a = rows(at(0), s, 64), b = rows(at(0), 192, s), one = rows(at(1), s, s);
    refused(call(base, 4, 3, 64, &a, &y), HYTOPK_EINVAL, "more memory", "token stride");
    refused(call(base, 4, 3, 64, &x, &b), HYTOPK_EINVAL, "more memory", "head stride");
    refused(call(base, 1, 1, 64, &x, &one), HYTOPK_EINVAL, kForward, "strides of one row");
    refused(call(base, 1, 1, 64, &one, &one), HYTOPK_EINVAL, kForward, "one row in place");
  }
  for (int64_t s : {kBottom, int64_t(-1)}) {
    const hytopk_rows a = rows(at(0), s, 64);
    refused(call(base, 4, 3, 64, &a, &y), HYTOPK_EINVAL, "strides must be >= 0", "negative stride");
  }
  for (float eps : {-1.0f, std::nanf(""), std::numeric_limits<float>::infinity()}) {
    hytopk_norm p = base;
    p.eps = eps;
    refused(call(p, 4, 3, 64, &x, &y), HYTOPK_EINVAL, "eps", "eps");
  }
  for (int32_t v : {kBottom32, -1, 2, kTop32}) {
    hytopk_norm p = base;
    p.dtype = v;
    refused(call(p, 4, 3, 64, &x, &y), HYTOPK_EINVAL, "norm's parameters", "parameters' type");
  }
  for (int64_t L : {kBottom, int64_t(0), int64_t(11), kTop, int64_t(1) << 31}) {
    hytopk_cache k = c;
    k.L = L;
    expect(call(base, 4, 3, 64, &x, &y, &k) != HYTOPK_OK, "checkpoint rows");
  }
  for (int32_t v : {kBottom32, -1, 0, 2, kTop32}) {
    hytopk_cache k = c;
    k.heads = v;
    expect(call(base, 4, 3, 64, &x, &y, &k) != HYTOPK_OK, "checkpoint heads");
    k = c;
    k.d = v;
    expect(call(base, 4, 3, 64, &x, &y, &k) != HYTOPK_OK, "checkpoint d");
    k = c;
    k.dtype = v == 2 ? 3 : v;
    expect(call(base, 4, 3, 64, &x, &y, &k) != HYTOPK_OK, "checkpoint format");
  }
  const hytopk_rows none = rows(nullptr, 0, 0);
  expect(hytopk_layer_norm(&base, 0, 3, 64, &none, &none, nullptr, &c, nullptr) == HYTOPK_OK, "no rows");
  expect(hytopk_layer_norm(nullptr, 4, 3, 64, &x, &y, nullptr, nullptr, nullptr) == HYTOPK_EINVAL, "no norm");
  expect(call(base, 4, 3, 64, nullptr, &y) == HYTOPK_EINVAL && call(base, 4, 3, 64, &x, nullptr) == HYTOPK_EINVAL, "no rows given");
}

static void backward() {
  const hytopk_rows dy = rows(at(0), 192, 64), x = rows(at(1), 192, 64), dx = rows(at(2), 192, 64);
  const hytopk_norm base{at(3), nullptr, HYTOPK_ROWS_FP32, 0.0f};
  const hytopk_cache c{at(4), at(5), 1 << 20, 1, 64, HYTOPK_MXFP8_E4M3, 0};
  // dbias lies over dweight: looked for last
  auto call = [&](int64_t n, int32_t heads, int32_t d, const hytopk_rows* a, const hytopk_rows* b, const hytopk_cache* saved,
                  const hytopk_rows* e, size_t ws = size_t(1) << 40) {
    return hytopk_layer_norm_backward(&base, n, heads, d, a, b, saved, at<const float>(6), e, at<float>(7), at<float>(7, 8), at(8),
                                      ws, nullptr);
  };
  for (int64_t n : {int64_t(1), int64_t(4), int64_t(100), int64_t(1) << 20}) {
    refused(call(n, 3, 64, &dy, &x, nullptr, &dx), HYTOPK_EINVAL, kBackward, "backward");
    refused(call(n, 3, 64, &dy, &x, nullptr, &dy), HYTOPK_EINVAL, kBackward, "over dy");
    refused(call(n, 3, 64, &dy, &x, nullptr, nullptr), HYTOPK_EINVAL, kBackward, "sums alone");
  }
  refused(call(4, 3, 64, &dy, nullptr, &c, &dx), HYTOPK_EINVAL, kBackward, "from a checkpoint");
  refused(call(1 << 20, 3, 64, &dy, &x, nullptr, &dx, 0), HYTOPK_EWORKSPACE, "too small", "workspace");
  refused(call(4, 3, 64, &dy, &x, &c, &dx), HYTOPK_EINVAL, "input or its checkpoint", "both");
  refused(call(4, 3, 64, &dy, nullptr, nullptr, &dx), HYTOPK_EINVAL, "input or its checkpoint", "neither");
  for (int64_t n : {kBottom, int64_t(-1), kTop, int64_t(1) << 31}) {
    expect(call(n, 3, 64, &dy, &x, nullptr, &dx) != HYTOPK_OK, "n");
    expect(hytopk_layer_norm_backward_workspace(n, 3, 64) == 0, "workspace of n");
  }
  for (int32_t v : {kBottom32, -1, 0, kTop32}) {
    expect(call(4, v, 64, &dy, &x, nullptr, &dx) != HYTOPK_OK && hytopk_layer_norm_backward_workspace(4, v, 64) == 0, "heads");
    expect(call(4, 3, v, &dy, &x, nullptr, &dx) != HYTOPK_OK && hytopk_layer_norm_backward_workspace(4, 3, v) == 0, "d");
  }
  for (int64_t s : {kTop, int64_t(1) << 60, kBottom, int64_t(-1)}) {
    const hytopk_rows a = rows(at(0), s, 64);
    expect(call(4, 3, 64, &a, &x, nullptr, &dx) == HYTOPK_EINVAL, "dy's stride");
    expect(call(4, 3, 64, &dy, &a, nullptr, &dx) == HYTOPK_EINVAL, "x's stride");
    expect(call(4, 3, 64, &dy, &x, nullptr, &a) == HYTOPK_EINVAL, "dx's stride");
  }
  const size_t most = hytopk_layer_norm_backward_workspace((int64_t(1) << 31) - 1, 1, 8192);
  expect(most > 0 && most <= size_t(64) << 20, "workspace of the most rows");
  const hytopk_rows none = rows(nullptr, 0, 0);
  expect(hytopk_layer_norm_backward(&base, 0, 3, 64, &none, &none, nullptr, nullptr, &none, nullptr, nullptr, nullptr, 0, nullptr) ==
             HYTOPK_OK, "no rows");
}

static void axes() {
  const hytopk_rows x = rows(at(0), 192, 64), y = rows(at(1), 192, 64);
  auto call = [&](int32_t axes, int64_t n, const int32_t* pos) {
    const hytopk_rotary_plan p{at<double>(1), 1.0, 32, 0, HYTOPK_ROTARY_HALF, axes};  // over y: looked for last
    return hytopk_rotary(&p, n, 3, 64, &x, &y, pos, 0, 0, nullptr);
  };
  for (int32_t a : {0, 1, 2, 16})
    for (int64_t n : {int64_t(1), int64_t(4), int64_t(1) << 30})
      refused(call(a, n, at<int32_t>(20)), HYTOPK_EINVAL, "the positions or the plan", "axes");
  for (int32_t a : {kBottom32, -1}) refused(call(a, 4, nullptr), HYTOPK_EINVAL, "axes", "negative axes");
  for (int32_t a : {17, kTop32}) refused(call(a, 4, nullptr), HYTOPK_EUNSUPPORTED, "axes > 16", "many axes");
}

int main() {
  forward();
  backward();
  axes();
  std::printf("ok: %d failure(s)\n", failures);
  return failures != 0;
}
