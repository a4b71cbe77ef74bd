// Host-only check of the C ABI of linear attention and rotary positions under
// AddressSanitizer and UndefinedBehaviorSanitizer: every call below fails, sizes
// or has no work, so there is no HIP call (no GPU needed).  Built and run by
// tests/test_linear_sanitize.py; exits non-zero on a mismatch.
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "gdn_linear.h"

static char message[512];
namespace gdn {   // the library's error slot, which lives with the frame operators
gdn_status fail(gdn_status s, const char* format, ...) {
  va_list a;
  va_start(a, format);
  std::vsnprintf(message, sizeof message, format, a);
  va_end(a);
  return s;
}
void clear_error() { message[0] = 0; }
}  // namespace gdn

static int failures = 0;
#define EXPECT(cond)                                                            \
  do {                                                                          \
    if (!(cond)) {                                                              \
      std::fprintf(stderr, "FAILED %s:%d: %s\n", __FILE__, __LINE__, #cond);    \
      ++failures;                                                               \
    }                                                                           \
  } while (0)

// Deterministic 64-bit LCG for the field fuzz.
static uint64_t rng = 0x9e3779b97f4a7c15ull;
static int64_t draw(int64_t lo, int64_t hi) {
  rng = rng * 6364136223846793005ull + 1442695040888963407ull;
  return lo + (int64_t)((rng >> 33) % (uint64_t)(hi - lo + 1));
}
// Mostly in [lo, hi], now and then an extreme.
static int32_t field(int64_t lo, int64_t hi) {
  const int32_t odd[] = {0, -1, INT32_MAX, INT32_MIN, 65536};
  return draw(0, 19) == 0 ? odd[draw(0, 4)] : (int32_t)draw(lo, hi);
}
static int64_t tokens() {
  const int64_t odd[] = {0, -1, (1ll << 31) - 256, 1ll << 31, INT64_MAX, INT64_MIN};
  return draw(0, 9) == 0 ? odd[draw(0, 5)] : draw(0, 1ll << draw(0, 30));
}
static float real() {
  const float odd[] = {0.f, -1.f, NAN, INFINITY, -INFINITY};
  return draw(0, 9) == 0 ? odd[draw(0, 4)] : 0.125f;
}

static void linear() {
  void* const at = reinterpret_cast<void*>(uintptr_t{0x10000});
  void* const off = reinterpret_cast<void*>(uintptr_t{0x10004});
  float* const f = static_cast<float*>(at);
  int32_t* const i = static_cast<int32_t*>(at);
  size_t a = 0, b = 0;
  EXPECT(gdn_linear_workspace_size(nullptr, 0, &a) == GDN_ERR_INVALID_ARGUMENT && message[0]);
  int good = 0;
  for (int it = 0; it < 20000; ++it) {
    gdn_linear_problem p;
    std::memset(&p, 0, sizeof p);
    p.abi_version = draw(0, 30) ? GDN_ABI_VERSION : field(0, 3);
    p.heads_k = field(1, 8);
    p.heads_v = draw(0, 9) ? (int32_t)(p.heads_k % 100000LL * draw(1, 4)) : field(1, 8);
    p.d_k = 16 * (int32_t)draw(0, 9);
    p.d_v = 16 * (int32_t)draw(0, 9);
    p.qkv_dtype = field(0, 1);
    p.out_dtype = field(0, 1);
    p.state_rows = field(0, 100);
    p.tokens = tokens();
    if (draw(0, 3) == 0) p.q_stride = field(0, 4096);
    if (draw(0, 3) == 0) p.v_stride = field(0, 4096);
    p.sequences = field(0, 1 << draw(0, 18));
    p.gate_per_head = draw(0, 20) ? (int32_t)draw(0, 1) : field(0, 1);
    p.scale = real();
    if (draw(0, 40) == 0) p.reserved[draw(0, 4)] = 1;
    const gdn_status s = gdn_linear_workspace_size(&p, 0, &a);
    EXPECT(gdn_linear_workspace_size(&p, 1, &b) == s);
    if (s != GDN_OK) {
      EXPECT(s == GDN_ERR_INVALID_ARGUMENT && message[0]);
      EXPECT(gdn_linear_forward(&p, at, at, at, f, i, nullptr, f, at, f, at, SIZE_MAX, nullptr) == GDN_ERR_INVALID_ARGUMENT);
      EXPECT(gdn_linear_backward(&p, at, at, at, f, i, f, at, f, at, at, at, f, f, at, SIZE_MAX, nullptr) ==
             GDN_ERR_INVALID_ARGUMENT);
      continue;
    }
    ++good;
    // every plan: whole chunks, at least one segment a sequence, places for every bound
    for (int grad = 0; grad < 2; ++grad) {
      gdn::LinearProblem q;
      q.hk = p.heads_k;
      q.hv = p.heads_v;
      q.dk = p.d_k;
      q.dv = p.d_v;
      q.in_bf16 = p.qkv_dtype == GDN_BF16;
      q.tokens = p.tokens;
      q.sequences = p.sequences;
      const gdn::LinearPlan plan = gdn::linear_plan(q, grad != 0);
      EXPECT(plan.L >= 64 && plan.L % 64 == 0);
      EXPECT(plan.bounds == p.tokens / plan.L && plan.slots == plan.bounds + p.sequences);
      EXPECT(plan.slots * p.heads_v < (1ll << 26));
    }
    if (p.sequences > 0 && p.tokens > 0) {
      EXPECT(gdn_linear_forward(&p, nullptr, at, at, f, i, nullptr, f, at, f, at, SIZE_MAX, nullptr) == GDN_ERR_INVALID_ARGUMENT);
      EXPECT(gdn_linear_forward(&p, off, at, at, f, i, nullptr, f, at, f, at, SIZE_MAX, nullptr) == GDN_ERR_INVALID_ARGUMENT);
      EXPECT(gdn_linear_backward(&p, at, at, at, f, i, f, nullptr, f, at, at, at, f, f, at, SIZE_MAX, nullptr) ==
             GDN_ERR_INVALID_ARGUMENT);
      if (a > 0) EXPECT(gdn_linear_forward(&p, at, at, at, f, i, nullptr, f, at, f, at, a - 1, nullptr) == GDN_ERR_WORKSPACE_TOO_SMALL);
      EXPECT(gdn_linear_backward(&p, at, at, at, f, i, f, at, f, at, at, at, f, f, at, b - 1, nullptr) == GDN_ERR_WORKSPACE_TOO_SMALL);
    }
    if (p.sequences == 0) EXPECT(gdn_linear_forward(&p, at, at, at, f, i, nullptr, f, at, f, at, a, nullptr) == GDN_OK);
    if (p.tokens == 0) EXPECT(gdn_linear_decode(&p, at, at, at, f, f, nullptr, at, nullptr) == GDN_OK);
  }
  EXPECT(good > 2000);
}

static void rotary() {
  void* const at = reinterpret_cast<void*>(uintptr_t{0x10000});
  void* const off = reinterpret_cast<void*>(uintptr_t{0x10008});
  int32_t* const i = static_cast<int32_t*>(at);
  double* const d = static_cast<double*>(at);
  int good = 0;
  EXPECT(gdn_rotary(nullptr, at, at, i, d, at, at, nullptr) == GDN_ERR_INVALID_ARGUMENT);
  for (int it = 0; it < 20000; ++it) {
    gdn_rotary_problem p;
    std::memset(&p, 0, sizeof p);
    p.abi_version = draw(0, 30) ? GDN_ABI_VERSION : field(0, 3);
    p.dtype = field(0, 1);
    p.tokens = tokens();
    p.heads_q = field(1, 40);
    p.heads_k = field(0, 40);
    p.width = draw(0, 9) ? 8 * (int32_t)draw(1, 128) : field(0, 2000);
    p.pairs = draw(0, 9) ? (int32_t)draw(1, p.width > 2 ? p.width / 2 : 1) : field(0, 1024);
    p.layout = field(0, 1);
    p.inverse = field(0, 1);
    p.axes = field(1, 4);
    int left = p.pairs;
    for (int a = 0; a < 4; ++a) {
      p.sections[a] = a + 1 < p.axes ? (int32_t)(left > 0 ? draw(0, left) : 0) : a + 1 == p.axes ? left : 0;
      left -= p.sections[a] > left ? 0 : p.sections[a];
    }
    if (draw(0, 20) == 0) p.sections[draw(0, 3)] = field(0, 100);
    p.magnitude = real();
    if (draw(0, 3) == 0) p.q_stride = field(0, 1 << 16);
    if (draw(0, 3) == 0) p.k_out_stride = field(0, 1 << 16);
    if (draw(0, 40) == 0) p.reserved[draw(0, 3)] = 1;
    // a call that would be enqueued is stopped by a pointer
    const gdn_status s = gdn_rotary(&p, off, at, i, d, at, at, nullptr);
    if (s == GDN_OK) {
      EXPECT(p.tokens == 0);
      ++good;
    } else {
      EXPECT(s == GDN_ERR_INVALID_ARGUMENT && message[0]);
      good += std::strstr(message, "16-byte aligned") != nullptr;
    }
  }
  EXPECT(good > 2000);
}

int main() {
  linear();
  rotary();
  if (failures) return 1;
  std::puts("linear host checks passed");
  return 0;
}
