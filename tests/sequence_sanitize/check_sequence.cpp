// Host-only check of the sequence operators' C ABI under AddressSanitizer and
// UndefinedBehaviorSanitizer: every call below fails, sizes or has no work, so
// there is no HIP call (no GPU needed).  Built and run by
// tests/test_sequence_sanitize.py; exits non-zero on a mismatch.
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "gdn_common.h"
#include "gdn_seq.h"

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

static void sequences() {
  void* const at = reinterpret_cast<void*>(uintptr_t{0x10000});
  float* const f = static_cast<float*>(at);
  int32_t* const i = static_cast<int32_t*>(at);
  size_t a = 0, b = 0;
  EXPECT(gdn_packed_workspace_size(nullptr, 0, &a) == GDN_ERR_INVALID_ARGUMENT && message[0]);
  for (int it = 0; it < 20000; ++it) {
    gdn_seq_problem p;
    std::memset(&p, 0, sizeof p);
    p.abi_version = draw(0, 30) ? GDN_ABI_VERSION : field(0, 3);
    p.heads_k = field(1, 8);
    p.heads_v = draw(0, 9) ? (int32_t)(p.heads_k % 100000LL * draw(1, 4)) : field(1, 8);
    p.d_k = 16 * (int32_t)draw(0, 9);
    p.d_v = 16 * (int32_t)draw(0, 9);
    p.qkv_dtype = (int32_t)draw(0, 9) ? (draw(0, 1) ? GDN_BF16 : GDN_F32) : field(0, 3);
    p.out_dtype = draw(0, 1) ? GDN_BF16 : GDN_F32;
    p.state_rows = field(0, 100);
    p.tokens = draw(0, 9) ? draw(0, 1 << 20) : draw(0, 1) ? (1LL << 31) - 256 : (int64_t)field(0, 9) * (int64_t{1} << draw(0, 30));
    p.sequences = field(0, 1000);
    if (!draw(0, 5)) p.q_stride = field(0, 1 << 24);
    if (!draw(0, 5)) p.v_stride = (int64_t)field(0, 1 << 20) * 8;
    const gdn_status s = gdn_packed_workspace_size(&p, 0, &a);
    EXPECT(s == GDN_OK || (s == GDN_ERR_INVALID_ARGUMENT && message[0]));
    EXPECT(gdn_packed_workspace_size(&p, 1, &b) == s);
    // each call below lacks something or has nothing to do
    if (p.tokens > 0) {
      EXPECT(gdn_decode(&p, at, at, at, f, f, nullptr, nullptr, at, nullptr) == GDN_ERR_INVALID_ARGUMENT);
      if (s == GDN_OK) EXPECT(gdn_decode(&p, at, at, at, f, f, (float*)((char*)at + 4), nullptr, at, nullptr) == GDN_ERR_INVALID_ARGUMENT);
    }
    if (s != GDN_OK) continue;
    EXPECT(b >= a && a < (size_t{1} << 62));
    const gdn_status none = p.sequences == 0 ? GDN_OK : GDN_ERR_WORKSPACE_TOO_SMALL;
    if (p.sequences == 0 || a > 0) {
      EXPECT(gdn_packed_forward(&p, at, at, at, f, f, i, nullptr, f, at, f, nullptr, 0, nullptr) == none);
      EXPECT(gdn_packed_forward(&p, at, at, at, f, f, i, nullptr, f, at, f, at, a ? a - 1 : 0, nullptr) == none);
      EXPECT(gdn_packed_backward(&p, at, at, at, f, f, i, f, at, f, at, at, at, f, f, f, at, b ? b - 1 : 0, nullptr) == none);
    }
    if (p.sequences > 0) {
      EXPECT(gdn_packed_forward(&p, at, at, at, f, f, nullptr, nullptr, f, at, f, at, a, nullptr) == GDN_ERR_INVALID_ARGUMENT);
      EXPECT(gdn_packed_backward(&p, at, at, at, f, f, i, f, at, f, at, (char*)at + 8, at, f, f, f, at, b, nullptr) ==
             GDN_ERR_INVALID_ARGUMENT);
    }
    // more tokens never need less
    gdn_seq_problem q = p;
    q.tokens = p.tokens / 2;
    size_t less = 0;
    EXPECT(gdn_packed_workspace_size(&q, 0, &less) == GDN_OK && less <= a);
  }
}

static void norms() {
  void* const at = reinterpret_cast<void*>(uintptr_t{0x10000});
  float* const f = static_cast<float*>(at);
  size_t a = 0, b = 0;
  EXPECT(gdn_group_norm_workspace_size(nullptr, 0, &a) == GDN_ERR_INVALID_ARGUMENT && message[0]);
  for (int it = 0; it < 20000; ++it) {
    gdn_norm_problem p;
    std::memset(&p, 0, sizeof p);
    p.abi_version = GDN_ABI_VERSION;
    p.dtype = draw(0, 1) ? GDN_BF16 : GDN_F32;
    p.batch = draw(0, 9) ? draw(0, 300) : (int64_t)field(0, 9) * (int64_t{1} << draw(0, 30));
    p.spatial = draw(0, 1) ? 1 : field(1, 5000);
    p.groups = field(1, 64);
    p.channels = draw(0, 9) ? (int32_t)((int64_t)p.groups * draw(1, 300) % (1 << 25)) : field(1, 1 << 24);
    p.activation = field(GDN_ACT_NONE, GDN_ACT_RELU);
    p.center = (int32_t)draw(0, 1);
    p.eps = draw(0, 30) ? 1e-5f : std::nanf("");
    const gdn_status s = gdn_group_norm_workspace_size(&p, 0, &a);
    EXPECT(s == GDN_OK || (s == GDN_ERR_INVALID_ARGUMENT && message[0]));
    EXPECT(gdn_group_norm_workspace_size(&p, 1, &b) == s);
    if (s != GDN_OK) {
      EXPECT(gdn_group_norm(&p, at, f, f, at, at, f, f, at, SIZE_MAX, nullptr) == GDN_ERR_INVALID_ARGUMENT);
      continue;
    }
    EXPECT(a < (size_t{1} << 62) && b < (size_t{1} << 62));
    if (p.batch == 0) {
      EXPECT(gdn_group_norm(&p, at, f, f, at, at, f, f, at, 0, nullptr) == GDN_OK);
      EXPECT(gdn_group_norm_backward(&p, at, at, f, f, nullptr, f, f, at, nullptr, nullptr, nullptr, at, 0, nullptr) == GDN_OK);
      continue;
    }
    EXPECT(gdn_group_norm(&p, at, f, f, at, at, f, nullptr, at, SIZE_MAX, nullptr) == GDN_ERR_INVALID_ARGUMENT);
    EXPECT(gdn_group_norm(&p, (char*)at + 2, f, f, at, at, f, f, at, SIZE_MAX, nullptr) == GDN_ERR_INVALID_ARGUMENT);
    EXPECT(gdn_group_norm_backward(&p, at, at, f, f, at, f, f, at, f, f, nullptr, at, SIZE_MAX, nullptr) == GDN_ERR_INVALID_ARGUMENT);
    if (a > 0) EXPECT(gdn_group_norm(&p, at, f, f, at, at, f, f, at, a - 1, nullptr) == GDN_ERR_WORKSPACE_TOO_SMALL);
    if (b > 0)
      EXPECT(gdn_group_norm_backward(&p, at, at, f, f, nullptr, f, f, at, f, f, nullptr, at, b - 1, nullptr) ==
             GDN_ERR_WORKSPACE_TOO_SMALL);
  }
}

int main() {
  sequences();
  norms();
  if (failures) return 1;
  std::printf("sequence host checks passed\n");
  return 0;
}
