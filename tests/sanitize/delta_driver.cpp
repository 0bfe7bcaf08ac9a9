// delta_driver.cpp -- drives the host-side validation of the delta rule, the
// group norm and 8-bit storage over many shapes and row strides, extreme values
// included, in a build under AddressSanitizer and UndefinedBehaviorSanitizer
// (test infrastructure).  Every call carries one argument that must be
// rejected; the workspace queries and the statuses must agree on a shape.
#include <cstdint>
#include <cstdio>
#include <cstdlib>

#include "ssd.h"

static uint64_t g_state = 0x9E3779B97F4A7C15ull;
static uint64_t next_u64() {  // splitmix64
  uint64_t z = (g_state += 0x9E3779B97F4A7C15ull);
  z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
  z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
  return z ^ (z >> 31);
}

static int g_fail = 0;
#define EXPECT(cond, what)                                     \
  do {                                                         \
    if (!(cond)) {                                             \
      std::fprintf(stderr, "line %d: %s\n", __LINE__, what);   \
      if (++g_fail > 20) std::exit(1);                         \
    }                                                          \
  } while (0)

int main(int argc, char** argv) {
  const long iters = argc > 1 ? std::atol(argv[1]) : 100000;
  const int64_t extreme[] = {INT64_MIN, -(int64_t(1) << 40), -1, 0, 1, 3, 15, 17, 255, 257, 4097, 65536,
                             int64_t(1) << 24, int64_t(1) << 31, int64_t(1) << 40, int64_t(1) << 62, INT64_MAX};
  const int64_t sane[5] = {1, 2, 16, 32, 64};
  auto pick = [&]() {
    const uint64_t r = next_u64();
    return (r & 7) == 0 ? extreme[(r >> 3) % (sizeof(extreme) / sizeof(extreme[0]))] : sane[(r >> 3) % 5];
  };
  void* F = reinterpret_cast<void*>(uintptr_t(0x100000));
  float* f = static_cast<float*>(F);
  int8_t* b = static_cast<int8_t*>(F);
  const int32_t* q = static_cast<int32_t*>(F);
  const ssd_dtype BAD = static_cast<ssd_dtype>(99);
  long nvalid = 0;
  for (long it = 0; it < iters; ++it) {
    const ssd_delta_shape s = {pick(), pick(), pick(), pick(), pick(), pick()};
    const ssd_delta_rows r = {pick(), pick(), pick(), pick(), pick()};
    const bool ok = ssd_delta_rule_workspace_bytes(&s) > 0;
    EXPECT(ok == (ssd_delta_rule_backward_workspace_bytes(&s) > 0), "queries agree");
    nvalid += ok;
    int st = ssd_delta_rule(&s, &r, F, F, F, F, F, f, f, 7, 1.f, BAD, f, q, F, f, 0, nullptr, nullptr, F, SIZE_MAX, nullptr);
    EXPECT(ok ? st == SSD_ERR_DTYPE : st == SSD_ERR_SHAPE || st == SSD_ERR_UNSUPPORTED, "delta dtype");
    st = ssd_delta_rule(&s, &r, F, F, F, F, F, f, f, 7, 1.f, SSD_BF16, f, q, nullptr, f, 0, nullptr, nullptr, F, SIZE_MAX,
                        nullptr);
    EXPECT(st != SSD_OK && st != SSD_ERR_HIP, "delta without y");
    st = ssd_delta_rule(&s, nullptr, F, F, F, F, F, f, f, 7, 1.f, SSD_F32, f, q, F, f, 0, nullptr, nullptr, F, 0, nullptr);
    EXPECT(ok ? st == SSD_ERR_WORKSPACE || st == SSD_ERR_UNSUPPORTED : st == SSD_ERR_SHAPE || st == SSD_ERR_UNSUPPORTED,
           "delta workspace");
    st = ssd_delta_rule_backward(&s, &r, F, F, F, F, F, f, f, 7, 1.f, SSD_F32, f, q, F, f, &r, F, F, F, F, F, nullptr, f, f,
                                 F, SIZE_MAX, nullptr);
    EXPECT(st != SSD_OK && st != SSD_ERR_HIP, "delta backward without dA");
    st = ssd_delta_step(&s, &r, F, F, F, F, F, f, f, 7, 1.f, SSD_F32, f, nullptr, F, nullptr);
    EXPECT(st != SSD_OK && st != SSD_ERR_HIP, "delta step without a state");

    const int64_t rows = pick(), dim = pick(), groups = pick();
    const bool gv = ssd_group_norm_backward_workspace_bytes(rows, dim, groups) > 0;
    nvalid += gv;
    st = ssd_group_norm(rows, dim, groups, F, SSD_BF16, F, pick(), f, f, 1e-5f, 1, nullptr, nullptr, f, nullptr);
    EXPECT(gv ? st == SSD_ERR_NULL : st == SSD_ERR_SHAPE || st == SSD_ERR_UNSUPPORTED, "group norm without y");
    st = ssd_group_norm_backward(rows, dim, groups, F, SSD_BF16, F, F, F, pick(), F, f, f, f, f, 0, F, F, pick(), f, f, F, 0,
                                 nullptr);
    EXPECT(st != SSD_OK && st != SSD_ERR_HIP, "group norm backward workspace");
    st = ssd_pack8(rows, dim, F, pick(), SSD_BF16, b, nullptr, nullptr);
    EXPECT(st != SSD_OK && st != SSD_ERR_HIP, "pack without scales");
    st = ssd_unpack8(rows, dim, nullptr, F, F, pick(), SSD_F32, nullptr);
    EXPECT(st != SSD_OK && st != SSD_ERR_HIP, "unpack without values");
  }
  std::printf("%ld shapes, %ld valid, %d mismatches\n", iters, nvalid, g_fail);
  return g_fail != 0;
}
