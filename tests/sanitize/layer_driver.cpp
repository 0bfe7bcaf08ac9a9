// layer_driver.cpp -- drives the layer operators' host-side validation over
// many shapes and row strides, extreme values included, in a build under
// AddressSanitizer and UndefinedBehaviorSanitizer (test infrastructure).  Every
// call carries one argument that must be rejected; the workspace queries and
// the statuses must agree on a shape's validity.
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
  const int64_t extreme[] = {INT64_MIN, -(int64_t(1) << 40), -1, 0, 1, 3, 15, 17, 255, 257, 4097, 65535, 65536,
                             int64_t(1) << 24, int64_t(1) << 31, int64_t(1) << 40, int64_t(1) << 62, INT64_MAX};
  const int64_t sane[5] = {1, 2, 4, 16, 64};
  auto pick = [&]() {
    const uint64_t r = next_u64();
    return (r & 3) == 0 ? extreme[(r >> 3) % (sizeof(extreme) / sizeof(extreme[0]))] : sane[(r >> 3) % 5];
  };
  void* F = reinterpret_cast<void*>(uintptr_t(0x100000));
  float* f = static_cast<float*>(F);
  int32_t* q = static_cast<int32_t*>(F);
  const ssd_dtype BAD = static_cast<ssd_dtype>(99);
  long nvalid = 0;
  for (long it = 0; it < iters; ++it) {
    ssd_conv_shape c = {pick(), pick(), pick(), pick()};
    const bool cv = ssd_causal_conv_backward_workspace_bytes(&c) > 0;
    const int64_t row = pick();
    int st = ssd_causal_conv(&c, F, row, f, f, SSD_BF16, 1, F, q, nullptr, F, 0, nullptr, nullptr, nullptr);
    EXPECT(st == (cv ? SSD_ERR_NULL : st) && st != SSD_OK, "conv without y");
    st = ssd_causal_conv(&c, F, row, f, f, BAD, 1, F, q, F, F, 0, nullptr, nullptr, nullptr);
    EXPECT(cv ? st == SSD_ERR_DTYPE : st == SSD_ERR_SHAPE || st == SSD_ERR_UNSUPPORTED, "conv dtype");
    st = ssd_causal_conv(&c, F, row, f, f, SSD_F32, 1, F, q, F, F, -1, nullptr, nullptr, nullptr);
    EXPECT(st == SSD_ERR_SHAPE || st == SSD_ERR_UNSUPPORTED, "conv nseq");
    st = ssd_causal_conv_backward(&c, F, row, f, f, SSD_F32, 1, F, q, F, F, F, pick(), f, f, F, F, 0, nullptr);
    EXPECT(st == SSD_ERR_SHAPE || st == SSD_ERR_UNSUPPORTED || st == SSD_ERR_WORKSPACE, "conv backward workspace");
    st = ssd_causal_conv_step(&c, F, row, F, f, f, SSD_F32, 1, F, nullptr, nullptr);
    EXPECT(st != SSD_OK && st != SSD_ERR_HIP, "conv step without y");

    ssd_scan_shape s = {pick(), pick(), pick(), pick(), pick()};
    const ssd_scan_rows r = {pick(), pick(), pick(), pick(), pick()};
    const bool sv = ssd_selective_scan_workspace_bytes(&s) > 0;
    nvalid += sv + cv;
    EXPECT((ssd_selective_scan_backward_workspace_bytes(&s) > 0) == sv, "scan queries disagree");
    st = ssd_selective_scan(&s, &r, F, F, f, F, F, f, F, f, 1, BAD, f, q, F, f, 0, nullptr, nullptr, F, SIZE_MAX, nullptr);
    EXPECT(sv ? st == SSD_ERR_DTYPE : st == SSD_ERR_SHAPE || st == SSD_ERR_UNSUPPORTED, "scan dtype");
    st = ssd_selective_scan(&s, &r, F, F, f, F, F, f, F, f, 1, SSD_BF16, f, q, nullptr, f, 0, nullptr, nullptr, F,
                            SIZE_MAX, nullptr);
    EXPECT(st != SSD_OK && st != SSD_ERR_HIP, "scan without y");
    st = ssd_selective_scan(&s, nullptr, F, F, f, F, F, f, F, f, 1, SSD_F32, f, q, F, f, 0, nullptr, nullptr, F, 0,
                            nullptr);
    EXPECT(sv ? st == SSD_ERR_WORKSPACE : st == SSD_ERR_SHAPE || st == SSD_ERR_UNSUPPORTED, "scan workspace");
    st = ssd_selective_step(&s, &r, F, F, f, F, F, f, F, f, 1, SSD_F32, f, f, nullptr, nullptr);
    EXPECT(st != SSD_OK && st != SSD_ERR_HIP, "scan step without y");
    st = ssd_selective_scan_backward(&s, &r, F, F, f, F, F, f, F, f, 1, SSD_F32, f, q, F, f, &r, F, F, f, F, F, f, F, f,
                                     f, F, 0, nullptr);
    EXPECT(st != SSD_OK && st != SSD_ERR_HIP, "scan backward without workspace");

    const int64_t rows = pick(), dim = pick();
    st = ssd_layer_norm(rows, dim, F, SSD_BF16, F, SSD_F32, f, f, 1e-5f, 0, F, nullptr, f, f, nullptr);
    EXPECT(st == SSD_ERR_SHAPE || st == SSD_ERR_UNSUPPORTED || st == SSD_ERR_NULL, "norm without the sum's place");
    st = ssd_layer_norm_backward(rows, dim, F, SSD_BF16, F, SSD_F32, f, f, f, 0, F, F, F, f, f, F, 0, nullptr);
    EXPECT(st == SSD_ERR_SHAPE || st == SSD_ERR_UNSUPPORTED || st == SSD_ERR_WORKSPACE, "norm backward workspace");
  }
  std::printf("%ld iterations, %ld valid shapes, %d mismatches\n", iters, nvalid, g_fail);
  return g_fail ? 1 : 0;
}
