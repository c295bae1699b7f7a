// The division by 448 of the quantizers (fp8_scale.cuh) against the IEEE division, on the CPU: every
// fp32 mantissa, at the exponents given. Prints the number of differences.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "fp8_scale.cuh"

int main(int argc, char** argv) {
  long bad = 0;
  for (int i = 1; i < argc; ++i) {
    const uint32_t e = (uint32_t)(atoi(argv[i]) + 127) << 23;
    for (uint32_t m = 0; m < (1u << 23); ++m) {
      const uint32_t b = e | m;
      float a;
      memcpy(&a, &b, 4);
      volatile float want = a / 448.f;
      const float got = gptq::div_e4m3_max(a);
      bad += got != want;
    }
  }
  printf("%ld\n", bad);
  return 0;
}
