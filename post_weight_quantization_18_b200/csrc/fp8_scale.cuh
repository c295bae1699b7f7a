// fp8_scale.cuh — the scale of an e4m3 block from its largest magnitude. Host-and-device code, run
// on the CPU over every fp32 mantissa by the tests.
#pragma once

#include <math.h>

#include "hd.cuh"

namespace gptq {

// fl(a / 448) for finite a >= 0 with a / 448 >= 2^-126: Markstein's correction of a product with the
// rounded reciprocal (P. Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990). The remainder a - 448 q is exact, and the corrected quotient is
// the correctly rounded one. Three multiply-adds and no branch, where the general division made a
// third of the quantizers' instructions.
GPTQ_HD float div_e4m3_max(float a) {
  const float r = 1.f / 448.f;
  const float q = a * r;
  return fmaf(fmaf(-448.f, q, a), r, q);
}

}  // namespace gptq
