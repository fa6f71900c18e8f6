// angles.cuh -- the rotary embedding's cosines and sines, in fp64.
#pragma once

#include <cuda_runtime.h>
#include <math.h>

namespace rglru {

// base^(-2j/d) = 2^(-j log2(base) / 128) for d = 256, with log2(base) in two parts, the first short enough that its
// product with j is exact: within 2 units of the last place of the power itself, at a fifth of the fp64
// operations of pow.
struct RopeBase {
    double hi, lo;                     // log2(base)
};
__device__ __forceinline__ void rope_cos_sin(RopeBase base, int j, double p, double& c, double& s) {
    const double x = exp2(base.hi * (-j / 128.0));
    sincos(p * fma(x, base.lo * (-j / 128.0) * 0.69314718055994530942, x), &s, &c);
}
inline RopeBase rope_base(float base) {
    const long double l = log2l((long double)base);
    RopeBase b;
    b.hi = (double)(float)l;           // 24 bits
    b.lo = (double)(l - (long double)b.hi);
    return b;
}

}  // namespace rglru
