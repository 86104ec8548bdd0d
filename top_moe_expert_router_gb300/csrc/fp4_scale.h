// fp4_scale.h — the quotient that an NVFP4 block's scale is rounded from; plain
// C++, so that it is tested on the host too.
#pragma once

#include <math.h>

#ifdef __CUDACC__
#define MOE_HD __host__ __device__ __forceinline__
#else
#define MOE_HD inline
#endif

namespace moe {

// t / 6 for t with no more than 11 significant bits (of 16-bit values, a power of two aside): near enough that E4M3
// rounds it as it does the exact quotient. The product is exact wherever that is the middle between two E4M3 values
// (checked for all of them), and elsewhere further from it than the product's error.
MOE_HD float fp4_sixth_of_short(float t) { return t * (1.f / 6.f); }

// t / 6 to nearest, for any t whose sixth is a normal number: the product, and what 6 times it lacks of t, which is a
// float. (fp32's 1/6 is the nearest float and the product within a unit in the last place of the quotient, so that the
// corrected sum rounds as the quotient does; checked for all mantissas.) The nearest float is never a middle that the
// quotient is not: t misses 6 times a middle by at least a unit of its own last place, a sixth of which is more than
// half a unit of the quotient's. The product alone meets 19/16 for t one unit below 57/8, and the scale is then a step
// too large.
MOE_HD float fp4_sixth(float t) {
    const float q = t * (1.f / 6.f);
    return fmaf(fmaf(-6.f, q, t), 1.f / 6.f, q);
}

}  // namespace moe
