// rope.cuh -- device code shared by the kernels that turn rows by their tokens' positions
// (rope.cu, norm_rope.cu).
//
// Angles: theta_i is held as a 64-bit fraction of a turn, f_i = 2^64 theta_i / 2 pi.
// m * f_i mod 2^64 is then the angle of position m reduced to one turn -- exactly,
// for every int32 m of either sign -- and its top 32 bits, as a signed fraction of
// half a turn, go to sincospi.  theta_i carries the 2^-53 of double precision, so
// the reduced angle of m = 2^24 is off by under 2^-30 turns; made a float, of 24 bits, it is
// rounded by up to 2^-26 turns at any m, about 10^-7 of what turns.
#pragma once

#include <stdint.h>

namespace apex {
namespace {

// (cos, sin) of the angle of position m at `turn` = theta / 2 pi in 64-bit fractions;
// sign: +1, or -1 for the inverse rotation
__device__ __forceinline__ void turn_angle(uint64_t turn, int m, float sign, float &c, float &s)
{
    const int32_t top = (int32_t)(((uint64_t)(int64_t)m * turn) >> 32);
    sincospif((float)top * 0x1p-31f, &s, &c);
    s *= sign;
}

__device__ __forceinline__ void rotate2(float x, float y, float c, float s, float &u, float &w)
{
    u = fmaf(x, c, -y * s);
    w = fmaf(x, s, y * c);
}

}  // namespace
}  // namespace apex
