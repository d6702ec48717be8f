// The angle of a pair of channels, shared by the kernels that rotate.
#pragma once

#include "common.cuh"

namespace favor {

// Sine and cosine of a pair's angle.  The position times the pair's fraction of
// a turn per unit, in 64-bit fixed point, wraps to the exact fraction of a
// turn, of which the upper 32 bits are kept.  The nearest quarter turn is taken
// off exactly, in whole numbers; what is left, z in [-pi/4, pi/4], goes into
// the Taylor series of sin (to z^9) and cos (to z^10), whose remainders there
// are below 2e-9 and 2e-10, and the quarters turn the two.
__device__ __forceinline__ void sine_cosine(int32_t pos, uint64_t per_unit, float* sn, float* cs) {
  const uint64_t turn = static_cast<uint64_t>(static_cast<int64_t>(pos)) * per_unit;
  const uint32_t u = static_cast<uint32_t>(turn >> 32);
  const uint32_t quarter = (u + (1u << 29)) >> 30;
  const float z = static_cast<float>(static_cast<int32_t>(u - (quarter << 30))) * (6.283185307179586f * 0x1p-32f);
  const float z2 = z * z;
  float s = 1.f / 362880;
  s = fmaf(s, z2, -1.f / 5040);
  s = fmaf(s, z2, 1.f / 120);
  s = fmaf(s, z2, -1.f / 6);
  s = fmaf(s * z2, z, z);
  float c = -1.f / 3628800;
  c = fmaf(c, z2, 1.f / 40320);
  c = fmaf(c, z2, -1.f / 720);
  c = fmaf(c, z2, 1.f / 24);
  c = fmaf(c, z2, -0.5f);
  c = fmaf(c, z2, 1.f);
  const bool odd = quarter & 1;
  const float a = odd ? c : s, b = odd ? s : c;
  *sn = __uint_as_float(__float_as_uint(a) ^ ((quarter & 2) << 30));
  *cs = __uint_as_float(__float_as_uint(b) ^ (((quarter + 1) & 2) << 30));
}

}  // namespace favor
