// Rotary positions: the angle of a far position, exactly enough, without 64-bit
// trigonometry.
//
// Pair j of a head is turned by the angle p w_j (position p, w_j radians a position).
// With f = frac(w_j / 2 pi) as a 64-bit fixed-point number F = f 2^64, the turn's
// fraction is the wrapped integer product p F mod 2^64: whole turns fall off the top
// by themselves and what stays is p w_j 2^-52 radians (the roundings of 1 / (2 pi) and of
// its product with w_j, each 2^-53 of w_j / 2 pi turns a position) at any 32-bit position,
// negative ones included.  Its upper 32 bits as a signed number are half turns in [-1, 1), which
// sincospif takes in fp32: 2^-25 of a turn at most, 2e-7 radians.  An fp32 product p w_j would be off by p w_j 2^-24: 0.06
// radians at position 2^20.
#pragma once

#include <cstdint>

namespace da {

struct RopeParams {
  const double* inv_freq;  // [rot / 2]; null: no rotation
  int offset, rot;         // the rotated elements [offset, offset + rot) of a head
  int interleaved;         // pairs (2j, 2j + 1), else (j, j + rot / 2)
  float magnitude;         // multiplies cosine and sine
  float sin_sign;          // -1: the transposed rotation (the gradient)
};

// F of w radians a position.
__device__ __forceinline__ unsigned long long rope_turn_step(double w) {
  double f = w * 0.15915494309189533577;  // 1 / (2 pi)
  f -= floor(f);
  return (unsigned long long)(f * 18446744073709551616.0);
}

// (cosine, sine) of position p, times the magnitude.
__device__ __forceinline__ float2 rope_cos_sin(unsigned long long step, int p, const RopeParams& r) {
  const unsigned long long turn = step * (unsigned long long)(long long)p;
  float s, c;
  sincospif((float)(int)(turn >> 32) * 4.656612873077393e-10f, &s, &c);  // 2^-31
  return make_float2(c * r.magnitude, s * r.magnitude * r.sin_sign);
}

}  // namespace da
