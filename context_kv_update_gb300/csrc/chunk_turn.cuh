// chunk_turn.cuh -- the rotary angles of a ragged chunk's stores.
//
// Pair j of a head turns by the angle p * f_j, kept in turns as 64-bit fixed point:
// (p * round(f_j / (2 pi) * 2^64)) mod 2^64.  One integer product reduces it exactly, whatever
// the position, where a float product would lose the low bits; its top 32 bits go to sincospi.
#pragma once

#include <cmath>
#include <cstring>

#include "dflash_internal.cuh"

namespace dflash {

struct TurnFreqs {
  uint64_t f[kMaxHeadDim / 2];  // turns per position, 2^64 to a turn
};

// cos and sin (times the magnitude) of position p at f turns per position.
__device__ __forceinline__ float2 turn_cos_sin(int p, uint64_t f, float mag) {
  const uint64_t t = static_cast<uint64_t>(static_cast<uint32_t>(p)) * f;
  float s, c;  // top 32 bits: a signed fraction of half a turn in units of 2^-31
  sincospif(static_cast<float>(static_cast<int32_t>(t >> 32)) * 0x1p-31f, &s, &c);
  return make_float2(c * mag, s * mag);
}

// Turns per position of every pair, and the factor on cos and sin.
inline void fill_turn_freqs(TurnFreqs *tf, float *mag, const dflash_rope_spec &r, int rot,
                            double theta) {
  const double two_pi = 6.283185307179586476925286766559;
  double j0 = 0.0, j1 = 0.0;
  *mag = 1.f;
  if (r.scaling == DFLASH_ROPE_YARN) {
    const double per = rot / (2.0 * std::log(theta));
    j0 = std::fmax(std::floor(per * std::log(r.trained_ctx / (two_pi * r.beta_fast))), 0.0);
    j1 = std::fmin(std::ceil(per * std::log(r.trained_ctx / (two_pi * r.beta_slow))), rot - 1.0);
    *mag = static_cast<float>(r.magnitude > 0.0 ? r.magnitude : 0.1 * std::log(r.factor) + 1.0);
  }
  for (int j = 0; j < rot / 2; ++j) {
    double f = std::pow(theta, -2.0 * j / rot);
    if (r.scaling == DFLASH_ROPE_LINEAR) f /= r.factor;
    if (r.scaling == DFLASH_ROPE_YARN) {
      const double u = std::fmin(std::fmax((j - j0) / std::fmax(j1 - j0, 1e-3), 0.0), 1.0);
      f = f / r.factor * u + f * (1.0 - u);
    }
    const double turns = f / two_pi;
    // the fraction of a turn; 2^64 times it is an integer below 2^64 (a
    // double's 53 bits)
    tf->f[j] = static_cast<uint64_t>(std::ldexp(turns - std::floor(turns), 64));
  }
}

struct TurnTable {
  dflash_rope_spec spec;
  double theta;
  float mag;
  TurnFreqs tf;
};
// (The powers of a 128-wide head take the host ~5 us: the calling thread's last table is
// kept with the specification it was made from.)
inline const TurnTable &turn_table(const dflash_rope_spec &rope, double theta) {
  static thread_local TurnTable last = {};  // rot_dim 0: made from nothing yet
  if (std::memcmp(&last.spec, &rope, sizeof(rope)) != 0 || last.theta != theta) {
    last.spec = rope;
    last.theta = theta;
    fill_turn_freqs(&last.tf, &last.mag, rope, rope.rot_dim, theta);
  }
  return last;
}

}  // namespace dflash
