// rope.cuh -- the several-axes rotary encoding shared by the rotation of
// queries and keys (rope.cu) and the cache's append (cache_append.cu): the
// channel pairs' axes and rates, and one pair's cosine and sine.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace salad {

constexpr int kMaxRopePairs = 128;

// Axis and rate of every channel pair.  Rates are in turns (angle / 2 pi) per
// unit of position, so that whole turns drop out exactly in float64.
struct RopeRates {
  double turns[kMaxRopePairs];
  int first1, first2;          // first pair of axis 1, of axis 2
};

// Where the tokens stand: a position tensor, or the latent grid.
struct RopeWhere {
  const int32_t* positions;    // [N,3] or [B,N,3], or null
  long long batch_stride;      // 3 N, or 0 where the samples share positions
  int Hh, Wh, offset;
};

const RopeRates& rope_rates(const int (&split)[3], float base);

#ifdef __CUDACC__
// (f, y, x) of token n of sample b; p: its place on the grid.
__device__ __forceinline__ int3 rope_position(const RopeWhere& w, int b, int n, int p) {
  if (w.positions != nullptr) {
    const int32_t* at = w.positions + b * w.batch_stride + 3ll * n;
    return make_int3(__ldg(at), __ldg(at + 1), __ldg(at + 2));
  }
  const int line = p / w.Wh;
  return make_int3(line / w.Hh, line % w.Hh, p - line * w.Wh);
}

// (cos, sin) of 2 pi * pos * turns, float64 rounded once to float32.
// |pos| < 2^31 and rates of at most 1/(2 pi) keep the product below 2^29
// turns, so adding and taking off 1.5 * 2^52 rounds it to whole turns and to
// quarters exactly.  What is left, z in [-pi/4, pi/4], goes into the Taylor
// polynomials of sine and cosine through z^13 and z^14, whose next terms are
// below 2^-45.  22 float64 operations per token and pair, shared by all heads:
// the bits do not depend on a fast sine's error, and a key lands on the same
// 8-bit code as one that is turned in float64.
__device__ __forceinline__ float2 rope_cos_sin(double turns, int pos) {
  constexpr double kWhole = 6755399441055744.0;   // 1.5 * 2^52
  const double a = static_cast<double>(pos) * turns;
  const double t = a - ((a + kWhole) - kWhole);
  const double fourth = t * 4.0 + kWhole;
  const int quadrant = __double2loint(fourth);
  const double z = (t - (fourth - kWhole) * 0.25) * 6.283185307179586;
  const double z2 = z * z;
  double s = 1.0 / 6227020800.0;
  s = fma(s, z2, -1.0 / 39916800.0);
  s = fma(s, z2, 1.0 / 362880.0);
  s = fma(s, z2, -1.0 / 5040.0);
  s = fma(s, z2, 1.0 / 120.0);
  s = fma(s, z2, -1.0 / 6.0);
  s = fma(s * z2, z, z);
  double c = -1.0 / 87178291200.0;
  c = fma(c, z2, 1.0 / 479001600.0);
  c = fma(c, z2, -1.0 / 3628800.0);
  c = fma(c, z2, 1.0 / 40320.0);
  c = fma(c, z2, -1.0 / 720.0);
  c = fma(c, z2, 1.0 / 24.0);
  c = fma(c, z2, -0.5);
  c = fma(c, z2, 1.0);
  const float fs = static_cast<float>(s), fc = static_cast<float>(c);
  // Quarter turns: (cos, sin) -> (-sin, cos) each.
  const float x = quadrant & 1 ? -fs : fc, y = quadrant & 1 ? fc : fs;
  return quadrant & 2 ? make_float2(-x, -y) : make_float2(x, y);
}

// The rotated pair.  Products and sums are rounded one by one (no fused
// multiply-add), so that every caller gets the same bits for a token.
__device__ __forceinline__ float2 rope_turn(float u, float w, float2 cs) {
  return make_float2(__fsub_rn(__fmul_rn(u, cs.x), __fmul_rn(w, cs.y)),
                     __fadd_rn(__fmul_rn(u, cs.y), __fmul_rn(w, cs.x)));
}
#endif

}  // namespace salad
