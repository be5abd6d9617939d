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

// (cos, sin) of 2 pi * pos * turns.  The product and the reduction to
// [-1/2, 1/2] turns are float64: |pos| < 2^31 and rates below 1/(2 pi) leave an
// error under 2^-25 turns at the farthest position and under 2^-44 within
// 4096.  The reduced turn is rounded to float32 once (2^-25 of a turn at
// most), where sincospif is accurate to an ulp.
__device__ __forceinline__ float2 rope_cos_sin(double turns, int pos) {
  const double a = static_cast<double>(pos) * turns;
  const float r = static_cast<float>(2.0 * (a - rint(a)));
  float sn, cs;
  sincospif(r, &sn, &cs);
  return make_float2(cs, sn);
}

// The rotated pair.  Products and sums are rounded one by one (no fused
// multiply-add), so that every caller gets the same bits for a token.
__device__ __forceinline__ float2 rope_turn(float u, float w, float2 cs) {
  return make_float2(__fsub_rn(__fmul_rn(u, cs.x), __fmul_rn(w, cs.y)),
                     __fadd_rn(__fmul_rn(u, cs.y), __fmul_rn(w, cs.x)));
}
#endif

}  // namespace salad
