// cache_attn.cuh -- what the two attention kernels over the 8-bit block cache
// share: e4m3 codes as bf16 pairs, and the parameters.
#pragma once

#include "cache_index.h"
#include "common.cuh"
#include "internal.h"

namespace salad {

struct CacheAttnParams {
  CacheView c;
  const int32_t* seq;
  const char* q;
  char* o;
  long long qb, qh, qn, ob, oh, on;   // bytes
  float* lse;
  int Hq, group, N;                   // group = Hq / H query heads to a key head
  const int32_t* counts;
  int frame, window;
  float scale_log2;                   // softmax scale * log2(e)
  int tiles;                          // row tiles of one (sequence, key head)
  int splits;
  float* part_o;                      // [splits][B * H * tiles * rows][d]
  float2* part_ml;                    // [splits][B * H * tiles * rows]
  unsigned* err;
  unsigned long long wait_ns;
};

// Four e4m3 codes as two bf16 pairs: even = (byte 0, byte 2), odd = (byte 1,
// byte 3).  A code's seven magnitude bits, put at bit 4 of a bf16, are its
// value times 2^-120 for normals and subnormals alike (the exponent biases
// are 7 and 127), so one exact multiplication by 2^120 finishes it.  The code
// of NaN comes out as 480: a block that holds one has a NaN scale.
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void e4m3_pairs(uint32_t w, uint32_t& even, uint32_t& odd) {
  constexpr uint32_t kMag = 0x07f007f0u, kSign = 0x80008000u, k2p120 = 0x7b807b80u;
  even = mul_bf16x2(((w << 4) & kMag) | ((w << 8) & kSign), k2p120);
  odd = mul_bf16x2(((w >> 4) & kMag) | (w & kSign), k2p120);
}

__device__ __forceinline__ float ex2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// log2 and reciprocal of a power of two (exponent bits only).
__device__ __forceinline__ float pow2_log(float s) {
  return static_cast<float>(static_cast<int>((__float_as_uint(s) >> 23) & 255u) - 127);
}
__device__ __forceinline__ float pow2_inv(float s) {
  return __uint_as_float((254u << 23) - (__float_as_uint(s) & 0x7f800000u));
}

// What a query row sees, and where it is.  Row r of a (sequence, key head) is
// query token r / group under query head h * group + r % group.
struct CacheRow {
  int n, head;
  bool valid;
  CacheSpan see;
};
__device__ __forceinline__ CacheRow cache_row(const CacheAttnParams& P, int r, int h, int len, int count) {
  CacheRow x;
  x.n = r / P.group;
  x.head = h * P.group + r % P.group;
  x.valid = x.n < count;
  x.see = x.valid ? cache_visible(len - count + x.n, len, count, P.frame, P.window) : CacheSpan{0, 0};
  if (x.see.lo >= x.see.end) x.see = CacheSpan{0, 0};
  return x;
}

size_t cache_attn_tc_ws_bytes(const CacheAttnArgs& a, int num_sms);
cudaError_t launch_cache_attn_tc(const Ctx& c, const CacheAttnArgs& a, CacheAttnParams P);

}  // namespace salad
