// cache_attn.cuh -- what the two attention kernels over the 8-bit block cache
// share: e4m3 codes as fp16 pairs, and the parameters.
#pragma once

#include <cuda_fp16.h>

#include "cache_index.h"
#include "common.cuh"
#include "operators.h"

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
  float* part_o;                      // means of parts of rows, for the merging launch
  float2* part_ml;                    // their maxima and sums
  int2* plan;                         // [B], first CTA of a sequence's parts, and how many
  unsigned* err;
  unsigned long long wait_ns;
};

// Two e4m3 codes as fp16 (exact).
__device__ __forceinline__ uint32_t e4m3_to_f16x2(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<unsigned short>(codes)));
  return r;
}
__device__ __forceinline__ uint4 eight_codes(uint2 c) {
  return make_uint4(e4m3_to_f16x2(c.x), e4m3_to_f16x2(c.x >> 16), e4m3_to_f16x2(c.y), e4m3_to_f16x2(c.y >> 16));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// bf16 pairs times a power of two as fp16.
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t x, float factor) {
  const float2 f = unpack_bf16x2(x);
  return pack_f16x2(f.x * factor, f.y * factor);
}
__device__ __forceinline__ uint4 scaled_f16(uint4 x, float factor) {
  return make_uint4(bf16x2_to_f16x2(x.x, factor), bf16x2_to_f16x2(x.y, factor), bf16x2_to_f16x2(x.z, factor),
                    bf16x2_to_f16x2(x.w, factor));
}

__device__ __forceinline__ uint32_t finite_or_zero(uint32_t pair) {
  if ((pair & 0x7f80u) == 0x7f80u) pair &= 0xffff0000u;
  if ((pair & 0x7f800000u) == 0x7f800000u) pair &= 0xffffu;
  return pair;
}

// mbar_wait with the timer read every 64 polls only: reading it costs hundreds
// of cycles, which a wait inside a short dependency chain feels.
__device__ __forceinline__ bool mbar_wait_poll(uint32_t bar, uint32_t parity, uint64_t limit_ns,
                                               volatile int* abort) {
  uint64_t t0 = 0;
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if (abort != nullptr && *abort) return false;
    if ((i & 63u) == 0) {
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      else if (now - t0 > limit_ns) return false;
    }
  }
}

// The same without suspending between polls: for one thread whose wake-up
// is on the critical path.
__device__ __forceinline__ bool mbar_wait_spin(uint32_t bar, uint32_t parity, uint64_t limit_ns,
                                               volatile int* abort) {
  uint64_t t0 = 0;
  for (uint32_t i = 1;; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return true;
    if ((i & 255u) == 0) {
      if (abort != nullptr && *abort) return false;
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      else if (now - t0 > limit_ns) return false;
    }
  }
}

// idesc_bf16 with fp16 A and B.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool a_mn_major, bool b_mn_major) {
  return idesc_bf16(M, N, a_mn_major, b_mn_major) & ~((1u << 7) | (1u << 10));
}

// Untiled bulk copy global -> shared completing on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

__device__ __forceinline__ float ex2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 1 / x of a sum of weights, 0 for a row that has none.
__device__ __forceinline__ float weight_inv(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return x == 0.0f ? 0.0f : y;
}

// log2 and reciprocal of a power of two (exponent bits only).
__device__ __forceinline__ float pow2_log(float s) {
  return static_cast<float>(static_cast<int>((__float_as_uint(s) >> 23) & 255u) - 127);
}
__device__ __forceinline__ float pow2_inv(float s) {
  return __uint_as_float((254u << 23) - (__float_as_uint(s) & 0x7f800000u));
}

// P is held in fp16 times a power of two, 2^kTopP at the most: below 2^-14
// fp16 has a fixed step of 2^-24, and the weights that a long row has many of may
// be that small beside its largest.
constexpr float kTopP = 15.0f;

// The weight of a part of a row: its sum (of 2^(s - x)) against a maximum of
// `top`.  A part that saw no key (its sum is 0) counts for nothing; one whose sum
// is NaN does.
__device__ __forceinline__ float part_weight(float2 part, float top) {
  if (part.y == 0.0f) return 0.0f;
  return part.x == -INFINITY ? part.y : part.y * ex2_ftz(part.x - top);
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
