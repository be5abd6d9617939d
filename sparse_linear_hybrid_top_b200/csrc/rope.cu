// rope.cu -- rotary positions with several axes on queries and keys.
//
// y_u = x_u cos a - x_w sin a, y_w = x_u sin a + x_w cos a with a = position *
// rate for every channel pair (u, w): the 3-D encoding of "SALAD ...
// (paper.rainbus.top)" 方法步骤详情 step 3 for the tensors that enter the sparse
// branch.  The backward pass is the same with -a.
//
// HBM-bound: every element is read and written once, three operations each.
// The angles depend on the token alone, so a thread owns 16 channels of one
// token (8 pairs), keeps their 8 cosines and sines in registers and walks
// over the heads of q and of k with four heads' loads in flight: the float64
// reduction and the sine are paid once per token and pair, not per head.  Where
// tokens are few, the heads are spread over more CTAs instead (grid.y).
// A thread's channels are 8 from the row's first half and the 8 across from
// them in the second, which holds whole pairs under both pairings; a warp
// reads 512 contiguous bytes per load at d = 128 in 16-bit types.
//
// Measured: q and k of 31200 tokens, 12 heads, d = 128 in bf16 60.9 us (6.3
// TB/s, 96% of the copy rate); gradients of 100800 tokens, 40 heads, 314 us (as
// fast as a copy); eight single tokens of 40 heads 3.3 us; float32 gradients of
// 3 x 4097 tokens, 12 heads of 64, q and k, 30.3 us (5.0 TB/s; the launch and
// the ramps of a short kernel).
#include <cmath>
#include <cuda_fp16.h>

#include "common.cuh"
#include "operators.h"
#include "rope.cuh"

namespace salad {
namespace {

constexpr int kThreads = 256;

struct Side {
  const char* x;
  char* y;
  long long xb, xh, xn, yb, yh, yn;   // bytes
  int H;
};

struct RopeParams {
  Side s[2];
  int B, N, d;
  int heads_per_cta;
  RopeWhere where;
  RopeRates rates;
  float sign;
};

// Eight consecutive elements as float.
template <typename T>
struct Vec8;
template <>
struct Vec8<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const char* p) { v = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = unpack_bf16x2(w[i]);
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    }
  }
  static __device__ __forceinline__ void store(char* p, const float (&f)[8]) {
    __stcs(reinterpret_cast<uint4*>(p),
           make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7])));
  }
};
template <>
struct Vec8<__half> {
  uint4 v;
  __device__ __forceinline__ void load(const char* p) { v = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    }
  }
  static __device__ __forceinline__ void store(char* p, const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
  }
};
template <>
struct Vec8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const char* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  static __device__ __forceinline__ void store(char* p, const float (&f)[8]) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(f[0], f[1], f[2], f[3]));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(f[4], f[5], f[6], f[7]));
  }
};

template <typename T, bool HALVES>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams P) {
  __shared__ double turns[kMaxRopePairs];
  for (int i = threadIdx.x; i < P.d / 2; i += kThreads) turns[i] = P.rates.turns[i];
  __syncthreads();
  const int per_row = P.d / 16;                    // threads per token
  const int rows = kThreads / per_row;             // tokens per CTA
  const int row = threadIdx.x / per_row, c = threadIdx.x % per_row;
  const long long t = static_cast<long long>(blockIdx.x) * rows + row;
  if (row >= rows || t >= static_cast<long long>(P.B) * P.N) return;
  const int b = static_cast<int>(t / P.N), n = static_cast<int>(t % P.N);
  const int3 pos = rope_position(P.where, b, n, P.where.offset + n);
  float2 cs[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // Adjacent pairs: four in each of the thread's two chunks.  Halves: the
    // eight pairs across the chunks.
    const int m = HALVES ? 8 * c + i : (i < 4 ? 4 * c + i : P.d / 4 + 4 * c + i - 4);
    const int at = m < P.rates.first1 ? pos.x : (m < P.rates.first2 ? pos.y : pos.z);
    cs[i] = rope_cos_sin(turns[m], at);
    cs[i].y *= P.sign;
  }
  const long long col = static_cast<long long>(c) * 8 * sizeof(T);
  const long long half = static_cast<long long>(P.d) / 2 * sizeof(T);
  const int lo = blockIdx.y * P.heads_per_cta;
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    const Side& s = P.s[side];
    const int first = side == 0 ? lo : lo - P.s[0].H;
    const int h0 = first > 0 ? first : 0;
    const int h1 = min(s.H, first + P.heads_per_cta);
    const char* x = s.x + b * s.xb + n * s.xn + col;
    char* y = s.y + b * s.yb + n * s.yn + col;
    for (int h = h0; h < h1; h += 4) {
      Vec8<T> u[4], w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (h + i < h1) {
          u[i].load(x + (h + i) * s.xh);
          w[i].load(x + (h + i) * s.xh + half);
        }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (h + i < h1) {
          float f[8], g[8];
          u[i].get(f);
          w[i].get(g);
          if (HALVES) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float2 r = rope_turn(f[e], g[e], cs[e]);
              f[e] = r.x;
              g[e] = r.y;
            }
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 r = rope_turn(f[2 * e], f[2 * e + 1], cs[e]);
              f[2 * e] = r.x;
              f[2 * e + 1] = r.y;
              const float2 q = rope_turn(g[2 * e], g[2 * e + 1], cs[4 + e]);
              g[2 * e] = q.x;
              g[2 * e + 1] = q.y;
            }
          }
          Vec8<T>::store(y + (h + i) * s.yh, f);
          Vec8<T>::store(y + (h + i) * s.yh + half, g);
        }
    }
  }
}

template <typename T>
void launch_t(const Ctx& c, const RopeParams& P, bool halves, dim3 grid) {
  if (halves) rope_kernel<T, true><<<grid, kThreads, 0, c.stream>>>(P);
  else rope_kernel<T, false><<<grid, kThreads, 0, c.stream>>>(P);
}

}  // namespace

const RopeRates& rope_rates(const int (&split)[3], float base) {
  // The last table of this thread: up to 128 calls of pow() would cost a
  // single-token call more than its kernel.
  thread_local RopeRates r;
  thread_local int of[3] = {-1, -1, -1};
  thread_local float of_base = 0.0f;
  if (of[0] == split[0] && of[1] == split[1] && of[2] == split[2] && of_base == base) return r;
  int m = 0;
  for (int axis = 0; axis < 3; ++axis) {
    if (axis == 1) r.first1 = m;
    if (axis == 2) r.first2 = m;
    for (int i = 0; i < split[axis] / 2; ++i)
      r.turns[m++] = std::pow(static_cast<double>(base), -2.0 * i / split[axis]) / 6.283185307179586;
  }
  for (; m < kMaxRopePairs; ++m) r.turns[m] = 0.0;
  for (int axis = 0; axis < 3; ++axis) of[axis] = split[axis];
  of_base = base;
  return r;
}

cudaError_t launch_rope(const Ctx& c, const RopeArgs& a) {
  RopeParams P;
  const int size = a.dtype == 2 ? 4 : 2;
  auto side = [&](Side& s, const void* x, void* y, const long long (&xs)[3], const long long (&ys)[3],
                  int H) {
    s.x = static_cast<const char*>(x);
    s.y = static_cast<char*>(y);
    s.xb = xs[0] * size; s.xh = xs[1] * size; s.xn = xs[2] * size;
    s.yb = ys[0] * size; s.yh = ys[1] * size; s.yn = ys[2] * size;
    s.H = H;
  };
  side(P.s[0], a.q, a.q_out, a.q_st, a.qo_st, a.Hq);
  side(P.s[1], a.k, a.k_out, a.k_st, a.ko_st, a.Hk);
  P.B = a.B;
  P.N = a.N;
  P.d = a.d;
  P.where = a.where;
  P.rates = rope_rates(a.split, a.base);
  P.sign = a.inverse ? -1.0f : 1.0f;
  const int rows = kThreads / (a.d / 16);
  const long long ctas = (static_cast<long long>(a.B) * a.N + rows - 1) / rows;
  // Every head in one CTA where the tokens alone give each SM eight CTAs;
  // otherwise the heads are split until they do (or four are left, the
  // loads that one thread keeps in flight).
  const int heads = a.Hq + a.Hk;
  const long long want = 8ll * c.num_sms;
  long long parts = (want + ctas - 1) / ctas;
  const long long most = (heads + 3) / 4;
  if (parts > most) parts = most;
  P.heads_per_cta = static_cast<int>((heads + parts - 1) / parts);
  const dim3 grid(static_cast<unsigned>(ctas),
                  static_cast<unsigned>((heads + P.heads_per_cta - 1) / P.heads_per_cta));
  const bool halves = a.pairing == 1;
  if (a.dtype == 0) launch_t<__nv_bfloat16>(c, P, halves, grid);
  else if (a.dtype == 1) launch_t<__half>(c, P, halves, grid);
  else launch_t<float>(c, P, halves, grid);
  return cudaGetLastError();
}

}  // namespace salad
