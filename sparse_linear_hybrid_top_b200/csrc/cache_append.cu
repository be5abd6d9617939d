// cache_append.cu -- appending keys and values to the 8-bit block cache, the
// keys turned by the several-axes rotary encoding on the way.
//
// A block of 64 tokens that becomes full is written as e4m3 codes with one
// power-of-two scale per head for its keys and one for its values: the
// smallest 2^e, e >= -100, with max |x| <= 448 * 2^e.  e4m3 is itself a
// floating format, so a power of two costs no precision against max/448 except
// among its subnormals, and code * scale is exact in bf16, which is what the
// attention multiplies.  The rows of the block that stays open are kept in
// bf16, so every token is rounded to 8 bits once, from its bf16 value.
//
// HBM-bound.  CTA (block of the sequence, group of heads, sequence): 256
// threads, four to a row; a thread holds its quarter of the row's keys and
// values in registers, so the block is read once, its two maxima are taken
// over registers, and the codes are written from them.  The next head's rows
// travel while one is encoded, the first one's while the cosines and sines of
// the block's rows are formed: once, in shared memory, for every head of the
// group.
//
// Measured: 4680 tokens of 12 heads, d = 128, 11.7 us (3.7 TB/s: a launch, the
// way from the lengths to the first rows, 64 x 64 float64 angles and one wave of
// CTAs); 4 sequences of up to 3600 tokens, 40 heads, 65.5 us (5.0 TB/s; 77% of
// the copy rate); one token of 16 sequences 4.5 us.
#include <cuda_fp8.h>

#include "cache_index.h"
#include "common.cuh"
#include "operators.h"

namespace salad {
namespace {

constexpr int kThreads = 256;

struct AppendParams {
  CacheView c;
  const int32_t* seq;
  int32_t* seq_out;              // null where a second launch writes it
  const char* k;
  const char* v;
  long long kb, kh, kn, vb, vh, vn;   // bytes
  int N;
  const int32_t* counts;
  int rotate;
  RopeWhere where;
  RopeRates rates;
  int heads_per_cta;
  unsigned* err;
};

// Largest of |x| over a packed pair, as bf16 bit patterns (which order like
// the magnitudes, infinities above every finite value and NaN above those).
__device__ __forceinline__ uint32_t abs_max2(uint32_t m, uint32_t x) {
  return __vmaxu2(m, x & 0x7fff7fffu);
}

// 2^-e and 2^e of a block whose largest magnitude has bf16 bits `top`.
// 448 = 1.75 * 2^8, and 1.75 is mantissa 96 of bf16's 128.
__device__ __forceinline__ void block_scale(uint32_t top, float* inverse, float* scale) {
  if (top >= 0x7f80u) {            // an infinity or a NaN
    *inverse = *scale = __int_as_float(0x7fffffff);
    return;
  }
  int e = static_cast<int>(top >> 7) - 127 - 8 + ((top & 127u) > 96u ? 1 : 0);
  e = e < -100 ? -100 : e;
  *scale = __int_as_float((127 + e) << 23);
  *inverse = __int_as_float((127 - e) << 23);
}

// Eight bf16 values times `inverse` as e4m3 codes.
__device__ __forceinline__ uint2 to_codes(uint4 x, float inverse) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack_bf16x2(w[i]);
    c[i] = __nv_cvt_float2_to_fp8x2(make_float2(f.x * inverse, f.y * inverse), __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

template <int D, bool HALVES>
__global__ void __launch_bounds__(kThreads, 2) append_kernel(const __grid_constant__ AppendParams P) {
  constexpr int CH = D / 32;                     // 16-byte chunks of a row per thread
  __shared__ double turns[D / 2];
  // Cosines and sines of the rows' pairs; a row's pad keeps its neighbour's in
  // other banks.
  __shared__ __align__(16) float2 cs[kCacheBlock][D / 2 + 2];
  __shared__ uint32_t top[2][2][kThreads / 32];  // [parity][K or V][warp]
  const int b = blockIdx.z;
  bool bad = false;
  const CacheSeq s = cache_seq(__ldg(P.seq + 2 * b), __ldg(P.seq + 2 * b + 1), P.c.blocks, &bad);
  const int count = P.counts == nullptr ? P.N : cache_count(__ldg(P.counts + b), P.N, &bad);
  const CacheAppend plan = cache_append_plan(s, count, P.c.blocks, &bad);
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) {
    if (bad) atomicOr(P.err, kErrRange);
    if (P.seq_out != nullptr) {
      P.seq_out[2 * b] = s.len + plan.n;
      P.seq_out[2 * b + 1] = plan.slot_out;
    }
  }
  const int j = plan.first + blockIdx.x;
  if (plan.n == 0 || j > plan.last) return;
  const bool closes = j < plan.last;
  const int row = threadIdx.x / 4, quarter = threadIdx.x % 4;
  const int i = j * kCacheBlock + row - s.len;   // the row's token in this call
  const bool fresh = i >= 0 && i < plan.n;
  if (!closes && (s.len + plan.n) % kCacheBlock == 0) return;   // the open block is empty

  int page = -1;
  if (closes) {
    page = cache_page(__ldg(P.c.page_table + static_cast<long long>(b) * P.c.blocks + j), P.c.pages);
    if (page < 0) {
      if (threadIdx.x == 0) atomicOr(P.err, kErrRange);
      return;
    }
  }
  const int h0 = blockIdx.y * P.heads_per_cta, h1 = min(P.c.H, h0 + P.heads_per_cta);
  // A row that is neither new nor part of a closing block is not touched.
  const bool has = fresh || closes;
  auto load = [&](int h, uint4 (&k)[CH], uint4 (&v)[CH]) {
    const long long old = (((static_cast<long long>(b) * 2 + s.slot) * P.c.H + h) * kCacheBlock + row) * D * 2;
    const char* kp = fresh ? P.k + b * P.kb + h * P.kh + i * P.kn : reinterpret_cast<const char*>(P.c.k_tail) + old;
    const char* vp = fresh ? P.v + b * P.vb + h * P.vh + i * P.vn : reinterpret_cast<const char*>(P.c.v_tail) + old;
#pragma unroll
    for (int x = 0; x < CH; ++x) {
      k[x] = has ? __ldcs(reinterpret_cast<const uint4*>(kp) + quarter + 4 * x) : make_uint4(0, 0, 0, 0);
      v[x] = has ? __ldcs(reinterpret_cast<const uint4*>(vp) + quarter + 4 * x) : make_uint4(0, 0, 0, 0);
    }
  };
  uint4 k_next[CH], v_next[CH];
  load(h0, k_next, v_next);
  if (P.rotate) {
    for (int m = threadIdx.x; m < D / 2; m += kThreads) turns[m] = P.rates.turns[m];
    __syncthreads();
    if (fresh) {
      // Each thread the pairs that it uses itself.
      const int3 pos = rope_position(P.where, b, i, s.len + i);
#pragma unroll 4
      for (int x = 0; x < D / 8; ++x) {
        // Adjacent: chunk quarter + 4 (x / 4) holds pairs 4 chunk ..; halves:
        // the eight pairs of chunk quarter + 4 (x / 8) and the one D/2 on.
        const int m = HALVES ? 8 * (quarter + 4 * (x / 8)) + x % 8 : 4 * (quarter + 4 * (x / 4)) + x % 4;
        const int at = m < P.rates.first1 ? pos.x : (m < P.rates.first2 ? pos.y : pos.z);
        cs[row][m] = rope_cos_sin(turns[m], at);
      }
    }
  }
  for (int h = h0; h < h1; ++h) {
    uint4 k[CH], v[CH];
#pragma unroll
    for (int x = 0; x < CH; ++x) {
      k[x] = k_next[x];
      v[x] = v_next[x];
    }
    if (h + 1 < h1) load(h + 1, k_next, v_next);
    if (P.rotate && fresh) {
      // Four cosines and sines at an address: two 16-byte reads.
      auto pairs = [&](int m, float2 (&c)[4]) {
        const float4 lo = *reinterpret_cast<const float4*>(&cs[row][m]);
        const float4 hi = *reinterpret_cast<const float4*>(&cs[row][m + 2]);
        c[0] = make_float2(lo.x, lo.y);
        c[1] = make_float2(lo.z, lo.w);
        c[2] = make_float2(hi.x, hi.y);
        c[3] = make_float2(hi.z, hi.w);
      };
      if (HALVES) {
#pragma unroll
        for (int x = 0; x < CH / 2; ++x) {
          uint32_t* u = &k[x].x;
          uint32_t* w = &k[x + CH / 2].x;
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            float2 c[4];
            pairs(8 * (quarter + 4 * x) + 4 * y, c);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float2 p = unpack_bf16x2(u[2 * y + e]), q = unpack_bf16x2(w[2 * y + e]);
              const float2 lo = rope_turn(p.x, q.x, c[2 * e]);
              const float2 hi = rope_turn(p.y, q.y, c[2 * e + 1]);
              u[2 * y + e] = pack_bf16x2(lo.x, hi.x);
              w[2 * y + e] = pack_bf16x2(lo.y, hi.y);
            }
          }
        }
      } else {
#pragma unroll
        for (int x = 0; x < CH; ++x) {
          uint32_t* u = &k[x].x;
          float2 c[4];
          pairs(4 * (quarter + 4 * x), c);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 p = unpack_bf16x2(u[e]);
            const float2 r = rope_turn(p.x, p.y, c[e]);
            u[e] = pack_bf16x2(r.x, r.y);
          }
        }
      }
    }
    if (!closes) {
      if (fresh) {
        const long long at =
            (((static_cast<long long>(b) * 2 + plan.slot_out) * P.c.H + h) * kCacheBlock + row) * D * 2;
#pragma unroll
        for (int x = 0; x < CH; ++x) {
          reinterpret_cast<uint4*>(reinterpret_cast<char*>(P.c.k_tail) + at)[quarter + 4 * x] = k[x];
          reinterpret_cast<uint4*>(reinterpret_cast<char*>(P.c.v_tail) + at)[quarter + 4 * x] = v[x];
        }
      }
      continue;
    }
    uint32_t mk = 0, mv = 0;
#pragma unroll
    for (int x = 0; x < CH; ++x) {
      mk = abs_max2(abs_max2(abs_max2(abs_max2(mk, k[x].x), k[x].y), k[x].z), k[x].w);
      mv = abs_max2(abs_max2(abs_max2(abs_max2(mv, v[x].x), v[x].y), v[x].z), v[x].w);
    }
    mk = __reduce_max_sync(0xffffffffu, max(mk & 0xffffu, mk >> 16));
    mv = __reduce_max_sync(0xffffffffu, max(mv & 0xffffu, mv >> 16));
    // One barrier per head: the two parities keep a fast warp's next maxima
    // apart from the ones that a slow warp still reads.
    const int par = h & 1;
    if (threadIdx.x % 32 == 0) {
      top[par][0][threadIdx.x / 32] = mk;
      top[par][1][threadIdx.x / 32] = mv;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      mk = max(mk, top[par][0][w]);
      mv = max(mv, top[par][1][w]);
    }
    float ik, sk, iv, sv;
    block_scale(mk, &ik, &sk);
    block_scale(mv, &iv, &sv);
    const long long at = static_cast<long long>(page) * P.c.H + h;
    if (threadIdx.x == 0) {
      P.c.k_scale[at] = sk;
      P.c.v_scale[at] = sv;
    }
    uint2* kq = reinterpret_cast<uint2*>(P.c.k_pages + (at * kCacheBlock + row) * D);
    uint2* vq = reinterpret_cast<uint2*>(P.c.v_pages + (at * kCacheBlock + row) * D);
#pragma unroll
    for (int x = 0; x < CH; ++x) {
      kq[quarter + 4 * x] = to_codes(k[x], ik);
      vq[quarter + 4 * x] = to_codes(v[x], iv);
    }
  }
}

// seq += counts in place, after the append has read it.
__global__ void advance_kernel(int32_t* seq, const int32_t* counts, int B, int N, int blocks) {
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= B) return;
  bool bad = false;   // reported by the append
  const CacheSeq s = cache_seq(seq[2 * b], seq[2 * b + 1], blocks, &bad);
  const int count = counts == nullptr ? N : cache_count(counts[b], N, &bad);
  const CacheAppend plan = cache_append_plan(s, count, blocks, &bad);
  seq[2 * b] = s.len + plan.n;
  seq[2 * b + 1] = plan.slot_out;
}

}  // namespace

cudaError_t launch_cache_append(const Ctx& c, const CacheAppendArgs& a) {
  AppendParams P;
  P.c = a.cache;
  P.seq = a.seq;
  P.seq_out = a.seq_out == a.seq ? nullptr : a.seq_out;
  P.k = static_cast<const char*>(a.k);
  P.v = static_cast<const char*>(a.v);
  P.kb = a.k_st[0] * 2; P.kh = a.k_st[1] * 2; P.kn = a.k_st[2] * 2;
  P.vb = a.v_st[0] * 2; P.vh = a.v_st[1] * 2; P.vn = a.v_st[2] * 2;
  P.N = a.N;
  P.counts = a.counts;
  P.rotate = a.rotate;
  P.where = a.where;
  if (a.rotate) P.rates = rope_rates(a.split, a.base);
  else P.rates = RopeRates{};
  P.err = c.err;
  // Blocks that N tokens can touch.
  const int span = (a.N + kCacheBlock - 1) / kCacheBlock + 1;
  // Heads of a CTA, which share its angles: up to eight (so that CTAs behind a
  // padded batch's counts, which end at once, do not leave others a second turn:
  // 4 x 40 heads x 3600 padded tokens take 66 us with eight and 72 with
  // twelve), as many as cost least where a CTA takes 1.5 heads' time to begin,
  // two are on an SM, and the last ones leave half a turn unused (7800 tokens of
  // 12 heads: 21.4 us in 3 groups, a turn and a quarter, 18.3 in 2; 512
  // tokens of 8 heads, 16 sequences: 18.3 in 3, 14.2 in 2).
  const double touched = ((a.N - 1) / static_cast<double>(kCacheBlock) + 1.0) * a.cache.B;
  int per = 1;
  double least = 0.0;
  for (int n = 1; n <= 8 && n <= a.cache.H; ++n) {
    const double turns = touched * ((a.cache.H + n - 1) / n) / (2.0 * c.num_sms);
    const double cost = (turns <= 1.02 ? 1.0 : turns + 0.5) * (n + 1.5);
    if (n == 1 || cost < least) {
      per = n;
      least = cost;
    }
  }
  P.heads_per_cta = per;
  const dim3 grid(span, static_cast<unsigned>((a.cache.H + per - 1) / per), a.cache.B);
  const bool halves = a.pairing == 1;
  if (a.cache.d == 128) {
    if (halves) append_kernel<128, true><<<grid, kThreads, 0, c.stream>>>(P);
    else append_kernel<128, false><<<grid, kThreads, 0, c.stream>>>(P);
  } else {
    if (halves) append_kernel<64, true><<<grid, kThreads, 0, c.stream>>>(P);
    else append_kernel<64, false><<<grid, kThreads, 0, c.stream>>>(P);
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.seq_out != a.seq) return e;
  advance_kernel<<<(a.cache.B + 127) / 128, 128, 0, c.stream>>>(a.seq_out, a.counts, a.cache.B, a.N,
                                                                a.cache.blocks);
  return cudaGetLastError();
}

}  // namespace salad
