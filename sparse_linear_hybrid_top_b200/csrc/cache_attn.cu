// cache_attn.cu -- attention of few query rows over the 8-bit block cache:
// o = softmax(scale q k^T + M) v for single tokens and short chunks.
//
// Memory-bound: a query token reads every key and value of its sequence once,
// 2 d bytes a token and head.  So the keys are split over as many warps as
// fill the GPU, and every warp streams its own part from global memory to
// registers with no shared-memory stage and no barrier in its loop: while one
// half page (32 keys) is multiplied, the loads of the next one's keys and of
// its own values are in flight (8 KB a warp at d = 128).  The products are
// 16-row mma.sync tiles (query heads of a key head, and query tokens, fill
// the rows); with so few rows the tensor pipe is far from its limit and
// tcgen05's 128-row tiles would be mostly empty.
//
// Both contractions are reordered so that a lane's 16-byte loads are its MMA
// fragments.  QK: a lane holds 16 (32) consecutive channels of one key; MMA
// step i multiplies channels {4i, 4i+2 | 4i+1, 4i+3} of each lane's run, and
// the query fragments in shared memory are laid out the same way.  PV: a lane
// holds 16 consecutive channels of four keys; column tile j is channels = j
// mod 16, so lane group t ends with channels [32t, 32t+32) of its rows.
//
// Keys are multiplied as code values: their page's scale joins the softmax
// scale.  Values too: a page's scale, a power of two, is added to the exponent
// of its P (exact), and taken off the row sum again.  P is rounded to bf16
// (half a step, 2^-8 of each weight); maxima, sums and O are float32.
//
// Partial results of the splits are merged by a second kernel, launched only
// where there is more than one split.
#include "cache_attn.cuh"

namespace salad {
namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t part(const uint4& v, int i) {
  return i == 0 ? v.x : (i == 1 ? v.y : (i == 2 ? v.z : v.w));
}

// A lane's run of V codes: 16 bytes at d = 128, 8 at d = 64.
template <int D>
struct Run;
template <>
struct Run<128> {
  uint4 v;
  __device__ __forceinline__ void load(const unsigned char* p) { v = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ uint32_t word(int i) const { return part(v, i); }
};
template <>
struct Run<64> {
  uint2 v;
  __device__ __forceinline__ void load(const unsigned char* p) { v = __ldg(reinterpret_cast<const uint2*>(p)); }
  __device__ __forceinline__ uint32_t word(int i) const { return i == 0 ? v.x : v.y; }
};

__device__ __forceinline__ uint32_t finite_or_zero(uint32_t pair) {
  if ((pair & 0x7f80u) == 0x7f80u) pair &= 0xffff0000u;
  if ((pair & 0x7f800000u) == 0x7f800000u) pair &= 0xffffu;
  return pair;
}

// RW: warps over row tiles of 16; the other warps of the CTA split the keys.
template <int D, int RW>
__global__ void __launch_bounds__(kThreads) cache_attn_kernel(const __grid_constant__ CacheAttnParams P) {
  constexpr int KW = 4 / RW;           // warps over the keys
  constexpr int KS = D / 16;           // MMA steps of QK
  constexpr int NT = D / 8;            // column tiles of O
  __shared__ uint4 qs[RW][KS][32];
  __shared__ float os[KW > 1 ? RW : 1][KW > 1 ? KW : 1][16][D + 4];
  __shared__ float2 mls[RW][KW][16];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane / 4, t = lane % 4;
  const int rt = warp % RW, kw = warp / RW;
  const int tile = blockIdx.x / P.splits, split = blockIdx.x % P.splits;
  const int b = blockIdx.y / P.c.H, h = blockIdx.y % P.c.H;
  bool bad = false;
  const CacheSeq s = cache_seq(__ldg(P.seq + 2 * b), __ldg(P.seq + 2 * b + 1), P.c.blocks, &bad);
  const int count = P.counts == nullptr ? P.N : cache_count(__ldg(P.counts + b), P.N, &bad);
  if (bad && threadIdx.x == 0) atomicOr(P.err, kErrRange);
  if (tile * RW * 16 >= count * P.group) return;      // no row of this tile exists

  // Query fragments: entry (tile, step, lane) is the lane's A operand.
  for (int e = threadIdx.x; e < RW * KS * 32; e += kThreads) {
    const int l = e % 32, ks = (e / 32) % KS, w = e / (32 * KS);
    const int c0 = (l % 4) * 16 + (ks % 4) * 4 + (ks / 4) * 64;
    uint2 x[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = (tile * RW + w) * 16 + l / 4 + 8 * i;
      const int n = r / P.group;
      x[i] = make_uint2(0u, 0u);
      if (n < count)
        x[i] = *reinterpret_cast<const uint2*>(P.q + b * P.qb + (h * P.group + r % P.group) * P.qh + n * P.qn + 2 * c0);
    }
    qs[w][ks][l] = make_uint4(__byte_perm(x[0].x, x[0].y, 0x5410), __byte_perm(x[1].x, x[1].y, 0x5410),
                              __byte_perm(x[0].x, x[0].y, 0x7632), __byte_perm(x[1].x, x[1].y, 0x7632));
  }
  __syncthreads();

  const int r0 = (tile * RW + rt) * 16;
  const CacheRow row[2] = {cache_row(P, r0 + g, h, s.len, count), cache_row(P, r0 + g + 8, h, s.len, count)};
  // Keys that any row of the tile sees, and keys that every row sees.
  int lo = 0x7fffffff, end = 0, all_lo = 0, all_end = 0x7fffffff;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (row[i].see.end > 0) lo = min(lo, row[i].see.lo);
    end = max(end, row[i].see.end);
    if (row[i].valid) {
      all_lo = max(all_lo, row[i].see.lo);
      all_end = min(all_end, row[i].see.end);
    }
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  end = __reduce_max_sync(0xffffffffu, end);
  all_lo = __reduce_max_sync(0xffffffffu, all_lo);
  all_end = __reduce_min_sync(0xffffffffu, all_end);

  float o[NT][4];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) o[j][i] = 0.0f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
  bool vbad[2] = {false, false};

  // This warp's half pages [u0, u1) of the tile's [lo, end).
  int u0 = 0, u1 = 0;
  if (end > 0) {
    const int h0 = lo / 32, nh = (end + 31) / 32 - h0;
    const int u = split * KW + kw, U = P.splits * KW;
    u0 = h0 + static_cast<int>(static_cast<long long>(nh) * u / U);
    u1 = h0 + static_cast<int>(static_cast<long long>(nh) * (u + 1) / U);
  }
  const int closed = 2 * (s.len / kCacheBlock);       // half pages of closed blocks

  // One half page's softmax on S, the products of q with the code values: x =
  // S * c2 in the base-2 domain; P, times 2^ev, back in sc.
  auto softmax = [&](float (&sc)[4][4], int kbase, float c2, float ev, float inv_v, bool none) {
    const bool partial = none || kbase < all_lo || kbase + 32 > all_end;
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sc[i][e] *= c2;
        if (partial) {
          const int key = kbase + 8 * i + 2 * t + (e & 1);
          const CacheSpan& v = row[e >> 1].see;
          if (none || key < v.lo || key >= v.end) sc[i][e] = -INFINITY;
        }
        top[e >> 1] = fmaxf(top[e >> 1], sc[i][e]);
      }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
      top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
    }
    float f[2], nm[2];
    bool grow = false;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float mn = fmaxf(m[i], top[i]);
      grow = grow || mn > m[i];
      f[i] = m[i] == -INFINITY ? 0.0f : ex2_ftz(m[i] - mn);
      m[i] = mn;
      // A row that has seen no key keeps m = -inf: exp2(-inf - 0) = 0.
      nm[i] = mn == -INFINITY ? 0.0f : ev - mn;
    }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int i = 0; i < 2; ++i) l[i] *= f[i];
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][e] *= f[e >> 1];
    }
    float sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sc[i][e] = ex2_ftz(sc[i][e] + nm[e >> 1]);
        sum[e >> 1] += sc[i][e];
      }
#pragma unroll
    for (int i = 0; i < 2; ++i) l[i] = fmaf(sum[i], inv_v, l[i]);
  };

  // ---- closed blocks
  const int uc = min(u1, closed);
  const unsigned char* kp = nullptr;
  uint4 kr[4][D / 64];
  Run<D> vr[2][4];
  const int32_t* table = P.c.page_table + static_cast<long long>(b) * P.c.blocks;
  int entry = u0 < uc ? __ldg(table + u0 / 2) : 0;
  long long slab = 0;                  // page * H + head
  float ks = 0.0f, vs = 0.0f;
  bool none = false;
  auto load_keys = [&](int u, int e) {
    const int page = cache_page(e, P.c.pages);
    none = page < 0;
    slab = static_cast<long long>(none ? 0 : page) * P.c.H + h;
    kp = P.c.k_pages + (slab * kCacheBlock + (u & 1) * 32 + g) * D + t * 16;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int x = 0; x < D / 64; ++x) kr[i][x] = __ldg(reinterpret_cast<const uint4*>(kp + i * 8 * D + 64 * x));
    ks = __ldg(P.c.k_scale + slab);
    vs = __ldg(P.c.v_scale + slab);
  };
  if (u0 < uc) load_keys(u0, entry);
  for (int u = u0; u < uc; ++u) {
    const int next = u + 1 < uc ? __ldg(table + (u + 1) / 2) : 0;
    const unsigned char* vp = P.c.v_pages + (slab * kCacheBlock + (u & 1) * 32 + 2 * t) * D + g * (D / 8);
#pragma unroll
    for (int st = 0; st < 2; ++st)
#pragma unroll
      for (int i = 0; i < 4; ++i) vr[st][i].load(vp + (16 * st + (i & 1) + 8 * (i >> 1)) * D);
    float sc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[i][e] = 0.0f;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const uint4 a = qs[rt][k][lane];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t b0, b1;
        e4m3_pairs(part(kr[i][k / 4], k % 4), b0, b1);
        mma_bf16(sc[i], a.x, a.y, a.z, a.w, b0, b1);
      }
    }
    const float c2 = P.scale_log2 * ks;
    const bool v_nan = isnan(vs);
    const float ev = v_nan ? 0.0f : pow2_log(vs), inv_v = v_nan ? 1.0f : pow2_inv(vs);
    const bool skip = none;
    if (skip && lane == 0) atomicOr(P.err, kErrRange);
    if (v_nan && !skip) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        vbad[i] = vbad[i] || (max(row[i].see.lo, 32 * u) < min(row[i].see.end, 32 * u + 32));
    }
    if (u + 1 < uc) load_keys(u + 1, next);
    softmax(sc, 32 * u, c2, ev, inv_v, skip);
#pragma unroll
    for (int st = 0; st < 2; ++st) {
      const uint32_t a0 = pack_bf16x2(sc[2 * st][0], sc[2 * st][1]), a1 = pack_bf16x2(sc[2 * st][2], sc[2 * st][3]);
      const uint32_t a2 = pack_bf16x2(sc[2 * st + 1][0], sc[2 * st + 1][1]);
      const uint32_t a3 = pack_bf16x2(sc[2 * st + 1][2], sc[2 * st + 1][3]);
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
        uint32_t lo0, lo1, hi0, hi1, lo2, lo3, hi2, hi3;
        e4m3_pairs(__byte_perm(vr[st][0].word(w), vr[st][1].word(w), 0x5410), lo0, lo1);
        e4m3_pairs(__byte_perm(vr[st][0].word(w), vr[st][1].word(w), 0x7632), lo2, lo3);
        e4m3_pairs(__byte_perm(vr[st][2].word(w), vr[st][3].word(w), 0x5410), hi0, hi1);
        e4m3_pairs(__byte_perm(vr[st][2].word(w), vr[st][3].word(w), 0x7632), hi2, hi3);
        mma_bf16(o[4 * w], a0, a1, a2, a3, lo0, hi0);
        mma_bf16(o[4 * w + 1], a0, a1, a2, a3, lo1, hi1);
        mma_bf16(o[4 * w + 2], a0, a1, a2, a3, lo2, hi2);
        mma_bf16(o[4 * w + 3], a0, a1, a2, a3, lo3, hi3);
      }
    }
  }

  // ---- the open block, in bf16 (at most two half pages of one warp)
  for (int u = max(u0, closed); u < u1; ++u) {
    const long long at = (((static_cast<long long>(b) * 2 + s.slot) * P.c.H + h) * kCacheBlock + (u & 1) * 32) * D;
    const __nv_bfloat16* kt = static_cast<const __nv_bfloat16*>(P.c.k_tail) + at;
    const __nv_bfloat16* vt = static_cast<const __nv_bfloat16*>(P.c.v_tail) + at;
    float sc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[i][e] = 0.0f;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const uint4 a = qs[rt][k][lane];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint2 x = *reinterpret_cast<const uint2*>(kt + (8 * i + g) * D + t * 16 + (k % 4) * 4 + (k / 4) * 64);
        mma_bf16(sc[i], a.x, a.y, a.z, a.w, __byte_perm(x.x, x.y, 0x5410), __byte_perm(x.x, x.y, 0x7632));
      }
    }
    softmax(sc, 32 * u, P.scale_log2, 0.0f, 1.0f, false);
    bool odd = false;                  // a value that is not finite
#pragma unroll
    for (int st = 0; st < 2; ++st) {
      const uint32_t a0 = pack_bf16x2(sc[2 * st][0], sc[2 * st][1]), a1 = pack_bf16x2(sc[2 * st][2], sc[2 * st][3]);
      const uint32_t a2 = pack_bf16x2(sc[2 * st + 1][0], sc[2 * st + 1][1]);
      const uint32_t a3 = pack_bf16x2(sc[2 * st + 1][2], sc[2 * st + 1][3]);
#pragma unroll
      for (int w = 0; w < D / 16; ++w) {
        uint32_t x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t y = *reinterpret_cast<const uint32_t*>(
              vt + (16 * st + 2 * t + (i & 1) + 8 * (i >> 1)) * D + g * (D / 8) + 2 * w);
          x[i] = finite_or_zero(y);
          odd = odd || x[i] != y;
        }
        mma_bf16(o[2 * w], a0, a1, a2, a3, __byte_perm(x[0], x[1], 0x5410), __byte_perm(x[2], x[3], 0x5410));
        mma_bf16(o[2 * w + 1], a0, a1, a2, a3, __byte_perm(x[0], x[1], 0x7632), __byte_perm(x[2], x[3], 0x7632));
      }
    }
    // Infinities and NaN reach only the rows that see their key (they would
    // spread as 0 * inf through the product).
    if (__any_sync(0xffffffffu, odd)) {
      for (int key = 0; key < 32; ++key) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float v = __bfloat162float(vt[key * D + (D / 4) * t + (D / 8) * (e & 1) + j]);
            const CacheSpan& see = row[e >> 1].see;
            if (!isfinite(v) && 32 * u + key >= see.lo && 32 * u + key < see.end) o[j][e] += v;
          }
      }
    }
  }

#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    if (vbad[i]) {
#pragma unroll
      for (int j = 0; j < NT; ++j) o[j][2 * i] = o[j][2 * i + 1] = __int_as_float(0x7fffffff);
    }
  }

  // ---- merge the CTA's key warps, then write the rows (or their part)
  const long long rows = static_cast<long long>(gridDim.y) * P.tiles * (RW * 16);
  auto put = [&](int r, const float* acc, float mm, float ll, int c0, int nc) {
    // acc: nc channels from c0 of row r of this tile, unnormalised.
    const CacheRow x = cache_row(P, tile * RW * 16 + r, h, s.len, count);
    if (!x.valid) return;
    if (P.splits > 1) {
      const long long at = (static_cast<long long>(split) * rows) +
                           (static_cast<long long>(blockIdx.y) * P.tiles + tile) * (RW * 16) + r;
      if (c0 == 0) P.part_ml[at] = make_float2(mm, ll);
      float* to = P.part_o + at * D + c0;
#pragma unroll
      for (int c = 0; c < nc; c += 4)
        *reinterpret_cast<float4*>(to + c) = make_float4(acc[c], acc[c + 1], acc[c + 2], acc[c + 3]);
      return;
    }
    const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
    char* to = P.o + b * P.ob + x.head * P.oh + x.n * P.on + 2 * c0;
#pragma unroll
    for (int c = 0; c < nc; c += 8)
      *reinterpret_cast<uint4*>(to + 2 * c) =
          make_uint4(pack_bf16x2(acc[c] * inv, acc[c + 1] * inv), pack_bf16x2(acc[c + 2] * inv, acc[c + 3] * inv),
                     pack_bf16x2(acc[c + 4] * inv, acc[c + 5] * inv), pack_bf16x2(acc[c + 6] * inv, acc[c + 7] * inv));
    if (c0 == 0 && P.lse != nullptr)
      P.lse[(static_cast<long long>(b) * P.Hq + x.head) * P.N + x.n] = (mm + log2f(ll)) * 0.6931471805599453f;
  };
  if constexpr (KW == 1) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float acc[D / 4];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        acc[j] = o[j][2 * i];
        acc[NT + j] = o[j][2 * i + 1];
      }
      put(rt * 16 + g + 8 * i, acc, m[i], l[i], t * (D / 4), D / 4);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int j = 0; j < NT; j += 4) {
        *reinterpret_cast<float4*>(&os[rt][kw][g + 8 * i][t * (D / 4) + j]) =
            make_float4(o[j][2 * i], o[j + 1][2 * i], o[j + 2][2 * i], o[j + 3][2 * i]);
        *reinterpret_cast<float4*>(&os[rt][kw][g + 8 * i][t * (D / 4) + NT + j]) =
            make_float4(o[j][2 * i + 1], o[j + 1][2 * i + 1], o[j + 2][2 * i + 1], o[j + 3][2 * i + 1]);
      }
      if (t == 0) mls[rt][kw][g + 8 * i] = make_float2(m[i], l[i]);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < RW * 16 * (D / 8); e += kThreads) {
      const int r = e / (D / 8), c0 = e % (D / 8) * 8;
      const int w = r / 16, rr = r % 16;
      float mm = -INFINITY, ll = 0.0f, acc[8] = {};
#pragma unroll
      for (int k = 0; k < KW; ++k) mm = fmaxf(mm, mls[w][k][rr].x);
#pragma unroll
      for (int k = 0; k < KW; ++k) {
        const float2 p = mls[w][k][rr];
        // A part that saw no key (its sum is 0) counts for nothing; one whose
        // sum is NaN does.
        if (p.y == 0.0f) continue;
        const float f = p.x == -INFINITY ? 1.0f : ex2_ftz(p.x - mm);
        ll = fmaf(p.y, f, ll);
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[c] = fmaf(os[w][k][rr][c0 + c], f, acc[c]);
      }
      put(r, acc, mm, ll, c0, 8);
    }
  }
}

// Merges the splits of every row: a warp per row.
template <int D>
__global__ void __launch_bounds__(kThreads) cache_merge_kernel(const __grid_constant__ CacheAttnParams P, int rows_per_tile) {
  const int lane = threadIdx.x % 32;
  const int per = P.tiles * rows_per_tile;            // rows of a (sequence, key head)
  const long long rows = static_cast<long long>(P.c.B) * P.c.H * per;
  const long long at = static_cast<long long>(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32;
  if (at >= rows) return;
  const int bh = static_cast<int>(at / per), r = static_cast<int>(at % per);
  const int b = bh / P.c.H, h = bh % P.c.H;
  bool bad = false;                                   // reported by the attention
  const int count = P.counts == nullptr ? P.N : cache_count(__ldg(P.counts + b), P.N, &bad);
  const int n = r / P.group, head = h * P.group + r % P.group;
  if (n >= count) return;
  float mm = -INFINITY;
  for (int k = lane; k < P.splits; k += 32) mm = fmaxf(mm, P.part_ml[k * rows + at].x);
#pragma unroll
  for (int i = 16; i > 0; i /= 2) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, i));
  constexpr int C = D / 32;
  float ll = 0.0f, acc[C] = {};
  for (int k = 0; k < P.splits; ++k) {
    const float2 p = P.part_ml[k * rows + at];
    if (p.y == 0.0f) continue;
    const float f = p.x == -INFINITY ? 1.0f : ex2_ftz(p.x - mm);
    ll = fmaf(p.y, f, ll);
    const float* from = P.part_o + (k * rows + at) * D + lane * C;
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = fmaf(from[c], f, acc[c]);
  }
  const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
  char* to = P.o + b * P.ob + head * P.oh + n * P.on + 2 * lane * C;
#pragma unroll
  for (int c = 0; c < C; c += 2)
    *reinterpret_cast<uint32_t*>(to + 2 * c) = pack_bf16x2(acc[c] * inv, acc[c + 1] * inv);
  if (lane == 0 && P.lse != nullptr)
    P.lse[(static_cast<long long>(b) * P.Hq + head) * P.N + n] = (mm + log2f(ll)) * 0.6931471805599453f;
}

// Row warps, row tiles and splits of a call.
struct Shape {
  int rw, tiles, splits;
  long long rows;              // padded rows of all (sequence, key head)
};
Shape shape_of(const CacheAttnArgs& a, int num_sms) {
  Shape s;
  const long long rows = static_cast<long long>(a.Hq / a.cache.H) * a.N;
  s.rw = rows <= 16 ? 1 : (rows <= 32 ? 2 : 4);
  s.tiles = static_cast<int>((rows + s.rw * 16 - 1) / (s.rw * 16));
  const long long bh = static_cast<long long>(a.cache.B) * a.cache.H;
  s.rows = bh * s.tiles * s.rw * 16;
  // Enough CTAs for three on every SM, each key warp with two half pages at
  // the least (of a full table).
  const long long ctas = bh * s.tiles;
  long long splits = (3ll * num_sms + ctas - 1) / ctas;
  const long long most = (a.cache.blocks + 1ll) * 2 / (2 * (4 / s.rw));
  if (splits > most) splits = most;
  if (splits > 64) splits = 64;
  s.splits = splits < 1 ? 1 : static_cast<int>(splits);
  return s;
}

template <int D>
cudaError_t launch_d(const Ctx& c, const CacheAttnParams& P, const Shape& s) {
  const dim3 grid(static_cast<unsigned>(s.tiles) * s.splits, P.c.B * P.c.H);
  if (s.rw == 1) cache_attn_kernel<D, 1><<<grid, kThreads, 0, c.stream>>>(P);
  else if (s.rw == 2) cache_attn_kernel<D, 2><<<grid, kThreads, 0, c.stream>>>(P);
  else cache_attn_kernel<D, 4><<<grid, kThreads, 0, c.stream>>>(P);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || s.splits == 1) return e;
  cache_merge_kernel<D><<<static_cast<unsigned>((s.rows + 3) / 4), kThreads, 0, c.stream>>>(P, s.rw * 16);
  return cudaGetLastError();
}

}  // namespace

// Rows of a (sequence, key head) from which the tensor-core kernel takes over.
static bool many_rows(const CacheAttnArgs& a) {
  return static_cast<long long>(a.Hq / a.cache.H) * a.N > 64;
}

size_t cache_attn_ws_bytes(const CacheAttnArgs& a, int num_sms) {
  if (many_rows(a)) return cache_attn_tc_ws_bytes(a, num_sms);
  const Shape s = shape_of(a, num_sms);
  if (s.splits == 1) return 0;
  const size_t rows = static_cast<size_t>(s.rows) * s.splits;
  return align256(rows * a.cache.d * sizeof(float)) + align256(rows * sizeof(float2));
}

cudaError_t launch_cache_attn(const Ctx& c, const CacheAttnArgs& a) {
  CacheAttnParams P;
  P.c = a.cache;
  P.seq = a.seq;
  P.q = static_cast<const char*>(a.q);
  P.o = static_cast<char*>(a.o);
  P.qb = a.q_st[0] * 2; P.qh = a.q_st[1] * 2; P.qn = a.q_st[2] * 2;
  P.ob = a.o_st[0] * 2; P.oh = a.o_st[1] * 2; P.on = a.o_st[2] * 2;
  P.lse = a.lse;
  P.Hq = a.Hq;
  P.group = a.Hq / a.cache.H;
  P.N = a.N;
  P.counts = a.counts;
  P.frame = a.frame;
  P.window = a.window;
  P.scale_log2 = a.scale * 1.4426950408889634f;
  P.err = c.err;
  P.wait_ns = c.wait_ns;
  P.part_o = nullptr;
  P.part_ml = nullptr;
  if (many_rows(a)) return launch_cache_attn_tc(c, a, P);
  const Shape s = shape_of(a, c.num_sms);
  P.tiles = s.tiles;
  P.splits = s.splits;
  if (s.splits > 1) {
    const size_t rows = static_cast<size_t>(s.rows) * s.splits;
    P.part_o = static_cast<float*>(a.workspace);
    P.part_ml = reinterpret_cast<float2*>(static_cast<char*>(a.workspace) + align256(rows * a.cache.d * sizeof(float)));
  }
  return a.cache.d == 128 ? launch_d<128>(c, P, s) : launch_d<64>(c, P, s);
}

}  // namespace salad
