// cache_attn.cu -- attention of few query rows over the 8-bit block cache:
// o = softmax(scale q k^T + M) v for single tokens and short chunks.
//
// Memory-bound: a query token reads every key and value of its sequence once,
// 2 d bytes a token and head.  So the keys are split over as many warps as
// fill the GPU, and every key group (a warp, or the warps of 32 or 64 query
// rows) streams its own part through a ring of half pages (32 keys, their
// codes: two tensor copies each, swizzled so that the fragment reads below do
// not meet in a bank: 74 us for 124800 keys of 12 heads, 85 unswizzled) with
// its own barriers and none across the CTA: 96 KB in flight per CTA, two CTAs
// per SM, where 45 KB per SM cover the latency at the memory's rate.  The products are 16-row
// mma.sync tiles (query heads of a key head, and query tokens, fill the rows);
// with so few rows the tensor pipe is far from its limit and tcgen05's 128-row
// tiles would be mostly empty.
//
// Both contractions are reordered so that a lane's 16-byte loads are its MMA
// fragments.  QK: a lane holds 32 (16 at d = 64) consecutive channels of one
// key; MMA step i multiplies channels {4i, 4i+1 | 4i+2, 4i+3} of each lane's
// run, and the query fragments in shared memory are laid out the same way.  PV: a lane
// holds 16 consecutive channels of four keys; column tile j is channels = j
// mod 16, so lane group t ends with channels [32t, 32t+32) of its rows.
//
// Operands of closed blocks are fp16, in which a code is exact and converts in
// one instruction per pair.  Key scales, and the power of two that brings a
// query row into fp16's range, join the softmax scale.  P carries the power of
// two of its value block and is kept against the largest product of weight and
// scale, the row sum against the largest weight.  P, at most 2^15, is rounded to
// fp16: by 2^-11 of itself, or, 2^29 and more below the row's largest product of
// weight and scale, by 2^-40 of that.  The open block is multiplied in bf16 as it
// is held, by P rounded to bf16 (2^-8 of each weight).  Maxima, sums and O are
// float32.
//
// Balance: lengths are known on the device only and differ in a batch.  Every
// CTA sums them (up to 512 sequences) and takes an equal run of a head's work,
// which may begin and end inside a sequence; its key groups share each
// sequence's part of the run.  The work is half pages, and kEnter more where a
// CTA enters a further sequence: it has nothing in flight from the last one's
// end to the next one's first page (40 heads on 8, 16 sequences of 1346 to 16001
// keys: 73.5 us with 0, 63.3 with 8, 63.7 with 16, 64.2 with 32; 16 of 1196 to
// 2111 keys and 12 heads 33.4, 31.5, 30.8, 33.9).  A sequence that one CTA holds
// whole is written at once, the parts of the others are merged by a second
// launch.
//
// Measured (d = 128): one token, 12 heads, 31200 keys 29.7 us, 124800 keys 73.6
// us (5.2 TB/s; 14 us are launches, the chain lengths - table - pages - rows, and
// the merge); 16 tokens on 31200 keys 30.7 us, 32 47 us: there each of the two row
// warps converts the same codes, and two key groups have half of four's chains;
// 16 unequal sequences of 40 heads on 8 66.0 us (4.3 TB/s).
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

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
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
  __device__ __forceinline__ void load(const unsigned char* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ uint32_t word(int i) const { return part(v, i); }
  __device__ __forceinline__ void clear() { v = make_uint4(0u, 0u, 0u, 0u); }
};
template <>
struct Run<64> {
  uint2 v;
  __device__ __forceinline__ void load(const unsigned char* p) { v = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ uint32_t word(int i) const { return i == 0 ? v.x : v.y; }
  __device__ __forceinline__ void clear() { v = make_uint2(0u, 0u); }
};

template <int D, int RW>
struct Ring {
  static constexpr int kGroups = 4 / RW;                 // key groups of a CTA
  static constexpr int kHalf = 32 * D;                   // codes of 32 keys
  // 80 KB with 64 query rows, whose fragments take 16 KB: two CTAs per SM.
  static constexpr int kStages = (RW == 4 ? 80 : 96) * 1024 / (kGroups * 2 * kHalf);
  static constexpr int kBytes = kGroups * kStages * 2 * kHalf;
  static constexpr int kBars = kGroups * kStages * 2 * 8;
  static constexpr int kSmem = kBytes + kBars;
};

// P of the open block, which is multiplied in bf16 by values of any size, is at
// most 2^(kTopP - kOpenLift) = 2^-7: 64 products do not pass the largest value.
// (The sums so far give way in float32: the open block comes last.)
constexpr float kOpenLift = kTopP + 7.0f;
constexpr int kScan = 512;             // sequences that a CTA sums
constexpr int kEnter = 16;              // half pages that a further sequence's entry counts for

struct SeqSpan {
  int len, slot, count;
  int first, n;                        // half pages that the query rows see; n >= 1 where there is a row
};
__device__ __forceinline__ SeqSpan seq_span(const CacheAttnParams& P, int b, bool* bad) {
  const CacheSeq s = cache_seq(__ldg(P.seq + 2 * b), __ldg(P.seq + 2 * b + 1), P.c.blocks, bad);
  SeqSpan x{s.len, s.slot, P.counts == nullptr ? P.N : cache_count(__ldg(P.counts + b), P.N, bad), 0, 0};
  if (x.count == 0) return x;
  // lo and end grow with the row.
  const int lo = cache_visible(x.len - x.count, x.len, x.count, P.frame, P.window).lo;
  const int end = cache_visible(x.len - 1, x.len, x.count, P.frame, P.window).end;
  x.n = 1;
  if (end > lo) {
    x.first = lo / 32;
    x.n = (end + 31) / 32 - x.first;
  }
  return x;
}

// CTAs of a head that share `total` half pages of work: two half pages to a key
// group at the least.
__device__ __forceinline__ long long run_ctas(long long total, int slots) {
  const long long most = (total + 7) / 8;
  return most < slots ? (most < 1 ? 1 : most) : slots;
}

// RW: warps over row tiles of 16; the other warps of the CTA split the keys.
template <int D, int RW>
__global__ void __launch_bounds__(kThreads) cache_attn_kernel(const __grid_constant__ CacheAttnParams P,
                                                              const __grid_constant__ CUtensorMap k_map,
                                                              const __grid_constant__ CUtensorMap v_map) {
  constexpr int KW = 4 / RW;           // key groups
  constexpr int KS = D / 16;           // MMA steps of QK
  constexpr int NT = D / 8;            // column tiles of O
  constexpr int ROWS = RW * 16;
  using R = Ring<D, RW>;
  constexpr int NST = R::kStages;
  extern __shared__ __align__(1024) unsigned char ring[];     // [group][stage][K, V][32 keys][d]; O, for the merge
  auto os = reinterpret_cast<float (*)[KW][16][D + 4]>(ring);
  static_assert(KW == 1 || RW * KW * 16 * (D + 4) * 4 <= R::kBytes, "the merge fits the ring");
  __shared__ uint4 qs[RW][KS][32];
  __shared__ float2 mls[RW][KW][16];
  __shared__ uint32_t q_top[ROWS];     // largest magnitude of a query row, as bf16 bits
  __shared__ long long plan[kScan + 1];
  __shared__ long long warp_sum[4];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane / 4, t = lane % 4;
  const int rt = warp % RW, kw = warp / RW;
  const int h = blockIdx.y;
  // The second launch's CTAs may take their places as this one's leave them.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // The swizzle counts rows from 1024-byte boundaries.
  if (smem_u32(ring) & 1023u) {
    if (threadIdx.x == 0) atomicOr(P.err, kErrLayout);
    return;
  }
  if (threadIdx.x == 0) {
    tma_prefetch_map(&k_map);
    tma_prefetch_map(&v_map);
  }

  // Barriers of a group's stage: landed, and free again (one arrival a warp).
  uint64_t* bars = reinterpret_cast<uint64_t*>(ring + R::kBytes);
  auto landed = [&](int st) { return smem_u32(bars + (kw * NST + st) * 2); };
  auto freed = [&](int st) { return smem_u32(bars + (kw * NST + st) * 2 + 1); };
  if (rt == 0 && lane == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(landed(i), 1);
      mbar_init(freed(i), RW);
    }
    fence_mbar_init();
  }
  // Prefix sums of the sequences' work, and this CTA's run [w0, w1).
  const bool scan = P.c.B <= kScan;
  int b = blockIdx.x, b_end = b + 1;
  long long w0 = 0, w1 = 0x7fffffffffffffffll;
  if (scan) {
    long long sum = 0;
    for (int b0 = 0; b0 < P.c.B; b0 += kThreads) {
      const int i = b0 + threadIdx.x;
      bool bad = false;
      long long x = i < P.c.B ? seq_span(P, i, &bad).n : 0;
      if (bad && blockIdx.x == 0 && blockIdx.y == 0) atomicOr(P.err, kErrRange);
      if (i > 0 && x > 0) x += kEnter;
      const long long own = x;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const long long y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
      }
      if (lane == 31) warp_sum[warp] = x;
      __syncthreads();
      long long before = sum;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (k < warp) before += warp_sum[k];
        sum += warp_sum[k];
      }
      if (i < P.c.B) plan[i] = before + x - own;
      __syncthreads();
    }
    if (threadIdx.x == 0) plan[P.c.B] = sum;
    __syncthreads();
    const long long ctas = run_ctas(sum, gridDim.x);
    if (blockIdx.x == 0 && h == 0 && P.plan != nullptr) {
      // CTA x holds [sum x / ctas, sum (x + 1) / ctas): the first with a half page
      // of a sequence, and how many.
      for (int i = threadIdx.x; i < P.c.B; i += kThreads) {
        const long long from = plan[i] + (i > 0 ? kEnter : 0), to = plan[i + 1];
        const int x0 = static_cast<int>(((from + 1) * ctas + sum - 1) / sum) - 1;
        P.plan[i] = plan[i] == to ? make_int2(0, 0) : make_int2(x0, static_cast<int>((to * ctas + sum - 1) / sum) - x0);
      }
    }
    if (blockIdx.x >= ctas) return;
    w0 = sum * blockIdx.x / ctas;
    w1 = sum * (blockIdx.x + 1) / ctas;
    int lo = 0, hi = P.c.B;            // plan[lo] <= w0 < plan[hi], the last such lo
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (plan[mid] <= w0) lo = mid; else hi = mid;
    }
    b = lo;
    b_end = P.c.B;
  } else {
    __syncthreads();                   // the barriers
  }
  int done = 0;                        // half pages of this group's ring so far
  bool ok = true;
  for (; b < b_end && (!scan || plan[b] < w1); ++b) {
    bool bad = false;                    // reported above, or by the sequence's own CTA
    const SeqSpan s = seq_span(P, b, &bad);
    if (bad && !scan && threadIdx.x == 0 && h == 0) atomicOr(P.err, kErrRange);
    if (s.n == 0) continue;
    const int count = s.count;
    const long long from_b = scan ? plan[b] + (b > 0 ? kEnter : 0) : 0;
    const int part0 = w0 > from_b ? static_cast<int>(w0 - from_b) : 0;
    const int part1 = w1 - from_b < s.n ? static_cast<int>(w1 - from_b) : s.n;
    if (part1 <= part0) continue;        // the run ends, or begins, at the entry
    const bool whole = part0 == 0 && part1 == s.n;

    // This group's half pages: u0 + KW i below u1, of which the first nc are of
    // closed blocks.  Taken in turn, the open block's two go to two groups.
    const int u0 = s.first + part0 + kw, u1 = s.first + part1;
    const int uc = min(u1, 2 * (s.len / kCacheBlock));
    const int nc = max(0, (uc - u0 + KW - 1) / KW);
    unsigned char* stages = ring + static_cast<size_t>(kw) * NST * 2 * R::kHalf;
    const int32_t* table = P.c.page_table + static_cast<long long>(b) * P.c.blocks;
    // Pages and scales of the 32 blocks from block `first` on, one per lane (-1:
    // the entry is no page); the next 32 are loaded when these begin.
    struct Blocks {
      int page;
      float ks, vs;
    };
    auto blocks_at = [&](int first) {
      Blocks x{-1, 1.0f, 1.0f};
      if (2 * (first + lane) < uc) {
        x.page = cache_page(__ldg(table + first + lane), P.c.pages);
        const long long at = static_cast<long long>(x.page < 0 ? 0 : x.page) * P.c.H + h;
        x.ks = __ldg(P.c.k_scale + at);
        x.vs = __ldg(P.c.v_scale + at);
      }
      return x;
    };
    const int b0 = u0 / 2;
    Blocks cur = blocks_at(b0), nxt = blocks_at(b0 + 32);

    // Query fragments: entry (tile, step, lane) is the lane's A operand, as fp16
    // times a power of two that brings the row's largest magnitude into
    // [2^14, 2^15) (a row with an infinity or a NaN stays as it is).
    auto query = [&](int w, int ks, int l, int i) {
      const int c0 = (l % 4) * (D / 4) + (ks / 4) * 16 + (ks % 4) * 4;
      const int r = w * 16 + l / 4 + 8 * i;
      const int n = r / P.group;
      if (n >= count) return make_uint2(0u, 0u);
      return *reinterpret_cast<const uint2*>(P.q + b * P.qb + (h * P.group + r % P.group) * P.qh + n * P.qn + 2 * c0);
    };
    auto row_exponent = [&](int r) {
      const uint32_t top = q_top[r];
      const int e = top >= 0x7f80u ? 0 : static_cast<int>(top >> 7) - 127 - 14;
      return e < -100 ? -100 : e;
    };
    constexpr int QE = RW * KS * 32 / kThreads;       // entries of a thread
    uint2 qx[QE][2];
#pragma unroll
    for (int x = 0; x < QE; ++x) {
      const int e = threadIdx.x + x * kThreads, l = e % 32, w = e / (32 * KS);
#pragma unroll
      for (int i = 0; i < 2; ++i) qx[x][i] = query(w, (e / 32) % KS, l, i);
    }
    if (threadIdx.x < ROWS) q_top[threadIdx.x] = 0;
    // Half page i's copies (by the group's first warp); a block without a page
    // reads page 0, and is masked.
    auto fetch = [&](int i, const Blocks& x) {
      const int u = u0 + KW * i;
      const int page = __shfl_sync(0xffffffffu, x.page, (u / 2 - b0) % 32);
      if (rt == 0 && lane == 0) {
        const int st = (done + i) % NST;
        const int slab = (page < 0 ? 0 : page) * P.c.H + h;
        const uint32_t dst = smem_u32(stages) + st * 2 * R::kHalf;
        mbar_arrive_expect_tx(landed(st), 2 * R::kHalf);
        tma_load_3d(dst, &k_map, landed(st), 0, 32 * (u & 1), slab);
        tma_load_3d(dst + R::kHalf, &v_map, landed(st), 0, 32 * (u & 1), slab);
      }
    };
    // Block groups of 32 that `cur` and `nxt` hold: in_cur is the first one's number.
    int in_cur = 0;
    auto blocks_of = [&](int i) -> const Blocks& { return ((u0 + KW * i) / 2 - b0) / 32 == in_cur ? cur : nxt; };
    static_assert(NST * KW <= 62, "the ring stays within two groups of blocks");
    int issued = 0;
    for (; issued < nc && issued < NST; ++issued) fetch(issued, blocks_of(issued));
    __syncthreads();
#pragma unroll
    for (int x = 0; x < QE; ++x) {
      const int e = threadIdx.x + x * kThreads, l = e % 32, w = e / (32 * KS);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t top = __vmaxu2(qx[x][i].x & 0x7fff7fffu, qx[x][i].y & 0x7fff7fffu);
        atomicMax(&q_top[w * 16 + l / 4 + 8 * i], max(top & 0xffffu, top >> 16));
      }
    }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < QE; ++x) {
      const int e = threadIdx.x + x * kThreads, l = e % 32, w = e / (32 * KS);
      const float f0 = __int_as_float((127 - row_exponent(w * 16 + l / 4)) << 23);
      const float f1 = __int_as_float((127 - row_exponent(w * 16 + l / 4 + 8)) << 23);
      qs[w][(e / 32) % KS][l] = make_uint4(bf16x2_to_f16x2(qx[x][0].x, f0), bf16x2_to_f16x2(qx[x][1].x, f1),
                                           bf16x2_to_f16x2(qx[x][0].y, f0), bf16x2_to_f16x2(qx[x][1].y, f1));
    }
    __syncthreads();
    const float q_factor[2] = {P.scale_log2 * __int_as_float((127 + row_exponent(rt * 16 + g)) << 23),
                               P.scale_log2 * __int_as_float((127 + row_exponent(rt * 16 + g + 8)) << 23)};

    const int r0 = rt * 16;
    const CacheRow row[2] = {cache_row(P, r0 + g, h, s.len, count), cache_row(P, r0 + g + 8, h, s.len, count)};
    // Keys that every row of the tile sees.
    int all_lo = 0, all_end = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (row[i].valid) {
        all_lo = max(all_lo, row[i].see.lo);
        all_end = min(all_end, row[i].see.end);
      }
    }
    all_lo = __reduce_max_sync(0xffffffffu, all_lo);
    all_end = __reduce_min_sync(0xffffffffu, all_end);

    float o[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[j][i] = 0.0f;
    // Of each row: the largest s + ev + lift (s the base-2 score, ev the exponent
    // of its value block's scale), the largest s, and the sum of 2^(s - ms).
    float mt[2] = {-INFINITY, -INFINITY}, ms[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    float ev_top = -INFINITY;
    bool vbad[2] = {false, false};

    // One half page's softmax on S, the products of q with the code values: s =
    // S * c2 in the base-2 domain; P = 2^(s + ev - mt + kTopP) back in sc, at most
    // 2^(kTopP - lift).
    auto softmax = [&](float (&sc)[4][4], int kbase, float c20, float c21, float ev, float lift, bool odd, bool none) {
      const bool partial = odd || kbase < all_lo || kbase + 32 > all_end;
      const float c2[2] = {c20, c21};
      float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sc[i][e] *= c2[e >> 1];
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
      ev_top = fmaxf(ev_top, ev);
      float f[2], nt[2], ns[2];
      bool grow = false;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float tn = fmaxf(mt[i], top[i] + (ev + lift)), sn = fmaxf(ms[i], top[i]);
        grow = grow || tn > mt[i];
        f[i] = mt[i] == -INFINITY ? 0.0f : ex2_ftz(mt[i] - tn);
        if (sn > ms[i]) l[i] *= ex2_ftz(ms[i] - sn);
        mt[i] = tn;
        ms[i] = sn;
        // A row that has seen no key keeps -inf: exp2(-inf - 0) = 0.
        nt[i] = tn == -INFINITY ? 0.0f : kTopP - tn;
        ns[i] = sn == -INFINITY ? 0.0f : -sn;
      }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[j][e] *= f[e >> 1];
      }
      if (ev_top - ev > 90.0f) {
        // P may vanish beside another block's; the sum must not.
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            l[e >> 1] += ex2_ftz(sc[i][e] + ns[e >> 1]);
            sc[i][e] = ex2_ftz(sc[i][e] + (nt[e >> 1] + ev));
          }
        return;
      }
      float sum[2] = {0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sc[i][e] = ex2_ftz(sc[i][e] + (nt[e >> 1] + ev));
          sum[e >> 1] += sc[i][e];
        }
#pragma unroll
      for (int i = 0; i < 2; ++i) l[i] = fmaf(sum[i], ex2_ftz(ns[i] - nt[i] - ev), l[i]);
    };

    // ---- closed blocks
    for (int n = 0; n < nc; ++n) {
      const int u = u0 + KW * n;
      const int st = (done + n) % NST;
      const uint32_t phase = static_cast<uint32_t>((done + n) / NST) & 1u;
      if ((u / 2 - b0) / 32 != in_cur) {
        cur = nxt;
        ++in_cur;
        nxt = blocks_at(b0 + 32 * (in_cur + 1));
      }
      const int at = (u / 2 - b0) % 32;
      const bool none = __shfl_sync(0xffffffffu, cur.page, at) < 0;
      const float ks = __shfl_sync(0xffffffffu, cur.ks, at), vs = __shfl_sync(0xffffffffu, cur.vs, at);
      if (!__all_sync(0xffffffffu, mbar_wait_poll(landed(st), phase, P.wait_ns, nullptr))) {
        ok = false;
        break;
      }
      const unsigned char* kp = stages + st * 2 * R::kHalf + g * D;
      const unsigned char* vp = stages + st * 2 * R::kHalf + R::kHalf + 2 * t * D;
      // 16-byte chunk c of row r is at chunk c ^ (r % 8), at d = 64 at c ^ (r / 2 % 4);
      // a lane's rows are g and 2 t (+ 1) apart from multiples of 8.
      uint4 kr[4][D / 64];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int x = 0; x < D / 64; ++x)
          kr[i][x] = *reinterpret_cast<const uint4*>(kp + i * 8 * D + 16 * (D == 128 ? (2 * t + x) ^ g : t ^ (g >> 1)));
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
          const uint32_t w = part(kr[i][k / 4], k % 4);
          mma_f16(sc[i], a.x, a.y, a.z, a.w, e4m3_to_f16x2(w), e4m3_to_f16x2(w >> 16));
        }
      }
      const bool v_nan = isnan(vs);
      const float ev = v_nan ? 0.0f : pow2_log(vs);
      if (none && lane == 0) atomicOr(P.err, kErrRange);
      softmax(sc, 32 * u, ks * q_factor[0], ks * q_factor[1], ev, 0.0f, none || isnan(ks), none);
      Run<D> vr[2][4];
#pragma unroll
      for (int st2 = 0; st2 < 2; ++st2)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          vr[st2][i].load(vp + (16 * st2 + (i & 1) + 8 * (i >> 1)) * D +
                          (D == 128 ? 16 * (g ^ (2 * t + (i & 1))) : 16 * ((g >> 1) ^ t) + 8 * (g & 1)));
      if (v_nan || none) {
        // The codes may be NaN: the rows that see them are marked instead.
#pragma unroll
        for (int st = 0; st < 2; ++st)
#pragma unroll
          for (int i = 0; i < 4; ++i) vr[st][i].clear();
#pragma unroll
        for (int i = 0; i < 2; ++i)
          vbad[i] = vbad[i] || (!none && max(row[i].see.lo, 32 * u) < min(row[i].see.end, 32 * u + 32));
      }
      // The stage is read: it can be filled again, by the group's first warp once
      // every warp of the group says so.
      __syncwarp();
      if (RW > 1 && lane == 0) mbar_arrive(freed(st));
      if (issued < nc) {
        if (RW > 1 && rt == 0 &&
            !__all_sync(0xffffffffu, mbar_wait_poll(freed(st), phase, P.wait_ns, nullptr))) {
          ok = false;
          break;
        }
        fetch(issued, blocks_of(issued));
        ++issued;
      }
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        const uint32_t a0 = pack_f16x2(sc[2 * st][0], sc[2 * st][1]), a1 = pack_f16x2(sc[2 * st][2], sc[2 * st][3]);
        const uint32_t a2 = pack_f16x2(sc[2 * st + 1][0], sc[2 * st + 1][1]);
        const uint32_t a3 = pack_f16x2(sc[2 * st + 1][2], sc[2 * st + 1][3]);
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          // Channels 0, 1 and 2, 3 of two keys each: (key, next key) pairs.
          const uint32_t x0 = __byte_perm(vr[st][0].word(w), vr[st][1].word(w), 0x5140);
          const uint32_t x1 = __byte_perm(vr[st][0].word(w), vr[st][1].word(w), 0x7362);
          const uint32_t y0 = __byte_perm(vr[st][2].word(w), vr[st][3].word(w), 0x5140);
          const uint32_t y1 = __byte_perm(vr[st][2].word(w), vr[st][3].word(w), 0x7362);
          mma_f16(o[4 * w], a0, a1, a2, a3, e4m3_to_f16x2(x0), e4m3_to_f16x2(y0));
          mma_f16(o[4 * w + 1], a0, a1, a2, a3, e4m3_to_f16x2(x0 >> 16), e4m3_to_f16x2(y0 >> 16));
          mma_f16(o[4 * w + 2], a0, a1, a2, a3, e4m3_to_f16x2(x1), e4m3_to_f16x2(y1));
          mma_f16(o[4 * w + 3], a0, a1, a2, a3, e4m3_to_f16x2(x1 >> 16), e4m3_to_f16x2(y1 >> 16));
        }
      }
    }

    if (!ok) atomicOr(P.err, kErrTimeout);
    // No copy may be in flight when the ring is used again, or at the exit: each
    // one issued is waited for here, unless the loop above has seen it land.
    if (!ok && rt == 0)
      for (int n = max(0, issued - NST); n < issued; ++n)
        mbar_wait_poll(landed((done + n) % NST), static_cast<uint32_t>((done + n) / NST) & 1u, P.wait_ns, nullptr);
    done += nc;

    // ---- the open block, in bf16 (at most two half pages).  All
    // loads of a half page are issued before the first is used.
    for (int u = u0 + KW * nc; u < u1 && ok; u += KW) {
      const long long at = (((static_cast<long long>(b) * 2 + s.slot) * P.c.H + h) * kCacheBlock + (u & 1) * 32) * D;
      const __nv_bfloat16* kt = static_cast<const __nv_bfloat16*>(P.c.k_tail) + at;
      const __nv_bfloat16* vt = static_cast<const __nv_bfloat16*>(P.c.v_tail) + at;
      // 16-channel runs of a key as two 16-byte loads, as queries and keys have
      // them; of a value 16 (8 at d = 64) channels of four keys a step.
      uint4 kx[4][D / 64][2];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int x = 0; x < D / 64; ++x)
#pragma unroll
          for (int y = 0; y < 2; ++y)
            kx[i][x][y] = __ldg(reinterpret_cast<const uint4*>(kt + (8 * i + g) * D + (D / 4) * t + 16 * x + 8 * y));
      float sc[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[i][e] = 0.0f;
      {
        uint2 qt[KS][2];
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          qt[k][0] = query(rt, k, lane, 0);
          qt[k][1] = query(rt, k, lane, 1);
        }
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4& x = kx[i][k / 4][(k % 4) / 2];
            mma_bf16(sc[i], qt[k][0].x, qt[k][1].x, qt[k][0].y, qt[k][1].y, part(x, 2 * (k % 2)), part(x, 2 * (k % 2) + 1));
          }
      }
      uint4 vx[2][4][D / 64];
#pragma unroll
      for (int st = 0; st < 2; ++st)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int y = 0; y < D / 64; ++y)
            vx[st][i][y] = __ldg(reinterpret_cast<const uint4*>(
                vt + (16 * st + 2 * t + (i & 1) + 8 * (i >> 1)) * D + g * (D / 8) + 8 * y));
      softmax(sc, 32 * u, P.scale_log2, P.scale_log2, 0.0f, kOpenLift, false, false);
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
            const uint32_t y = part(vx[st][i][w / 4], w % 4);
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
      // The rows' means: sums of large values need not be a float.
      const float inv = weight_inv(l[i]);
      const float unit = mt[i] == -INFINITY ? 1.0f : ex2_ftz(mt[i] - kTopP - ms[i]);
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) o[j][2 * i + e] = vbad[i] ? __int_as_float(0x7fffffff) : o[j][2 * i + e] * inv * unit;
    }

    // ---- merge the CTA's key groups, then write the rows (or their part, in
    // the place of (CTA + sequence): one of the two grows from part to part)
    auto put = [&](int r, const float* acc, float mm, float ll, int c0, int nc) {
      // acc: nc channels from c0 of row r.
      const CacheRow x = cache_row(P, r, h, s.len, count);
      if (!x.valid) return;
      if (!whole) {
        const long long at = (static_cast<long long>(blockIdx.x + b) * P.c.H + h) * ROWS + r;
        if (c0 == 0) P.part_ml[at] = make_float2(mm, ll);
        float* to = P.part_o + at * D + c0;
#pragma unroll
        for (int c = 0; c < nc; c += 4)
          *reinterpret_cast<float4*>(to + c) = make_float4(acc[c], acc[c + 1], acc[c + 2], acc[c + 3]);
        return;
      }
      char* to = P.o + b * P.ob + x.head * P.oh + x.n * P.on + 2 * c0;
#pragma unroll
      for (int c = 0; c < nc; c += 8)
        *reinterpret_cast<uint4*>(to + 2 * c) =
            make_uint4(pack_bf16x2(acc[c], acc[c + 1]), pack_bf16x2(acc[c + 2], acc[c + 3]),
                       pack_bf16x2(acc[c + 4], acc[c + 5]), pack_bf16x2(acc[c + 6], acc[c + 7]));
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
        put(rt * 16 + g + 8 * i, acc, ms[i], l[i], t * (D / 4), D / 4);
      }
    } else {
      __syncthreads();                 // every group is done with the ring
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int j = 0; j < NT; j += 4) {
          *reinterpret_cast<float4*>(&os[rt][kw][g + 8 * i][t * (D / 4) + j]) =
              make_float4(o[j][2 * i], o[j + 1][2 * i], o[j + 2][2 * i], o[j + 3][2 * i]);
          *reinterpret_cast<float4*>(&os[rt][kw][g + 8 * i][t * (D / 4) + NT + j]) =
              make_float4(o[j][2 * i + 1], o[j + 1][2 * i + 1], o[j + 2][2 * i + 1], o[j + 3][2 * i + 1]);
        }
        if (t == 0) mls[rt][kw][g + 8 * i] = make_float2(ms[i], l[i]);
      }
      __syncthreads();
      for (int e = threadIdx.x; e < RW * 16 * (D / 8); e += kThreads) {
        const int r = e / (D / 8), c0 = e % (D / 8) * 8;
        const int w = r / 16, rr = r % 16;
        float mm = -INFINITY, ll = 0.0f, f[KW], acc[8] = {};
#pragma unroll
        for (int k = 0; k < KW; ++k) mm = fmaxf(mm, mls[w][k][rr].x);
#pragma unroll
        for (int k = 0; k < KW; ++k) ll += f[k] = part_weight(mls[w][k][rr], mm);
        const float inv = weight_inv(ll);
#pragma unroll
        for (int k = 0; k < KW; ++k)
#pragma unroll
          for (int c = 0; c < 8; ++c) acc[c] = fmaf(os[w][k][rr][c0 + c], f[k] * inv, acc[c]);
        put(r, acc, mm, ll, c0, 8);
      }
    }
    // The ring and the fragments are the next sequence's.
    fence_proxy_async_smem();
    if (!__syncthreads_and(ok)) break;
  }
}

// Merges the parts of the sequences that more than one CTA worked on: a CTA
// per row, whose warps take a quarter of its parts each.
constexpr int kMergeLane = 3;          // parts of a lane
constexpr int kMaxParts = 4 * 32 * kMergeLane;
template <int D>
__global__ void __launch_bounds__(kThreads) cache_merge_kernel(const __grid_constant__ CacheAttnParams P, int rows, int slots) {
  constexpr int C = D / 32;
  constexpr int FLY = 16;              // parts whose loads are in flight
  __shared__ float os[4][D];
  __shared__ float2 mls[4];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int used = P.group * P.N;      // of the `rows` that a part holds
  const int r = blockIdx.x % used, h = blockIdx.x / used % P.c.H, b = blockIdx.x / used / P.c.H;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int2 parts = P.plan[b];
  const int x0 = parts.x, n = parts.y;
  if (n <= 1 || x0 < 0 || x0 + n > slots) return;
  bool bad = false;                                   // reported by the attention
  const int count = P.counts == nullptr ? P.N : cache_count(__ldg(P.counts + b), P.N, &bad);
  const int i_q = r / P.group, head = h * P.group + r % P.group;
  if (i_q >= count) return;
  const int k0 = n * warp / 4, nw = n * (warp + 1) / 4 - k0;
  const long long step = static_cast<long long>(P.c.H) * rows;
  const long long at = (static_cast<long long>(x0 + b + k0) * P.c.H + h) * rows + r;
  const float* from = P.part_o + at * D + lane * C;
  float v[FLY][C];
  auto load = [&](int k) {
#pragma unroll
    for (int i = 0; i < FLY; ++i)
#pragma unroll
      for (int c = 0; c < C; ++c) v[i][c] = k + i < nw ? from[(k + i) * step * D + c] : 0.0f;
  };
  load(0);
  float2 p[kMergeLane];
  float mm = -INFINITY;
#pragma unroll
  for (int i = 0; i < kMergeLane; ++i) {
    p[i] = lane + 32 * i < nw ? P.part_ml[at + (lane + 32 * i) * step] : make_float2(-INFINITY, 0.0f);
    mm = fmaxf(mm, p[i].x);
  }
#pragma unroll
  for (int i = 16; i > 0; i /= 2) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, i));
  // The parts' weights, and the warp's mean.
  float w[kMergeLane], ll = 0.0f, acc[C] = {};
#pragma unroll
  for (int i = 0; i < kMergeLane; ++i) ll += w[i] = part_weight(p[i], mm);
#pragma unroll
  for (int i = 16; i > 0; i /= 2) ll += __shfl_xor_sync(0xffffffffu, ll, i);
  const float inv = weight_inv(ll);
#pragma unroll
  for (int i = 0; i < kMergeLane; ++i) {
    for (int k = 32 * i; k < min(nw, 32 * i + 32); k += FLY) {
      if (k > 0) load(k);
#pragma unroll
      for (int j = 0; j < FLY; ++j) {
        const float f = __shfl_sync(0xffffffffu, w[i] * inv, (k + j) % 32);
#pragma unroll
        for (int c = 0; c < C; ++c) acc[c] = fmaf(v[j][c], f, acc[c]);
      }
    }
  }
#pragma unroll
  for (int c = 0; c < C; ++c) os[warp][lane * C + c] = acc[c];
  if (lane == 0) mls[warp] = make_float2(mm, ll);
  __syncthreads();
  if (warp > 0) return;
  mm = fmaxf(fmaxf(mls[0].x, mls[1].x), fmaxf(mls[2].x, mls[3].x));
  float sum = 0.0f, f[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) sum += f[k] = part_weight(mls[k], mm);
#pragma unroll
  for (int c = 0; c < C; ++c) acc[c] = 0.0f;
  const float all = weight_inv(sum);
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = fmaf(os[k][lane * C + c], f[k] * all, acc[c]);
  char* to = P.o + b * P.ob + head * P.oh + i_q * P.on + 2 * lane * C;
#pragma unroll
  for (int c = 0; c < C; c += 2)
    *reinterpret_cast<uint32_t*>(to + 2 * c) = pack_bf16x2(acc[c], acc[c + 1]);
  if (lane == 0 && P.lse != nullptr)
    P.lse[(static_cast<long long>(b) * P.Hq + head) * P.N + i_q] = (mm + log2f(sum)) * 0.6931471805599453f;
}

// Row warps and CTAs per head of a call.
struct Shape {
  int rw, slots;
  bool merge;                  // a sequence may be in more than one CTA
  size_t part_o, part_ml, plan, total;
};
Shape shape_of(const CacheAttnArgs& a, int num_sms) {
  Shape s;
  const int B = a.cache.B, H = a.cache.H;
  const long long rows = static_cast<long long>(a.Hq / H) * a.N;
  s.rw = rows <= 16 ? 1 : (rows <= 32 ? 2 : 4);
  // One wave of two CTAs to an SM, each with eight half pages at the least (of
  // a full table); kMaxParts of a sequence at most, which is what the merge
  // holds.  Past kScan sequences a CTA takes one of them each.
  long long slots = 2ll * num_sms / H;
  const long long most = (B * (2ll * a.cache.blocks + 2 + kEnter) + 7) / 8;
  if (slots > most) slots = most;
  if (slots > kMaxParts) slots = kMaxParts;
  if (slots < 1) slots = 1;
  s.merge = B <= kScan && slots > 1;
  s.slots = B <= kScan ? static_cast<int>(slots) : B;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += align256(bytes);
    return o;
  };
  s.part_o = s.part_ml = s.plan = 0;
  if (s.merge) {
    const size_t parts = (static_cast<size_t>(s.slots) + B) * H * s.rw * 16;
    s.part_o = take(parts * a.cache.d * sizeof(float));
    s.part_ml = take(parts * sizeof(float2));
    s.plan = take(static_cast<size_t>(B) * sizeof(int2));
  }
  s.total = off;
  return s;
}

template <int D, int RW>
cudaError_t launch_rw(const Ctx& c, const CacheAttnParams& P, const Shape& s) {
  const dim3 grid(s.slots, P.c.H);
  const cudaError_t e = cudaFuncSetAttribute(cache_attn_kernel<D, RW>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             Ring<D, RW>::kSmem);
  if (e != cudaSuccess) return e;
  CUtensorMap k_map, v_map;
  const long long slabs = static_cast<long long>(P.c.pages) * P.c.H;
  if (!make_tmap_codes(&k_map, P.c.k_pages, slabs, D) || !make_tmap_codes(&v_map, P.c.v_pages, slabs, D))
    return cudaErrorInvalidValue;
  cache_attn_kernel<D, RW><<<grid, kThreads, Ring<D, RW>::kSmem, c.stream>>>(P, k_map, v_map);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const Ctx& c, const CacheAttnParams& P, const Shape& s) {
  const cudaError_t e = s.rw == 1 ? launch_rw<D, 1>(c, P, s) : (s.rw == 2 ? launch_rw<D, 2>(c, P, s) : launch_rw<D, 4>(c, P, s));
  if (e != cudaSuccess || !s.merge) return e;
  const long long rows = static_cast<long long>(P.c.B) * P.c.H * P.group * P.N;
  // Launched while the attention runs; it waits for its end before it reads.
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = c.stream;
  cudaLaunchAttribute early = {};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_merge_kernel<D>, P, s.rw * 16, s.slots);
}

}  // namespace

// Whether the tensor-core kernel takes the call: with more than 64 rows of a
// (sequence, key head), which is what a CTA of this file's kernel holds, and
// with more than 32 where the tables have room for much work.  At 33 to 64 rows
// (64 here, 65 there; 12 heads) 1000 keys take 25 us and 27, 7800 36 and 38,
// 31200 82 and 75; 60 rows, 8 heads and 16 sequences of 8640 keys 234 and 154.
// Both are far from the 14.6 us that reading 31200 keys takes: neither shares a
// converted tile among as many warps as the rows leave room for.
// Lengths are not known here; a table much wider than its sequences costs the
// difference of the short ones.  At 17 to 32 rows this one is ahead at any
// length (31200 keys: 49 and 75).
static bool many_rows(const CacheAttnArgs& a, int num_sms) {
  const long long rows = static_cast<long long>(a.Hq / a.cache.H) * a.N;
  const long long blocks = static_cast<long long>(a.cache.B) * a.cache.H * a.cache.blocks;
  return rows > 64 || (rows > 32 && blocks > 16ll * num_sms);
}

size_t cache_attn_ws_bytes(const CacheAttnArgs& a, int num_sms) {
  if (many_rows(a, num_sms)) return cache_attn_tc_ws_bytes(a, num_sms);
  return shape_of(a, num_sms).total;
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
  P.plan = nullptr;
  if (many_rows(a, c.num_sms)) return launch_cache_attn_tc(c, a, P);
  const Shape s = shape_of(a, c.num_sms);
  P.tiles = 1;
  if (s.merge) {
    char* ws = static_cast<char*>(a.workspace);
    P.part_o = reinterpret_cast<float*>(ws + s.part_o);
    P.part_ml = reinterpret_cast<float2*>(ws + s.part_ml);
    P.plan = reinterpret_cast<int2*>(ws + s.plan);
  }
  return a.cache.d == 128 ? launch_d<128>(c, P, s) : launch_d<64>(c, P, s);
}

}  // namespace salad
