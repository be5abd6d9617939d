// cache_attn_tc.cu -- attention of many query rows (chunks of latent frames)
// over the 8-bit block cache, on tcgen05 tensor cores.
//
// Bound by the tensor pipe (4 d operations per query row, key and head) and,
// close behind it, by the exponentials.  A work item is 256 query rows of one
// sequence and key head: two 128-row slots that share every key tile, so each
// tile of codes is read and turned into bf16 once per 256 rows.  A key tile is
// 128 keys (two blocks).
//
// Warp roles (512 threads, one CTA per SM; warps 13..15 only fill the last
// warpgroup, whose registers the others take):
//   warps 0..3, 4..7   softmax and output of slots 0 and 1, a row per thread
//                      (warp w on TMEM lane quarter w % 4); they also load
//                      their slot's rows of Q
//   warps 8..11        codes -> bf16: global loads one operand tile ahead,
//                      conversion in registers, 128-byte-swizzled stores; they
//                      also pass the blocks' scales to the softmax warps
//   warp 12            TMEM allocation and the single MMA-issuing thread
// While the tensor pipe runs one slot's PV(t) and QK(t+1), the other slot's
// softmax runs.  P overwrites S in TMEM as bf16.
//
// The conversion leaves channels in the order (0, 2, 1, 3) within each group
// of four.  Q is stored in that order too (the dot products do not change),
// and the output's columns are put back when O is written.
//
// Balance: lengths are known on the device only, and tiles per item differ by
// frame.  A first launch sums the items' tiles; every CTA then takes an equal
// run of tiles, which may begin and end inside an item.  An item that one CTA
// holds whole is written at once; the others leave float32 parts (two per
// CTA at most), merged by a last launch.
#include "cache_attn.cuh"

namespace salad {
namespace {

constexpr int kRows = 256;            // query rows of an item
constexpr int kTile = 128;            // keys of a tile
constexpr int kThreads = 512;       // four warpgroups, see the register shares

template <int D>
struct CT {
  static constexpr int kSlabs = D / 64;
  static constexpr int kRowSlab = 128 * 128;            // 128 rows of 128 bytes
  static constexpr int kOperand = kSlabs * kRowSlab;    // 128 rows of Q, K or V
  static constexpr int kStages = 4;
  static constexpr int kBarBytes = 256;
  static constexpr int kScaleBytes = 4 * 16 + 4 * 8;    // scales of four tiles (K, K, V, V), four parts' (tiles, slots)
  static constexpr int kUsed = 2 * kOperand + kStages * kOperand + kBarBytes + kScaleBytes;
  // More than half of the SM's shared memory: one CTA (and its 512 TMEM columns) per SM.
  static constexpr int kSmem = kUsed > 120 * 1024 ? kUsed : 120 * 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
  __host__ __device__ static constexpr uint32_t o_col(int slot) { return slot ? D : 0; }
  __host__ __device__ static constexpr uint32_t s_col(int slot) { return 2 * D + (slot ? 128 : 0); }
  static constexpr uint32_t kCols = 512;
};

struct TcParams {
  CacheAttnParams a;          // tiles: items of a (sequence, key head)
  int* tile_prefix;           // [B][tiles + 1]
  long long* seq_prefix;      // [B + 1], tiles of all heads of the sequences before
};

// Tiles of keys that item `tile` of a sequence walks over: [first, first + n).
// An item with a valid row has at least one (a row that sees no key still has
// to be written).
struct TileRange {
  int first, n;
};
__device__ __forceinline__ TileRange item_tiles(const CacheAttnParams& P, int tile, int len, int count) {
  const int r0 = tile * kRows;
  const int valid = count * P.group;
  if (r0 >= valid) return TileRange{0, 0};
  const int n0 = r0 / P.group, n1 = (min(valid, r0 + kRows) - 1) / P.group;
  // lo and end grow with the row.
  const int lo = cache_visible(len - count + n0, len, count, P.frame, P.window).lo;
  const int end = cache_visible(len - count + n1, len, count, P.frame, P.window).end;
  if (end <= lo) return TileRange{0, 1};
  const int first = lo / kTile;
  return TileRange{first, (end + kTile - 1) / kTile - first};
}

struct SeqInfo {
  int len, slot, count;
};
__device__ __forceinline__ SeqInfo seq_info(const CacheAttnParams& P, int b, bool* bad) {
  const CacheSeq s = cache_seq(__ldg(P.seq + 2 * b), __ldg(P.seq + 2 * b + 1), P.c.blocks, bad);
  const int count = P.counts == nullptr ? P.N : cache_count(__ldg(P.counts + b), P.N, bad);
  return SeqInfo{s.len, s.slot, count};
}

// CTAs that share the work: all, or fewer where that leaves under two tiles each.
__device__ __forceinline__ long long work_ctas(long long total, int ctas) {
  const long long most = (total + 1) / 2;
  return most < ctas ? (most < 1 ? 1 : most) : ctas;
}

// Prefix sums of the items' tiles: one CTA, a warp per sequence.
__global__ void __launch_bounds__(1024) cache_plan_kernel(const __grid_constant__ TcParams T) {
  const CacheAttnParams& P = T.a;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  for (int b = warp; b < P.c.B; b += 32) {
    bool bad = false;
    const SeqInfo s = seq_info(P, b, &bad);
    if (bad && lane == 0) atomicOr(P.err, kErrRange);
    int* out = T.tile_prefix + static_cast<long long>(b) * (P.tiles + 1);
    int sum = 0;
    for (int t0 = 0; t0 < P.tiles; t0 += 32) {
      const int t = t0 + lane;
      const int n = t < P.tiles ? item_tiles(P, t, s.len, s.count).n : 0;
      int x = n;
#pragma unroll
      for (int i = 1; i < 32; i *= 2) {
        const int y = __shfl_up_sync(0xffffffffu, x, i);
        if (lane >= i) x += y;
      }
      if (t < P.tiles) out[t] = sum + x - n;
      sum += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) out[P.tiles] = sum;
  }
  __syncthreads();
  if (warp == 0) {
    long long sum = 0;
    for (int b0 = 0; b0 < P.c.B; b0 += 32) {
      const int b = b0 + lane;
      const long long n =
          b < P.c.B ? static_cast<long long>(T.tile_prefix[static_cast<long long>(b) * (P.tiles + 1) + P.tiles]) * P.c.H : 0;
      long long x = n;
#pragma unroll
      for (int i = 1; i < 32; i *= 2) {
        const long long y = __shfl_up_sync(0xffffffffu, x, i);
        if (lane >= i) x += y;
      }
      if (b < P.c.B) T.seq_prefix[b] = sum + x - n;
      sum += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) T.seq_prefix[P.c.B] = sum;
  }
}

// One CTA's part of an item.
struct Seg {
  int b, h, tile;
  SeqInfo s;
  TileRange all;       // the item's tiles
  int t0, t1;          // this part's, of all.n
  bool first;          // the CTA's first part
  bool two;            // slot 1 has rows
  long long left;      // tiles of the CTA from t0 on
};

__device__ __forceinline__ void seg_open(const CacheAttnParams& P, Seg& g) {
  bool bad = false;    // reported by the plan
  g.s = seq_info(P, g.b, &bad);
  g.all = item_tiles(P, g.tile, g.s.len, g.s.count);
}
__device__ __forceinline__ void seg_close(const CacheAttnParams& P, Seg& g) {
  g.t1 = g.all.n - g.t0 < g.left ? g.all.n : g.t0 + static_cast<int>(g.left);
  g.two = g.tile * kRows + 128 < g.s.count * P.group;
}

// The part that starts at global tile w; `left` tiles of the CTA remain.
__device__ __forceinline__ Seg seg_at(const TcParams& T, long long w, long long left) {
  const CacheAttnParams& P = T.a;
  Seg g;
  int lo = 0, hi = P.c.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (__ldg(T.seq_prefix + mid) <= w) lo = mid; else hi = mid;
  }
  g.b = lo;
  const int* pre = T.tile_prefix + static_cast<long long>(g.b) * (P.tiles + 1);
  const int per = __ldg(pre + P.tiles);
  const long long rem = w - __ldg(T.seq_prefix + g.b);
  g.h = static_cast<int>(rem / per);
  const int at = static_cast<int>(rem % per);
  lo = 0;
  hi = P.tiles;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (__ldg(pre + mid) <= at) lo = mid; else hi = mid;
  }
  g.tile = lo;
  g.left = left;
  g.first = true;
  seg_open(P, g);
  g.t0 = at - __ldg(pre + lo);
  seg_close(P, g);
  return g;
}

// The next part; left == 0 where there is none.
__device__ __forceinline__ Seg seg_next(const CacheAttnParams& P, const Seg& g) {
  Seg n = g;
  n.left = g.left - (g.t1 - g.t0);
  n.first = false;
  if (n.left <= 0) return n;
  do {
    if (++n.tile == P.tiles) {
      n.tile = 0;
      if (++n.h == P.c.H) {
        n.h = 0;
        ++n.b;
      }
    }
    seg_open(P, n);
  } while (n.all.n == 0);
  n.t0 = 0;
  seg_close(P, n);
  return n;
}

__device__ __forceinline__ float max64(const float* v) {
  float a[22];
#pragma unroll
  for (int i = 0; i < 21; ++i) a[i] = fmax3(v[3 * i], v[3 * i + 1], v[3 * i + 2]);
  a[21] = v[63];
  float b[8];
#pragma unroll
  for (int i = 0; i < 7; ++i) b[i] = fmax3(a[3 * i], a[3 * i + 1], a[3 * i + 2]);
  b[7] = a[21];
  return fmax3(fmax3(b[0], b[1], b[2]), fmax3(b[3], b[4], b[5]), fmaxf(b[6], b[7]));
}

// Pairs of floats in one register pair (two operations an instruction).
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// What a block's products are scaled by: positive, so that -inf stays -inf
// (under a NaN scale the scores that count are NaN already).
__device__ __forceinline__ float key_factor(float scale_log2, float ks) {
  return isnan(ks) ? 1.0f : fmaxf(scale_log2 * ks, 1e-37f);
}

// Channels in the order that e4m3_pairs leaves them: (0, 2, 1, 3) of each four.
__device__ __forceinline__ uint4 reorder(uint4 v) {
  return make_uint4(__byte_perm(v.x, v.y, 0x5410), __byte_perm(v.x, v.y, 0x7632),
                    __byte_perm(v.z, v.w, 0x5410), __byte_perm(v.z, v.w, 0x7632));
}

__device__ __forceinline__ uint32_t finite_or_zero(uint32_t pair) {
  if ((pair & 0x7f80u) == 0x7f80u) pair &= 0xffff0000u;
  if ((pair & 0x7f800000u) == 0x7f800000u) pair &= 0xffffu;
  return pair;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) cache_tc_kernel(const __grid_constant__ TcParams T) {
  using C = CT<D>;
  constexpr int NS = C::kStages;
  const CacheAttnParams& P = T.a;
  extern __shared__ __align__(1024) unsigned char smem[];
  if (reinterpret_cast<uintptr_t>(smem) & 1023u) {
    if (threadIdx.x == 0) atomicOr(P.err, kErrLayout);
    return;
  }
  const long long total = __ldg(T.seq_prefix + P.c.B);
  const long long ctas = work_ctas(total, gridDim.x);
  if (blockIdx.x >= ctas) return;
  const long long w0 = total * blockIdx.x / ctas, w1 = total * (blockIdx.x + 1) / ctas;
  if (w0 >= w1) return;

  unsigned char* qbuf = smem;                               // [2 slots][d-slab][128 rows]
  unsigned char* ring = smem + 2 * C::kOperand;             // [NS][d-slab][128 rows]
  uint64_t* bars = reinterpret_cast<uint64_t*>(ring + NS * C::kOperand);
  // full[NS] empty[NS] q_full[2] q_free[2] s_full[2] p_full[2] o_done[2] drain
  auto bar = [&](int i) { return smem_u32(bars + i); };
  auto full = [&](int i) { return bar(i); };
  auto empty = [&](int i) { return bar(NS + i); };
  auto q_full = [&](int i) { return bar(2 * NS + i); };
  auto q_free = [&](int i) { return bar(2 * NS + 2 + i); };
  auto s_full = [&](int i) { return bar(2 * NS + 4 + i); };
  auto p_full = [&](int i) { return bar(2 * NS + 6 + i); };
  auto o_done = [&](int i) { return bar(2 * NS + 8 + i); };
  const uint32_t drain = bar(2 * NS + 10);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 2 * NS + 11);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  // odd_seg[i % 4] = i + 1: part i's open block holds a value that is not finite.
  volatile int* odd_seg = abort_flag + 1;
  static_assert((2 * NS + 11) * 8 + 4 + 4 + 16 <= C::kBarBytes, "barrier region");
  // Scales of tile i's two blocks in entry i % 4: of the keys (0: no page, its
  // keys do not count), then of the values.  A converting thread writes them
  // before it hands over the tile's keys.  It reaches tile i + 4 only when the
  // values of tile i + 3 are stored, over those of tile i + 1: both slots have
  // read tile i's scales by then.
  float4* scales = reinterpret_cast<float4*>(reinterpret_cast<unsigned char*>(bars) + C::kBarBytes);
  // Tiles and slots of part i in entry i % 4, for the issuer: written and read
  // like the scales (a part has a tile at least).
  int2* part_info = reinterpret_cast<int2*>(scales + 4);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const unsigned long long wait_ns = P.wait_ns;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(full(i), 4);      // the four converting warps
      mbar_init(empty(i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full(i), 4);    // the slot's four softmax warps
      mbar_init(q_free(i), 1);
      mbar_init(s_full(i), 1);
      mbar_init(p_full(i), 4);
      mbar_init(o_done(i), 1);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    for (int i = 0; i < 4; ++i) odd_seg[i] = 0;
    fence_mbar_init();
  }
  if (warp == 12) {
    tmem_alloc(smem_u32(tmem_holder), C::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;

  // Register shares, 4 x 128 in all: 160 for each softmax warpgroup, 128 for
  // the converting one, 64 for the issuer's.
  if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == 12 && lane == 0) {
      // ===================================================== MMA issuer
      constexpr uint32_t idesc_qk = idesc_bf16(128, 128, false, false);
      constexpr uint32_t idesc_pv = idesc_bf16(128, D, false, true);
      const uint32_t ring_base = smem_u32(ring);
      const uint64_t qd[2] = {sdesc_sw128(smem_u32(qbuf), 16, 1024),
                              sdesc_sw128(smem_u32(qbuf) + C::kOperand, 16, 1024)};
      uint32_t at = 0;                      // ring stages consumed so far
      uint32_t qn[2] = {0, 0}, pn[2] = {0, 0};
      bool ok = true;
      auto wait_stage = [&](uint32_t i) -> bool { return mbar_wait(full(i % NS), (i / NS) & 1u, wait_ns, abort_flag); };
      auto issue_qk = [&](int slot, uint32_t i) {
        const uint64_t kd = sdesc_sw128(ring_base + (i % NS) * C::kOperand, 16, 1024);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint64_t off = static_cast<uint64_t>(((ks / 4) * C::kRowSlab + (ks % 4) * 32) >> 4);
          mma_ss(tmem + C::s_col(slot), qd[slot] + off, kd + off, idesc_qk, ks > 0 ? 1u : 0u);
        }
        mma_commit(s_full(slot));
      };
      int left = static_cast<int>(w1 - w0);
      for (int part_no = 0; left > 0 && ok; ++part_no) {
        // Stages of the part: K0 V0 K1 V1 ...
        if (!wait_stage(at)) { ok = false; break; }
        const int2 info = part_info[part_no % 4];
        const int n = info.x, slots = info.y;
        for (int slot = 0; slot < slots && ok; ++slot) {
          ok = mbar_wait(q_full(slot), qn[slot]++ & 1u, wait_ns, abort_flag);
          if (!ok) break;
          tc_fence_after();
          issue_qk(slot, at);
          if (n == 1) mma_commit(q_free(slot));
        }
        if (!ok) break;
        mma_commit(empty(at % NS));
        for (int t = 0; t < n && ok; ++t) {
          const uint32_t vi = at + 2 * t + 1;
          const uint64_t vd = sdesc_sw128(ring_base + (vi % NS) * C::kOperand, C::kRowSlab, 1024);
          for (int slot = 0; slot < slots && ok; ++slot) {
            ok = mbar_wait(p_full(slot), pn[slot]++ & 1u, wait_ns, abort_flag) && (slot > 0 || wait_stage(vi));
            if (!ok) break;
            tc_fence_after();
            const uint32_t sa = tmem + C::s_col(slot), oa = tmem + C::o_col(slot);
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)      // 16 keys each
              mma_ts(oa, sa + ks * 8, vd + static_cast<uint64_t>((ks * 2048) >> 4), idesc_pv,
                     ks > 0 ? 1u : (t > 0 ? 1u : 0u));
            mma_commit(o_done(slot));
            if (slot == slots - 1) mma_commit(empty(vi % NS));
            if (t + 1 < n) {
              if (slot == 0 && !wait_stage(vi + 1)) { ok = false; break; }
              tc_fence_after();
              issue_qk(slot, vi + 1);            // over this slot's P: behind its PV in issue order
              if (t + 2 == n) mma_commit(q_free(slot));
              if (slot == slots - 1) mma_commit(empty((vi + 1) % NS));
            }
          }
        }
        at += 2 * n;
        left -= n;
      }
      if (!ok) raise_timeout(P.err, abort_flag);
      mma_commit(drain);
      if (!mbar_wait(drain, 0, wait_ns, nullptr)) atomicOr(P.err, kErrTimeout);
    }
  } else if (warp >= 8) {
    // ================================================== codes -> bf16
    const int w = warp - 8;
    const int c16 = lane % 4;                   // 16 channels of a 64-channel slab
    const int r8 = 8 * w + lane / 4;            // rows r8 + 32 i; rows 64 and up are the tile's second block
    uint32_t at = 0;                            // operand tiles written so far
    int part_no = 0;
    bool ok = true;
    // Codes of one operand tile: rows i of block i / 2.
    auto load = [&](uint4 (&to)[4][C::kSlabs], const unsigned char* pages, const int (&page)[2], int h) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int pg = page[i / 2];
        const unsigned char* p =
            pages + ((static_cast<long long>(pg < 0 ? 0 : pg) * P.c.H + h) * kCacheBlock + (r8 + 32 * i) % 64) * D + 16 * c16;
#pragma unroll
        for (int s = 0; s < C::kSlabs; ++s)
          to[i][s] = pg == -2 ? make_uint4(0u, 0u, 0u, 0u) : __ldg(reinterpret_cast<const uint4*>(p + 64 * s));
      }
    };
    // Pages and scales of 32 blocks, one per lane: -2 where the block is not
    // closed.  A table entry that is no page reads page 0 with a key scale of
    // 0, by which the softmax masks its keys.
    struct Blocks {
      int page;
      float ks, vs;
    };
    auto blocks_at = [&](const Seg& g, int blk) {
      Blocks k{-2, 1.0f, 1.0f};
      if (blk + lane < g.s.len / kCacheBlock) {
        k.page = cache_page(__ldg(P.c.page_table + static_cast<long long>(g.b) * P.c.blocks + blk + lane), P.c.pages);
        if (k.page < 0) {
          k.page = 0;
          k.ks = 0.0f;
        } else {
          const long long at = static_cast<long long>(k.page) * P.c.H + g.h;
          k.ks = __ldg(P.c.k_scale + at);
          k.vs = __ldg(P.c.v_scale + at);
        }
      }
      return k;
    };
    auto pages_of = [&](const Blocks& k, int i, int (&page)[2]) {
      page[0] = __shfl_sync(0xffffffffu, k.page, 2 * i);
      page[1] = __shfl_sync(0xffffffffu, k.page, 2 * i + 1);
    };
    // The open block's rows over this thread's zeros of a tile, in bf16.  Values that are
    // not finite would spread as 0 * inf; they are left to the rows that see
    // them.  (Rolled up: the loop over closed tiles must stay in the
    // instruction cache.)
    auto store_open = [&](unsigned char* dst, const Seg& g, int half, bool value) {
      const int held = g.s.len % kCacheBlock;
      const __nv_bfloat16* tail = static_cast<const __nv_bfloat16*>(value ? P.c.v_tail : P.c.k_tail) +
                                  ((static_cast<long long>(g.b) * 2 + g.s.slot) * P.c.H + g.h) * kCacheBlock * D;
      bool odd = false;
      // This thread's own rows and chunks of the half.
#pragma unroll 1
      for (int e = 0; e < 4 * C::kSlabs; ++e) {
        const int row = r8 + 32 * (e & 1), c = 8 * (e >> 2) + 2 * c16 + ((e >> 1) & 1);
        if (row >= held) continue;
        uint4 x = reorder(__ldg(reinterpret_cast<const uint4*>(tail + row * D) + c));
        if (value) {
          const uint4 y = make_uint4(finite_or_zero(x.x), finite_or_zero(x.y), finite_or_zero(x.z), finite_or_zero(x.w));
          odd = odd || y.x != x.x || y.y != x.y || y.z != x.z || y.w != x.w;
          x = y;
        }
        const int at_row = 64 * half + row;
        *reinterpret_cast<uint4*>(dst + (c / 8) * C::kRowSlab + at_row * 128 + (((c % 8) ^ (at_row & 7)) << 4)) = x;
      }
      if (odd) odd_seg[part_no % 4] = part_no + 1;
    };
    Seg g = seg_at(T, w0, w1 - w0);
    uint32_t tile_no = 0;
    // 16 tiles' blocks, and the 16 after them (loaded 16 tiles early).
    Blocks cur = blocks_at(g, 2 * (g.all.first + g.t0)), nxt = cur;
    int page[2];
    pages_of(cur, 0, page);
    uint4 raw[4][C::kSlabs];
    load(raw, P.c.k_pages, page, g.h);
    // One operand tile a turn, K and V of a tile after one another; the next
    // one's loads are in flight while this one is converted.
    int t = g.t0;
    bool value = false, more = true;
#pragma unroll 1
    while (more && ok) {
      const int j = g.all.first + t, i = (t - g.t0) % 16;
      const int open = g.s.len / kCacheBlock - 2 * j;    // 0 or 1: the open block is that half
      Seg ng = g;
      int nt = t;
      uint4 ahead[4][C::kSlabs];
      if (!value) {
        if (i == 0) nxt = blocks_at(g, 2 * j + 32);
        const float k0 = __shfl_sync(0xffffffffu, cur.ks, 2 * i), k1 = __shfl_sync(0xffffffffu, cur.ks, 2 * i + 1);
        const float v0 = __shfl_sync(0xffffffffu, cur.vs, 2 * i), v1 = __shfl_sync(0xffffffffu, cur.vs, 2 * i + 1);
        if (w == 0 && lane == 0) {
          if (t == g.t0) part_info[part_no % 4] = make_int2(g.t1 - g.t0, g.two ? 2 : 1);
          scales[tile_no % 4] = make_float4(k0, k1, v0, v1);
          if (k0 == 0.0f || k1 == 0.0f) atomicOr(P.err, kErrRange);
        }
      } else {
        ++nt;
        if (nt == g.t1) {
          ng = seg_next(P, g);
          more = ng.left > 0;
          nt = ng.t0;
          if (more) cur = blocks_at(ng, 2 * (ng.all.first + nt));
          pages_of(cur, 0, page);
        } else {
          if (i == 15) cur = nxt;
          pages_of(cur, (i + 1) % 16, page);
        }
      }
      if (more) load(ahead, value ? P.c.k_pages : P.c.v_pages, page, ng.h);
      // Store this one, once the MMAs that read its stage have run.
      const int st = static_cast<int>(at % NS);
      const uint32_t n = at / NS;
      if (n > 0 && !__all_sync(0xffffffffu, mbar_wait(empty(st), (n - 1) & 1u, wait_ns, abort_flag))) {
        ok = false;
        break;
      }
      unsigned char* dst = ring + st * C::kOperand;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int row = r8 + 32 * x;
#pragma unroll
        for (int s = 0; s < C::kSlabs; ++s) {
          uint4 lo, hi;
          e4m3_pairs(raw[x][s].x, lo.x, lo.y);
          e4m3_pairs(raw[x][s].y, lo.z, lo.w);
          e4m3_pairs(raw[x][s].z, hi.x, hi.y);
          e4m3_pairs(raw[x][s].w, hi.z, hi.w);
          unsigned char* to = dst + s * C::kRowSlab + row * 128;
          *reinterpret_cast<uint4*>(to + (((2 * c16) ^ (row & 7)) << 4)) = lo;
          *reinterpret_cast<uint4*>(to + (((2 * c16 + 1) ^ (row & 7)) << 4)) = hi;
        }
      }
      if (open == 0 || open == 1) store_open(dst, g, open, value);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(full(st));
      ++at;
      if (value) {
        ++tile_no;
        if (t + 1 == g.t1) ++part_no;
        g = ng;
        t = nt;
      }
      value = !value;
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int s = 0; s < C::kSlabs; ++s) raw[x][s] = ahead[x][s];
    }
    if (!ok) raise_timeout(P.err, abort_flag);
  } else {
    // ============================================ softmax and output
    asm volatile("setmaxnreg.inc.sync.aligned.u32 160;");
    const int slot = warp / 4, quarter = warp % 4;
    const int r = quarter * 32 + lane;                  // row of the slot (TMEM lane)
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t sbuf = lane_base + C::s_col(slot), obuf = lane_base + C::o_col(slot);
    uint32_t sn = 0, on = 0, parts = 0;                 // S tiles, PVs and parts of this slot so far
    bool ok = true;
    // This slot's rows of a part's Q into shared memory (zeros where there is no row).
    auto load_q = [&](const Seg& g) {
      const CacheRow row = cache_row(P, g.tile * kRows + slot * 128 + r, g.h, g.s.len, g.s.count);
      const uint4* from = reinterpret_cast<const uint4*>(P.q + g.b * P.qb + row.head * P.qh + row.n * P.qn);
      unsigned char* to = qbuf + slot * C::kOperand + r * 128;
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        const uint4 v = row.valid ? from[c] : make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4*>(to + (c / 8) * C::kRowSlab + (((c % 8) ^ (r & 7)) << 4)) = reorder(v);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full(slot));
    };
    uint32_t tile_no = 0;                               // of the CTA
    Seg g = seg_at(T, w0, w1 - w0);
    int part_no = 0;
    // A slot without rows takes no part in an item; the next item of the CTA
    // may have some again.
    if (slot == 0 || g.two) load_q(g);
    while (g.left > 0 && ok) {
      const Seg ng = seg_next(P, g);
      const bool mine = slot == 0 || g.two;
      if (mine) {
        const CacheRow row = cache_row(P, g.tile * kRows + slot * 128 + r, g.h, g.s.len, g.s.count);
        const int n = g.t1 - g.t0;
        float m = -INFINITY, l = 0.0f;
        bool vbad = false;
        for (int t = 0; t < n; ++t) {
          const int j = g.all.first + g.t0 + t;
          if (!__all_sync(0xffffffffu, mbar_wait(s_full(slot), sn & 1u, wait_ns, abort_flag))) {
            ok = false;
            break;
          }
          ++sn;
          tc_fence_after();
          const float4 sc = scales[(tile_no + t) % 4];
          // Halves outside some row's range: scores there become -inf, in
          // TMEM.  (A NaN key scale makes the scores that are seen NaN.)  The
          // halves' loops are rolled up: the code of a whole tile, beside
          // the converting warps', must stay in the instruction cache.
          uint32_t any = 0;
#pragma unroll 1
          for (int x = 0; x < 2; ++x) {
            const int kb = j * kTile + 64 * x;
            const float ks = x ? sc.y : sc.x, vs = x ? sc.w : sc.z;
            const int lo = row.see.lo - kb, hi = ks == 0.0f ? -1 : row.see.end - 1 - kb;
            const bool live = lo < 64 && hi >= 0 && row.see.end > 0;
            vbad = vbad || (live && isnan(vs));
            if (!__any_sync(0xffffffffu, live)) continue;
            any |= 1u << x;
            if (!isnan(ks) && __all_sync(0xffffffffu, live && lo <= 0 && hi >= 63)) continue;
            const float seen = isnan(ks) ? ks : 0.0f;
#pragma unroll 1
            for (int c0 = 0; c0 < 64; c0 += 32) {
              uint32_t s32[32];
              tmem_ld32(sbuf + 64 * x + c0, s32);
#pragma unroll
              for (int c = 0; c < 32; ++c)
                s32[c] = live && c0 + c >= lo && c0 + c <= hi ? __float_as_uint(__uint_as_float(s32[c]) + seen) : 0xff800000u;
              tmem_st32(sbuf + 64 * x + c0, s32);
            }
            tmem_st_wait();
          }
          // Pass 1: the row's maximum.
          float pm = -INFINITY;
#pragma unroll 1
          for (int x = 0; x < 2; ++x) {
            if (!(any >> x & 1u)) continue;
            uint32_t s64[64];
            tmem_ld64(sbuf + 64 * x, s64);
            float sv[64];
#pragma unroll
            for (int c = 0; c < 64; ++c) sv[c] = __uint_as_float(s64[c]);
            pm = fmaxf(pm, max64(sv) * key_factor(P.scale_log2, x ? sc.y : sc.x));
          }
          // The maximum is raised lazily: O is rescaled only when it grows by
          // more than 2^8 (by anything under scales so large that P times 2^8
          // would leave float32).
          float f = 1.0f;
          const float slack = fmaxf(sc.z, sc.w) > 0x1p100f ? 0.0f : 8.0f;
          if (pm > m + slack) {
            f = m == -INFINITY ? 1.0f : ex2_ftz(m - pm);
            l *= f;
            m = pm;
          }
          const float nm = m == -INFINITY ? 0.0f : -m;
          // Pass 2: P = 2^(s c2 - m + ev) over the first 64 columns of S.
#pragma unroll 1
          for (int x = 0; x < 2; ++x) {
            uint32_t pk[32];
            if (any >> x & 1u) {
              const float vs0 = x ? sc.w : sc.z;
              const float vs = isnan(vs0) ? 1.0f : vs0;
              const float c2 = key_factor(P.scale_log2, x ? sc.y : sc.x);
              const uint64_t c22 = pack2(c2, c2), off = pack2(nm + pow2_log(vs), nm + pow2_log(vs));
              uint32_t s64[64];
              tmem_ld64(sbuf + 64 * x, s64);
              uint64_t a0 = 0, a1 = 0;
#pragma unroll
              for (int c = 0; c < 64; c += 4) {
                float p0, p1, p2, p3;
                unpack2(fma2(pack2(__uint_as_float(s64[c]), __uint_as_float(s64[c + 1])), c22, off), p0, p1);
                unpack2(fma2(pack2(__uint_as_float(s64[c + 2]), __uint_as_float(s64[c + 3])), c22, off), p2, p3);
                p0 = ex2_ftz(p0);
                p1 = ex2_ftz(p1);
                p2 = ex2_ftz(p2);
                p3 = ex2_ftz(p3);
                pk[c / 2] = pack_bf16x2(p0, p1);
                pk[c / 2 + 1] = pack_bf16x2(p2, p3);
                a0 = add2(a0, pack2(p0, p1));
                a1 = add2(a1, pack2(p2, p3));
              }
              float s0, s1;
              unpack2(add2(a0, a1), s0, s1);
              l = fmaf(s0 + s1, pow2_inv(vs), l);
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e) pk[e] = 0u;
            }
            tmem_st32(sbuf + 32 * x, pk);
          }
          // Every PV of the slot is observed in order: a parity wait is at
          // most one phase behind.
          if (t > 0) {
            if (!__all_sync(0xffffffffu, mbar_wait(o_done(slot), on & 1u, wait_ns, abort_flag))) {
              ok = false;
              break;
            }
            ++on;
            tc_fence_after();
          }
          if (t > 0 && __any_sync(0xffffffffu, f != 1.0f)) {
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
              uint32_t o32[32];
              tmem_ld32(obuf + c0, o32);
#pragma unroll
              for (int e = 0; e < 32; ++e) o32[e] = __float_as_uint(__uint_as_float(o32[e]) * f);
              tmem_st32(obuf + c0, o32);
            }
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full(slot));
        }
        if (!ok) break;
        // Every QK of the part has run: the next part's Q, while its last PV does.
        if (!__all_sync(0xffffffffu, mbar_wait(q_free(slot), parts & 1u, wait_ns, abort_flag))) {
          ok = false;
          break;
        }
        ++parts;
        if (ng.left > 0 && (slot == 0 || ng.two)) load_q(ng);
        if (!__all_sync(0xffffffffu, mbar_wait(o_done(slot), on & 1u, wait_ns, abort_flag))) {
          ok = false;
          break;
        }
        ++on;
        tc_fence_after();
        // ---- output
        const bool whole = g.t0 == 0 && g.t1 == g.all.n;
        const bool odd = odd_seg[part_no % 4] == part_no + 1;
        const float inv = whole ? (l == 0.0f ? 0.0f : 1.0f / l) : 1.0f;
        char* orow = P.o + g.b * P.ob + row.head * P.oh + row.n * P.on;
        const long long part_row = (2ll * blockIdx.x + (g.first ? 0 : 1)) * kRows + slot * 128 + r;
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
          uint32_t o32[32];
          tmem_ld32(obuf + c0, o32);
          float v[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            // Back to the channels' order.
            const int from = (e & ~3) | ((e & 1) << 1) | ((e & 2) >> 1);
            v[e] = vbad ? __int_as_float(0x7fffffff) : __uint_as_float(o32[from]);
          }
          if (odd && row.valid) {
            const int first = g.s.len / kCacheBlock * kCacheBlock;
            const __nv_bfloat16* tail = static_cast<const __nv_bfloat16*>(P.c.v_tail) +
                                        ((static_cast<long long>(g.b) * 2 + g.s.slot) * P.c.H + g.h) * kCacheBlock * D + c0;
            for (int key = max(first, row.see.lo); key < row.see.end; ++key)
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const float x = __bfloat162float(tail[(key - first) * D + e]);
                if (!isfinite(x)) v[e] += x;
              }
          }
          if (row.valid && whole) {
#pragma unroll
            for (int e = 0; e < 32; e += 8)
              *reinterpret_cast<uint4*>(orow + 2 * (c0 + e)) =
                  make_uint4(pack_bf16x2(v[e] * inv, v[e + 1] * inv), pack_bf16x2(v[e + 2] * inv, v[e + 3] * inv),
                             pack_bf16x2(v[e + 4] * inv, v[e + 5] * inv), pack_bf16x2(v[e + 6] * inv, v[e + 7] * inv));
          } else if (row.valid) {
            float4* to = reinterpret_cast<float4*>(P.part_o + part_row * D + c0);
#pragma unroll
            for (int e = 0; e < 32; e += 4) to[e / 4] = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
          }
        }
        if (row.valid && whole && P.lse != nullptr)
          P.lse[(static_cast<long long>(g.b) * P.Hq + row.head) * P.N + row.n] = (m + log2f(l)) * 0.6931471805599453f;
        if (row.valid && !whole) P.part_ml[part_row] = make_float2(m, l);
        tc_fence_before();
      } else if (ng.left > 0 && ng.two) {
        // No rows in this item: its slot's Q buffer is idle.
        load_q(ng);
      }
      tile_no += g.t1 - g.t0;
      ++part_no;
      g = ng;
    }
    if (!ok) raise_timeout(P.err, abort_flag);
    // No TMEM access of this warp may be in flight at the teardown.
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
    tmem_st_wait();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
}

// Merges the parts of the items that more than one CTA worked on: CTA (item,
// 32 rows), a warp per row.
template <int D>
__global__ void __launch_bounds__(256) cache_tc_merge_kernel(const __grid_constant__ TcParams T, int grid) {
  const CacheAttnParams& P = T.a;
  const int item = blockIdx.x / (kRows / 32), chunk = blockIdx.x % (kRows / 32);
  const int tile = item % P.tiles, bh = item / P.tiles;
  const int b = bh / P.c.H, h = bh % P.c.H;
  const int* pre = T.tile_prefix + static_cast<long long>(b) * (P.tiles + 1);
  const int n = __ldg(pre + tile + 1) - __ldg(pre + tile);
  if (n == 0) return;
  const long long total = __ldg(T.seq_prefix + P.c.B);
  const long long ctas = work_ctas(total, grid);
  const long long w0 = __ldg(T.seq_prefix + b) + static_cast<long long>(h) * __ldg(pre + P.tiles) + __ldg(pre + tile);
  // CTA c holds tiles [total c / ctas, total (c + 1) / ctas).
  const int c0 = static_cast<int>(((w0 + 1) * ctas + total - 1) / total) - 1;
  const int c1 = static_cast<int>(((w0 + n) * ctas + total - 1) / total) - 1;
  if (c0 == c1) return;
  bool bad = false;
  const SeqInfo s = seq_info(P, b, &bad);
  const int lane = threadIdx.x % 32;
  constexpr int C = D / 32;
  // The item is the first part of every CTA but, perhaps, its first one's.
  const int first_part = total * c0 / ctas >= w0 ? 0 : 1;
  for (int i = threadIdx.x / 32; i < 32; i += 8) {
    const int r = chunk * 32 + i;
    const CacheRow row = cache_row(P, tile * kRows + r, h, s.len, s.count);
    if (!row.valid) continue;
    float m = -INFINITY;
    for (int c = c0; c <= c1; ++c)
      m = fmaxf(m, P.part_ml[(2ll * c + (c == c0 ? first_part : 0)) * kRows + r].x);
    float l = 0.0f, acc[C] = {};
    for (int c = c0; c <= c1; ++c) {
      const long long at = (2ll * c + (c == c0 ? first_part : 0)) * kRows + r;
      const float2 p = P.part_ml[at];
      if (p.y == 0.0f) continue;
      const float f = p.x == -INFINITY ? 1.0f : ex2_ftz(p.x - m);
      l = fmaf(p.y, f, l);
      const float* from = P.part_o + at * D + lane * C;
#pragma unroll
      for (int e = 0; e < C; ++e) acc[e] = fmaf(from[e], f, acc[e]);
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    char* to = P.o + b * P.ob + row.head * P.oh + row.n * P.on + 2 * lane * C;
#pragma unroll
    for (int e = 0; e < C; e += 2)
      *reinterpret_cast<uint32_t*>(to + 2 * e) = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
    if (lane == 0 && P.lse != nullptr)
      P.lse[(static_cast<long long>(b) * P.Hq + row.head) * P.N + row.n] = (m + log2f(l)) * 0.6931471805599453f;
  }
}

struct Layout {
  int tiles;
  size_t part_o, part_ml, tile_prefix, seq_prefix, total;
};
Layout layout_of(const CacheAttnArgs& a, int num_sms) {
  Layout L;
  const long long rows = static_cast<long long>(a.Hq / a.cache.H) * a.N;
  L.tiles = static_cast<int>((rows + kRows - 1) / kRows);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += align256(bytes);
    return o;
  };
  const size_t parts = static_cast<size_t>(num_sms) * 2 * kRows;
  L.part_o = take(parts * a.cache.d * sizeof(float));
  L.part_ml = take(parts * sizeof(float2));
  L.tile_prefix = take(static_cast<size_t>(a.cache.B) * (L.tiles + 1) * sizeof(int));
  L.seq_prefix = take((static_cast<size_t>(a.cache.B) + 1) * sizeof(long long));
  L.total = off;
  return L;
}

template <int D>
cudaError_t launch_d(const Ctx& c, const TcParams& T) {
  const cudaError_t e = cudaFuncSetAttribute(cache_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, CT<D>::kSmem);
  if (e != cudaSuccess) return e;
  cache_plan_kernel<<<1, 1024, 0, c.stream>>>(T);
  cache_tc_kernel<D><<<c.num_sms, kThreads, CT<D>::kSmem, c.stream>>>(T);
  const long long items = static_cast<long long>(T.a.c.B) * T.a.c.H * T.a.tiles;
  cache_tc_merge_kernel<D><<<static_cast<unsigned>(items * (kRows / 32)), 256, 0, c.stream>>>(T, c.num_sms);
  return cudaGetLastError();
}

}  // namespace

size_t cache_attn_tc_ws_bytes(const CacheAttnArgs& a, int num_sms) { return layout_of(a, num_sms).total; }

cudaError_t launch_cache_attn_tc(const Ctx& c, const CacheAttnArgs& a, CacheAttnParams P) {
  const Layout L = layout_of(a, c.num_sms);
  char* ws = static_cast<char*>(a.workspace);
  TcParams T;
  P.tiles = L.tiles;
  P.splits = 0;
  P.part_o = reinterpret_cast<float*>(ws + L.part_o);
  P.part_ml = reinterpret_cast<float2*>(ws + L.part_ml);
  T.a = P;
  T.tile_prefix = reinterpret_cast<int*>(ws + L.tile_prefix);
  T.seq_prefix = reinterpret_cast<long long*>(ws + L.seq_prefix);
  return a.cache.d == 128 ? launch_d<128>(c, T) : launch_d<64>(c, T);
}

}  // namespace salad
