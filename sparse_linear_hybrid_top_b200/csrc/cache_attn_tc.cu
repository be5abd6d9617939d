// cache_attn_tc.cu -- attention of many query rows (chunks of latent frames)
// over the 8-bit block cache, on tcgen05 tensor cores.
//
// Bound by the tensor pipe (4 d operations per query row, key and head) and,
// as tightly, by the exponentials: a 128 x 128 tile of scores takes its two
// products 1024 cycles and its 16384 exponentials 1024 (16 lanes a cycle), and
// the shared memory carries 160 KB of codes and operands for it, 1250 cycles.
// A work item is 256 query rows of one sequence and key head: two 128-row slots
// that share every key tile, so each tile of codes is converted once per 256
// rows.  A key tile is 128 keys (two blocks).
//
// Operands are fp16, in which every e4m3 code is exact and converts in one
// instruction per pair (the bf16 route takes nine per four codes; the ALU
// pipe runs both at 16 lanes a cycle).  A query row is scaled by a power of
// two to a largest magnitude in [2^14, 2^15): its bf16 values stay exact down
// to 2^-28 of that, and those below err by 2^-39 of it.  The open block's bf16
// rows are scaled like a closed block's.  Key scales and the row's join the
// softmax scale.  P, times the value block's scale, is at most 2^15 in fp16:
// rounded by 2^-11, or, 2^25 and more below the row's largest such product, by
// 2^-36 of that (see the softmax for how its maximum and the row sum are kept
// apart).
//
// Warp roles (512 threads, one CTA per SM):
//   warps 0..3, 4..7   softmax and output of slots 0 and 1, a row per thread
//                      (warp w on TMEM lane quarter w % 4); they also load
//                      their slot's rows of Q
//   warps 8..11        codes -> fp16: from a ring of bulk-copied code tiles
//                      to swizzled operand tiles
//   warps 12, 14       the MMA issuers of slots 0 and 1 (12 holds the TMEM)
//   warp 13            bulk copies of code tiles; it also passes the closed
//                      blocks' scales to the softmax warps
//   warp 15            nothing: it fills the warpgroup that gives registers
// While the tensor pipe runs one slot's PV(t) and QK(t+1), the other slot's
// softmax runs.  P overwrites S in TMEM.
//
// Measured (d = 128): 4680 query tokens (three frames of 1560) on 18720 keys,
// their own among them and masked by frame, 12 heads, 562 to 568 us; 3600 on 100800,
// 8 heads, 1.74 ms: 870 and 855 TFLOP/s, 0.52 of the burst rate of a large matrix
// product.  A pair of tiles takes 1.75 times its products' cycles.  No unit bounds it alone (timed with parts left
// out: without the exponentials 0.85 of the time, without the conversion 0.9,
// with an eighth of the products 0.83): the way of a slot, S - maximum -
// exponentials - P - PV - QK, is as long as two slots' products, and TMEM has no
// room for a third.  For 3600 on 50400 keys the turns at the exponentials (see
// the softmax) brought 970 us to 857; 16 softmax warps, two to a row, took 871
// to 891.  An item of 128 rows and fewer leaves one slot idle, and the other has
// nothing beside its steps: 65 rows on 31200 keys of 12 heads take 77 us, where
// reading the cache takes 14.6 (the tensor pipe is active for 16% of it).
//
// Balance: lengths are known on the device only, and tiles per item differ by
// frame.  A first launch sums the items' tiles; every CTA then takes an equal
// run of tiles, which may begin and end inside an item.  An item that one CTA
// holds whole is written at once; the others leave float32 parts (two per
// CTA at most), merged by a last launch.  Every CTA notes the item that its run
// begins inside, so that the merge looks at those alone.
#include <cstring>

#include "cache_attn.cuh"

namespace salad {
namespace {

constexpr int kRows = 256;            // query rows of an item
constexpr int kTile = 128;            // keys of a tile
constexpr int kThreads = 512;
// What a row's products of weight and scale are counted against is raised to
// 2^kBaseP where one passes 2^kTopP: they lie between the two, at their largest.
constexpr float kBaseP = kTopP - 4.0f;
// Registers of a thread: at launch, and the warpgroups' shares after it (two
// of softmax warps, the converting one, the last).  Taking more than the
// others give would wait forever.
constexpr int kRegsLaunch = 128, kRegsSoft = 160, kRegsConvert = 112, kRegsLast = 80;
static_assert(2 * kRegsSoft + kRegsConvert + kRegsLast <= 4 * kRegsLaunch, "register shares");
static_assert(kThreads * kRegsLaunch == 65536 && kThreads == 4 * 128, "the launch holds the register file");

template <int D>
struct CT {
  static constexpr int kSlabs = D / 64;
  static constexpr int kRowSlab = 128 * 128;            // 128 rows of 128 bytes
  static constexpr int kOperand = kSlabs * kRowSlab;    // 128 rows of Q, K or V
  static constexpr int kStages = 4;                     // operand tiles
  static constexpr int kRaw = 128 * D;                  // codes of an operand tile
  static constexpr int kRaws = D == 128 ? 2 : 4;
  static constexpr int kBarBytes = 384;
  static constexpr int kScaleBytes = 8 * 16 + 8 * 8;    // scales of eight tiles (K, K, V, V), eight parts' (tiles, slots)
  static constexpr int kSegBytes = 8 * 64;              // the softmax warps' current parts
  static constexpr int kUsed = (2 + kStages) * kOperand + kRaws * kRaw + kBarBytes + kScaleBytes + kSegBytes;
  // More than half of the SM's shared memory: one CTA (and its 512 TMEM columns) per SM.
  static constexpr int kSmem = kUsed > 120 * 1024 ? kUsed : 120 * 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
  __host__ __device__ static constexpr uint32_t o_col(int slot) { return slot ? D : 0; }
  __host__ __device__ static constexpr uint32_t s_col(int slot) { return 2 * D + (slot ? 128 : 0); }
  static constexpr uint32_t kCols = 512;
};

// The item that a CTA's run begins inside (tile < 0: it begins with one).
struct Inside {
  long long start;            // the item's first tile, of all
  int b, h, tile, n;          // n: its tiles
};

struct TcParams {
  CacheAttnParams a;          // tiles: items of a (sequence, key head)
  int* tile_prefix;           // [B][tiles + 1]
  long long* seq_prefix;      // [B + 1], tiles of all heads of the sequences before
  Inside* inside;             // [CTAs]
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
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
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
    if (T.seq_prefix[mid] <= w) lo = mid; else hi = mid;
  }
  g.b = lo;
  const int* pre = T.tile_prefix + static_cast<long long>(g.b) * (P.tiles + 1);
  const int per = pre[P.tiles];
  const long long rem = w - T.seq_prefix[g.b];
  g.h = static_cast<int>(rem / per);
  const int at = static_cast<int>(rem % per);
  lo = 0;
  hi = P.tiles;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (pre[mid] <= at) lo = mid; else hi = mid;
  }
  g.tile = lo;
  g.left = left;
  g.first = true;
  seg_open(P, g);
  g.t0 = at - pre[lo];
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

// Maximum of 64 values by a tree of three-input maxima (64 -> 22 -> 8 -> 3 -> 1).
__device__ __forceinline__ float max64(const uint32_t* u) {
  auto v = [&](int i) { return __uint_as_float(u[i]); };
  float a[22];
#pragma unroll
  for (int i = 0; i < 21; ++i) a[i] = fmax3(v(3 * i), v(3 * i + 1), v(3 * i + 2));
  a[21] = v(63);
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

// Asynchronous TMEM load of 32 columns; the registers hold it after tmem_arrived.
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : SALAD_R8(r, 0), SALAD_R8(r, 8), SALAD_R8(r, 16), SALAD_R8(r, 24)
      : "r"(taddr)
      : "memory");
}
#define SALAD_RW8(a, o) "+r"(a[o + 0]), "+r"(a[o + 1]), "+r"(a[o + 2]), "+r"(a[o + 3]), \
                        "+r"(a[o + 4]), "+r"(a[o + 5]), "+r"(a[o + 6]), "+r"(a[o + 7])
// Waits for every load of this thread.
__device__ __forceinline__ void tmem_arrived() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// Keeps uses of r behind the wait before it.
__device__ __forceinline__ void pin32(uint32_t* r) {
  asm volatile("" : SALAD_RW8(r, 0), SALAD_RW8(r, 8));
  asm volatile("" : SALAD_RW8(r, 16), SALAD_RW8(r, 24));
}

// MMAs and commits by one elected thread of a converged warp.  (The same
// thread each time: commits track that thread's operations.)
__device__ __forceinline__ void mma_ss_elected(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ts_elected(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void commit_elected(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(bar)
      : "memory");
}

// The power of two that brings magnitudes up to bf16 bits `top` (finite) to
// at most 448: a closed block's rule.
__device__ __forceinline__ float tail_scale(uint32_t top) {
  int e = static_cast<int>(top >> 7) - 127 - 8 + ((top & 127u) > 96u ? 1 : 0);
  e = e < -100 ? -100 : e;
  return __int_as_float((127 + e) << 23);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) cache_tc_kernel(const __grid_constant__ TcParams T) {
  using C = CT<D>;
  constexpr int NS = C::kStages, NR = C::kRaws;
  const CacheAttnParams& P = T.a;
  extern __shared__ __align__(1024) unsigned char smem[];
  if (reinterpret_cast<uintptr_t>(smem) & 1023u) {
    if (threadIdx.x == 0) atomicOr(P.err, kErrLayout);
    return;
  }
  // Every CTA is on an SM by then; the merge's follow as these end.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long long total = T.seq_prefix[P.c.B];
  const long long ctas = work_ctas(total, gridDim.x);
  if (blockIdx.x >= ctas) return;
  const long long w0 = total * blockIdx.x / ctas, w1 = total * (blockIdx.x + 1) / ctas;
  if (w0 >= w1) return;

  unsigned char* qbuf = smem;                               // [2 slots][d-slab][128 rows]
  unsigned char* ring = qbuf + 2 * C::kOperand;             // [NS][d-slab][128 rows]
  unsigned char* raws = ring + NS * C::kOperand;            // [NR][128 keys][d codes]
  uint64_t* bars = reinterpret_cast<uint64_t*>(raws + NR * C::kRaw);
  // full[NS] empty[NS] raw_full[NR] raw_empty[NR] q_full[2] q_free[2] s_full[2] p_half[2] p_full[2] o_done[2] drain[2] turn[8] open_max
  auto bar = [&](int i) { return smem_u32(bars + i); };
  auto full = [&](int i) { return bar(i); };
  auto empty = [&](int i) { return bar(NS + i); };
  auto raw_full = [&](int i) { return bar(2 * NS + i); };
  auto raw_empty = [&](int i) { return bar(2 * NS + NR + i); };
  constexpr int B0 = 2 * NS + 2 * NR;
  auto q_full = [&](int i) { return bar(B0 + i); };
  auto q_free = [&](int i) { return bar(B0 + 2 + i); };
  auto s_full = [&](int i) { return bar(B0 + 4 + i); };
  auto p_half = [&](int i) { return bar(B0 + 6 + i); };
  auto p_full = [&](int i) { return bar(B0 + 8 + i); };
  auto o_done = [&](int i) { return bar(B0 + 10 + i); };
  auto drain = [&](int i) { return bar(B0 + 12 + i); };
  auto turn = [&](int w) { return bar(B0 + 14 + w); };      // of softmax warp w
  const uint32_t open_max = bar(B0 + 22);                   // the converting warps have their part of the open block
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + B0 + 23);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  // odd_seg[i % 8] = i + 1: part i's open block holds a value that is not finite.
  volatile int* odd_seg = abort_flag + 1;
  // Largest magnitudes of the open block's finite keys and values (bf16 bits, two
  // to a word), of each converting warp; two open blocks in turn.
  uint32_t* open_tops = reinterpret_cast<uint32_t*>(const_cast<int*>(odd_seg) + 8);
  static_assert((B0 + 23) * 8 + 4 + 4 + 32 + 32 <= C::kBarBytes, "barrier region");
  // Scales of tile i's two blocks in entry i % 8: of the keys (0: no page, its
  // keys do not count), then of the values.  Warp 13 writes them (the open
  // block's: warp 8, with its keys) with the bulk copy of the tile's keys: kRaws operand tiles before these are converted,
  // and kStages before the MMAs of what they replace, so at most five tiles
  // before the softmax reads them.
  float4* scales = reinterpret_cast<float4*>(reinterpret_cast<unsigned char*>(bars) + C::kBarBytes);
  // Tiles and slots of part i in entry i % 8, for the issuer: written and read
  // like the scales (a part has a tile at least).
  int2* part_info = reinterpret_cast<int2*>(scales + 8);
  // A softmax warp's current part: registers hold a row of scores instead.
  static_assert(sizeof(Seg) <= 64 && sizeof(Seg) % 4 == 0, "part record");
  volatile int* seg_mem = reinterpret_cast<volatile int*>(part_info + 8) + 16 * (threadIdx.x / 32 % 8);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const unsigned long long wait_ns = P.wait_ns;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(full(i), 4);      // the four converting warps
      mbar_init(empty(i), 2);     // the two issuers
    }
    for (int i = 0; i < NR; ++i) {
      mbar_init(raw_full(i), 1);
      mbar_init(raw_empty(i), 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full(i), 4);    // the slot's four softmax warps
      mbar_init(q_free(i), 1);
      mbar_init(s_full(i), 1);
      mbar_init(p_half(i), 4);
      mbar_init(p_full(i), 4);
      mbar_init(o_done(i), 1);
    }
    for (int i = 0; i < 2; ++i) mbar_init(drain(i), 1);
    for (int i = 0; i < 8; ++i) mbar_init(turn(i), 1);
    mbar_init(open_max, 4);
    *abort_flag = 0;
    for (int i = 0; i < 8; ++i) odd_seg[i] = 0;
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

  // Every warp of every warpgroup passes one of these three.
  if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLast));
    if (warp == 12 || warp == 14) {
      // ============================================ MMA issuer of a slot
      // An issuer a slot: every barrier that a warp looks at costs it some 300
      // cycles beside the converting warps' traffic, and one warp with both
      // slots' six a tile was the slowest of all.  The whole warp walks through
      // the tiles, so that descriptors stay in uniform registers; one elected
      // thread issues.
      const int slot = warp == 12 ? 0 : 1;
      constexpr uint32_t idesc_qk = idesc_f16(128, 128, false, false);
      constexpr uint32_t idesc_pv = idesc_f16(128, D, false, true);
      const uint32_t ring_base = smem_u32(ring);
      const uint64_t qd = sdesc_sw128(smem_u32(qbuf) + slot * C::kOperand, 16, 1024);
      const uint64_t kd0 = sdesc_sw128(ring_base, 16, 1024);
      const uint64_t vd0 = sdesc_sw128(ring_base, C::kRowSlab, 1024);
      constexpr uint64_t kStageStep = C::kOperand >> 4;
      const uint32_t s_at = tmem + C::s_col(slot), p_at = s_at, o_at = tmem + C::o_col(slot);
      // Operand stage and phase of the next K or V, in the order K0 V0 K1 V1 ...
      int st = 0;
      uint32_t ph = 0;
      uint32_t qn = 0, pn = 0;              // phases of q_full, and of p_half and p_full
      bool ok = true;
      auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait_spin(bar, parity, wait_ns, abort_flag));
      };
      // This slot is done with the stage (once the MMAs so far are).
      auto next_stage = [&](bool mine) {
        if (mine) commit_elected(empty(st));
        else if (lane == 0) mbar_arrive(empty(st));
        if (++st == NS) {
          st = 0;
          ph ^= 1u;
        }
      };
      auto issue_qk = [&](int stage) {
        const uint64_t kd = kd0 + static_cast<uint64_t>(stage) * kStageStep;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint64_t off = static_cast<uint64_t>(((ks / 4) * C::kRowSlab + (ks % 4) * 32) >> 4);
          mma_ss_elected(s_at, qd + off, kd + off, idesc_qk, ks > 0 ? 1u : 0u);
        }
        commit_elected(s_full(slot));
      };
      long long left = w1 - w0;
      for (int part_no = 0; left > 0; ++part_no) {
        if (!(ok = wait(full(st), ph))) break;
        const int2 info = part_info[part_no % 8];
        const int n = info.x;
        const bool mine = slot < info.y;
        if (mine) {
          if (!(ok = wait(q_full(slot), qn))) break;
          qn ^= 1u;
          tc_fence_after();
          issue_qk(st);
          if (n == 1) commit_elected(q_free(slot));
        }
        next_stage(mine);
        for (int t = 0; t < n; ++t) {
          // V(t) in this stage, K(t + 1) in the next; both are there before P,
          // as a rule.
          const int kst = st + 1 == NS ? 0 : st + 1;
          const uint32_t kph = st + 1 == NS ? ph ^ 1u : ph;
          const uint64_t vd = vd0 + static_cast<uint64_t>(st) * kStageStep;
          if (!(ok = wait(full(st), ph) && (t + 1 == n || wait(full(kst), kph)))) break;
          if (mine) {
            auto pv = [&](int ks, uint32_t acc) {   // 16 keys
              mma_ts_elected(o_at, p_at + ks * 8, vd + static_cast<uint64_t>((ks * 2048) >> 4), idesc_pv, acc);
            };
            // Half a tile's P at a time.
            if (!(ok = wait(p_half(slot), pn))) break;
            tc_fence_after();
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) pv(ks, ks > 0 || t > 0 ? 1u : 0u);
            if (!(ok = wait(p_full(slot), pn))) break;
            pn ^= 1u;
            tc_fence_after();
#pragma unroll
            for (int ks = 4; ks < 8; ++ks) pv(ks, 1u);
            if (t + 1 == n) {
              commit_elected(o_done(slot));
            } else {
              issue_qk(kst);                        // over this tile's P: behind its PV in issue order
              if (t + 2 == n) commit_elected(q_free(slot));
            }
          }
          next_stage(mine);
          if (t + 1 < n) next_stage(mine);
        }
        if (!ok) break;
        left -= n;
      }
      if (!ok && lane == 0) raise_timeout(P.err, abort_flag);
      commit_elected(drain(slot));
      if (!mbar_wait_poll(drain(slot), 0, wait_ns, nullptr) && lane == 0) atomicOr(P.err, kErrTimeout);
    } else if (warp == 13) {
      // ===================================================== bulk copies
      struct Blocks {                             // of 32 blocks, one per lane
        int page;                                 // -2: not closed
        float ks, vs;
      };
      // A table entry that is no page reads page 0; a key scale of 0 masks it.  So
      // does the block of the item's first tile that lies before its rows' window:
      // its page may have been given back.
      auto blocks_at = [&](const Seg& g, int blk) {
        Blocks k{-2, 1.0f, 1.0f};
        const int lo =
            cache_visible(g.s.len - g.s.count + g.tile * kRows / P.group, g.s.len, g.s.count, P.frame, P.window).lo;
        if (blk + lane < lo / kCacheBlock) {
          k.page = 0;
          k.ks = 0.0f;
        } else if (blk + lane < g.s.len / kCacheBlock) {
          k.page = cache_page(__ldg(P.c.page_table + static_cast<long long>(g.b) * P.c.blocks + blk + lane), P.c.pages);
          if (k.page < 0) {
            k.page = 0;
            k.ks = 0.0f;
            atomicOr(P.err, kErrRange);
          } else {
            const long long at = static_cast<long long>(k.page) * P.c.H + g.h;
            k.ks = __ldg(P.c.k_scale + at);
            k.vs = __ldg(P.c.v_scale + at);
          }
        }
        return k;
      };
      unsigned long long at = 0;                  // operand tiles so far
      uint32_t tile_no = 0;                       // key tiles so far
      int part_no = 0;
      bool ok = true;
      for (Seg g = seg_at(T, w0, w1 - w0); g.left > 0 && ok; g = seg_next(P, g), ++part_no) {
        // 16 tiles' blocks, and the 16 after them (loaded 16 tiles early).
        Blocks cur{}, nxt = blocks_at(g, 2 * (g.all.first + g.t0));
#pragma unroll 1
        for (int t = g.t0; t < g.t1 && ok; ++t, ++tile_no) {
          const int j = g.all.first + t, i = (t - g.t0) % 16;
          if (i == 0) {
            cur = nxt;
            nxt = blocks_at(g, 2 * j + 32);
          }
          const float4 sc = make_float4(__shfl_sync(0xffffffffu, cur.ks, 2 * i), __shfl_sync(0xffffffffu, cur.ks, 2 * i + 1),
                                  __shfl_sync(0xffffffffu, cur.vs, 2 * i), __shfl_sync(0xffffffffu, cur.vs, 2 * i + 1));
          const int p0 = __shfl_sync(0xffffffffu, cur.page, 2 * i), p1 = __shfl_sync(0xffffffffu, cur.page, 2 * i + 1);
#pragma unroll 1
          for (int value = 0; value < 2 && ok; ++value, ++at) {
            const int rs = static_cast<int>(at % NR);
            const unsigned long long n = at / NR;
            ok = n == 0 || __all_sync(0xffffffffu, mbar_wait_poll(raw_empty(rs), static_cast<uint32_t>(n - 1) & 1u, wait_ns, abort_flag));
            if (!ok) break;
            if (lane == 0) {
              if (!value) {
                if (t == g.t0) part_info[part_no % 8] = make_int2(g.t1 - g.t0, g.two ? 2 : 1);
                scales[tile_no % 8] = sc;
              }
              constexpr uint32_t bytes = kCacheBlock * D;
              const unsigned char* pages = value ? P.c.v_pages : P.c.k_pages;
              const uint32_t dst = smem_u32(raws) + rs * C::kRaw;
              mbar_arrive_expect_tx(raw_full(rs), (p0 >= 0 ? bytes : 0u) + (p1 >= 0 ? bytes : 0u));
              if (p0 >= 0) bulk_load(dst, pages + (static_cast<long long>(p0) * P.c.H + g.h) * bytes, bytes, raw_full(rs));
              if (p1 >= 0) bulk_load(dst + bytes, pages + (static_cast<long long>(p1) * P.c.H + g.h) * bytes, bytes, raw_full(rs));
            }
            __syncwarp();
          }
        }
      }
      if (!ok) raise_timeout(P.err, abort_flag);
      // No bulk copy may be in flight at the exit.
      if (lane == 0) {
        for (uint32_t i = 0; i < NR && i < at; ++i) {
          const uint32_t last = static_cast<uint32_t>((at - 1 - i) / NR);            // turns of raw slot i, less one
          if (!mbar_wait_poll(raw_full(static_cast<int>(i)), last & 1u, wait_ns, nullptr)) atomicOr(P.err, kErrTimeout);
        }
      }
    }
  } else if (warp >= 8) {
    // ================================================== codes -> fp16
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsConvert));
    const int w = warp - 8;
    constexpr int CPR = D / 16;                 // 16-code chunks of a row
    constexpr int RU = 32 / CPR;                // rows of one warp step
    constexpr int kSteps = 128 / (4 * RU);
    const int c = lane % CPR, row0 = w * RU + lane / CPR;
    // Which eight codes of a lane's sixteen go first: chosen so that neither
    // the 8-byte reads nor the swizzled 16-byte writes meet in a bank.
    const int swap = D == 128 ? (c >> 2) ^ (row0 & 1) : (row0 >> 1) & 1;
    const int from0 = row0 * D + 16 * c + 8 * swap, from1 = row0 * D + 16 * c + 8 * (swap ^ 1);
    const int to = (c / 4) * C::kRowSlab + row0 * 128, ch = (2 * c) & 7;
    const int to0 = to + (((ch + swap) ^ (row0 & 7)) << 4), to1 = to + (((ch + (swap ^ 1)) ^ (row0 & 7)) << 4);
    bool ok = true;
    Seg g = seg_at(T, w0, w1 - w0);
    int part_no = 0;
    uint32_t tile_no = 0;
    if (w == 0 && lane == 0) T.inside[blockIdx.x] = Inside{w0 - g.t0, g.b, g.h, g.t0 > 0 ? g.tile : -1, g.all.n};
    int st = 0, rs = 0;
    uint32_t sph = 1, rph = 0;                  // parities of empty (first turn passes) and raw_full
    uint32_t opens = 0;                         // open blocks so far
    float open_vs = 1.0f;                       // the values' scale of the last one
    while (g.left > 0 && ok) {
#pragma unroll 1
      for (int o = 2 * g.t0; o < 2 * g.t1 && ok; ++o) {
        const bool value = o & 1;
        const int j = g.all.first + (o >> 1);
        const int closed = g.s.len / kCacheBlock - 2 * j;   // of the tile's blocks: 2 and more, 1, 0 and less
        if (!__all_sync(0xffffffffu, mbar_wait_poll(raw_full(rs), rph, wait_ns, abort_flag) &&
                                         mbar_wait_poll(empty(st), sph, wait_ns, abort_flag))) {
          ok = false;
          break;
        }
        const unsigned char* src = raws + rs * C::kRaw;
        unsigned char* dst = ring + st * C::kOperand;
        const float4 sc = scales[tile_no % 8];
        // Value blocks of NaN, or of no page, are left out here (their codes
        // may be NaN; the softmax marks the rows that see them).
        const bool out0 = value && (isnan(sc.z) || sc.x == 0.0f), out1 = value && (isnan(sc.w) || sc.y == 0.0f);
        const int first = closed >= 1 && !out0 ? 0 : 64, last = closed >= 2 && !out1 ? 128 : 64;
        // Four warps: warp w's rows are row0 + (128 / kSteps) i, whose place in
        // the swizzle is the same for every i.
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          const int row = row0 + (128 / kSteps) * i;
          if (row < first || row >= last) continue;
          const uint2 a = *reinterpret_cast<const uint2*>(src + from0 + (128 / kSteps) * D * i);
          const uint2 b = *reinterpret_cast<const uint2*>(src + from1 + (128 / kSteps) * D * i);
          *reinterpret_cast<uint4*>(dst + to0 + (128 / kSteps) * 128 * i) = eight_codes(a);
          *reinterpret_cast<uint4*>(dst + to1 + (128 / kSteps) * 128 * i) = eight_codes(b);
        }
        if (last - first < 128) {
          // The open block's rows, scaled, and zeros elsewhere.  Values that
          // are not finite would spread as 0 * inf; they are left to the rows
          // that see them.
          const int open = closed == 0 || closed == 1 ? 64 * closed : 128;   // the open block's first row
          const int held = g.s.len % kCacheBlock;
#pragma unroll 1
          for (int e = w * 32 + lane; e < 128 * (D / 8); e += 128) {
            const int row = e / (D / 8), ch = e % (D / 8);
            if ((row >= first && row < last) || (row >= open && row < open + 64)) continue;
            *reinterpret_cast<uint4*>(dst + (ch / 8) * C::kRowSlab + row * 128 + (((ch % 8) ^ (row & 7)) << 4)) =
                make_uint4(0u, 0u, 0u, 0u);
          }
          if (open < 128) {
            // The block's loads are all in flight at once; with the keys the
            // values too, whose scale the softmax wants then.
            constexpr int E = D / 16;
            const long long at = ((static_cast<long long>(g.b) * 2 + g.s.slot) * P.c.H + g.h) * kCacheBlock * D;
            auto load = [&](const void* base, uint4 (&x)[E]) {
              const uint4* tail = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + at);
#pragma unroll
              for (int i = 0; i < E; ++i) {
                const int e = w * 32 + lane + 128 * i;
                x[i] = e < held * (D / 8) ? __ldg(tail + e) : make_uint4(0u, 0u, 0u, 0u);
              }
            };
            auto top_of = [&](const uint4 (&x)[E]) {
              uint32_t top = 0;
#pragma unroll
              for (int i = 0; i < E; ++i) {
                top = __vmaxu2(__vmaxu2(top, finite_or_zero(x[i].x) & 0x7fff7fffu), finite_or_zero(x[i].y) & 0x7fff7fffu);
                top = __vmaxu2(__vmaxu2(top, finite_or_zero(x[i].z) & 0x7fff7fffu), finite_or_zero(x[i].w) & 0x7fff7fffu);
              }
              return __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
            };
            uint4 x[E];
            load(value ? P.c.v_tail : P.c.k_tail, x);
            float scale = open_vs;
            if (!value) {
              uint4 y[E];
              load(P.c.v_tail, y);
              const uint32_t tops = top_of(x) | (top_of(y) << 16);
              uint32_t* at_tops = open_tops + 4 * (opens & 1);
              if (lane == 0) {
                at_tops[w] = tops;
                mbar_arrive(open_max);
              }
              if (!__all_sync(0xffffffffu, mbar_wait_poll(open_max, opens & 1u, wait_ns, abort_flag))) {
                ok = false;
                break;
              }
              ++opens;
              const uint32_t all = __vmaxu2(__vmaxu2(at_tops[0], at_tops[1]), __vmaxu2(at_tops[2], at_tops[3]));
              scale = tail_scale(all & 0xffffu);
              open_vs = tail_scale(all >> 16);
              if (w == 0 && lane == 0) {
                float* to = reinterpret_cast<float*>(scales + tile_no % 8) + closed;
                to[0] = scale;
                to[2] = open_vs;
              }
            }
            const float inv = pow2_inv(scale);
            bool odd = false;
#pragma unroll
            for (int i = 0; i < E; ++i) {
              const int e = w * 32 + lane + 128 * i, row = open + e / (D / 8), ch = e % (D / 8);
              if (value) {
                const uint4 y = make_uint4(finite_or_zero(x[i].x), finite_or_zero(x[i].y), finite_or_zero(x[i].z),
                                           finite_or_zero(x[i].w));
                odd = odd || y.x != x[i].x || y.y != x[i].y || y.z != x[i].z || y.w != x[i].w;
                x[i] = y;
              }
              *reinterpret_cast<uint4*>(dst + (ch / 8) * C::kRowSlab + row * 128 + (((ch % 8) ^ (row & 7)) << 4)) =
                  scaled_f16(x[i], inv);
            }
            if (odd) odd_seg[part_no % 8] = part_no + 1;
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(full(st));
          mbar_arrive(raw_empty(rs));
        }
        if (++st == NS) {
          st = 0;
          sph ^= 1u;
        }
        if (++rs == NR) {
          rs = 0;
          rph ^= 1u;
        }
        if (value) ++tile_no;
      }
      ++part_no;
      g = seg_next(P, g);
    }
    if (!ok) raise_timeout(P.err, abort_flag);
  } else {
    // ============================================ softmax and output
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
    const int slot = warp / 4, quarter = warp % 4;
    const int r = quarter * 32 + lane;                  // row of the slot (TMEM lane)
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t sbuf = lane_base + C::s_col(slot), obuf = lane_base + C::o_col(slot);
    uint32_t sn = 0, parts = 0;                         // S tiles and parts of this slot so far
    uint32_t turns = 0;                                 // tiles that both slots had rows in
    bool ok = true;
    // This slot's rows of a part's Q into shared memory (zeros where there is
    // no row), scaled; returns what the row's scores are to be multiplied by.
    // A warp's rows are all in flight at once, and are scaled in their places.
    auto load_q = [&](const Seg& g) -> float {
      constexpr int CR = D / 8;                         // 16-byte chunks of a row
      const CacheRow row = cache_row(P, g.tile * kRows + slot * 128 + r, g.h, g.s.len, g.s.count);
      const unsigned long long from =
          row.valid ? reinterpret_cast<unsigned long long>(P.q + g.b * P.qb + row.head * P.qh + row.n * P.qn) : 0ull;
      unsigned char* buf = qbuf + slot * C::kOperand + quarter * 32 * 128;
      auto chunk = [&](int i, int c) { return buf + (c / 8) * C::kRowSlab + i * 128 + ((c % 8 ^ (i & 7)) << 4); };
#pragma unroll 4
      for (int x = lane; x < 32 * CR; x += 32) {
        const unsigned long long at = __shfl_sync(0xffffffffu, from, x / CR);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(chunk(x / CR, x % CR))),
                     "l"(at != 0 ? at + 16 * (x % CR) : reinterpret_cast<unsigned long long>(P.q)), "r"(at != 0 ? 16 : 0)
                     : "memory");
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();
      uint32_t top = 0;
#pragma unroll 4
      for (int i = 0; i < CR; ++i) {
        const uint4 x = *reinterpret_cast<const uint4*>(chunk(lane, i));
        top = __vmaxu2(__vmaxu2(top, x.x & 0x7fff7fffu), x.y & 0x7fff7fffu);
        top = __vmaxu2(__vmaxu2(top, x.z & 0x7fff7fffu), x.w & 0x7fff7fffu);
      }
      top = max(top & 0xffffu, top >> 16);
      // A row with an infinity or a NaN stays as it is.
      int e = top >= 0x7f80u ? 0 : static_cast<int>(top >> 7) - 127 - 14;
      e = e < -100 ? -100 : e;
      const float down = __int_as_float((127 - e) << 23);
#pragma unroll 2
      for (int i = 0; i < CR; ++i) {
        uint4* x = reinterpret_cast<uint4*>(chunk(lane, i));
        *x = scaled_f16(*x, down);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full(slot));
      return __int_as_float((127 + e) << 23);
    };
    auto keep_seg = [&](const Seg& g) {
      int x[sizeof(Seg) / 4];
      memcpy(x, &g, sizeof(Seg));
      __syncwarp();
      if (lane == 0)
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(Seg) / 4); ++i) seg_mem[i] = x[i];
      __syncwarp();
    };
    auto kept_seg = [&]() {
      Seg g;
      int x[sizeof(Seg) / 4];
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(Seg) / 4); ++i) x[i] = seg_mem[i];
      memcpy(&g, x, sizeof(Seg));
      return g;
    };
    auto row_of = [&](const Seg& g) {
      return cache_row(P, g.tile * kRows + slot * 128 + r, g.h, g.s.len, g.s.count);
    };
    int part_no = 0;
    uint32_t tile_no = 0;                               // of the CTA
    bool more, mine;
    // A slot without rows takes no part in an item; the next item of the CTA
    // may have some again.
    float q_factor = 1.0f;
    auto start = [&](const Seg& g) {
      more = g.left > 0;
      mine = more && (slot == 0 || g.two);
      if (mine) q_factor = load_q(g);
    };
    {
      const Seg g = seg_at(T, w0, w1 - w0);
      keep_seg(g);
      start(g);
    }
    while (more && ok) {
      int j0, n, all_lo, all_end;
      bool paired;
      {
        const Seg g = kept_seg();
        paired = g.two;
        j0 = g.all.first + g.t0;
        n = g.t1 - g.t0;
        const CacheRow row = row_of(g);
        // Keys that every row of the warp sees.
        all_lo = __reduce_max_sync(0xffffffffu, row.valid ? row.see.lo : 0);
        all_end = __reduce_min_sync(0xffffffffu, row.valid ? row.see.end : 0x7fffffff);
      }
      if (mine) {
        const float c1 = P.scale_log2 * q_factor;
        // P = 2^(s + ev - mt), ev the exponent of the value block's scale and
        // mt + kBaseP a recent largest s + ev of the row (raised by 2^4 and more at
        // a time, which costs as little as 2^8; by 2^2 it took 4% more): what a
        // block adds to O is then rounded against the largest such product,
        // however the scales differ.  The row sum l is kept against the largest
        // score, ms.
        float mt = -INFINITY, ms = -INFINITY, l = 0.0f;
        float ev_top = -INFINITY;                       // largest ev so far
        bool vbad = false;
        for (int t = 0; t < n; ++t) {
          if (!__all_sync(0xffffffffu, mbar_wait_poll(s_full(slot), sn & 1u, wait_ns, abort_flag))) {
            ok = false;
            break;
          }
          ++sn;
          tc_fence_after();
          const float4 sc = scales[(tile_no + t) % 8];
          const int kb = (j0 + t) * kTile;
          // Halves outside some row's range: scores there become -inf, in
          // TMEM.  (A NaN key scale makes the scores that are seen NaN; a NaN
          // value scale marks the rows that see its block.)
          const bool full0 = sc.x > 0.0f && !isnan(sc.z) && kb >= all_lo && kb + 64 <= all_end;
          const bool full1 = sc.y > 0.0f && !isnan(sc.w) && kb + 64 >= all_lo && kb + 128 <= all_end;
          if (!(full0 && full1)) {
            const CacheSpan see = row_of(kept_seg()).see;
            vbad = vbad || (isnan(sc.z) && max(see.lo, kb) < min(see.end, kb + 64)) ||
                   (isnan(sc.w) && max(see.lo, kb + 64) < min(see.end, kb + 128));
#pragma unroll 1
            for (int c0 = 0; c0 < 128; c0 += 32) {
              const float ks = c0 < 64 ? sc.x : sc.y;
              const int lo = see.lo - kb - c0, hi = ks == 0.0f ? -1 : see.end - 1 - kb - c0;
              const float seen = isnan(ks) ? ks : 0.0f;
              uint32_t s32[32];
              tmem_ld32(sbuf + c0, s32);
#pragma unroll
              for (int c = 0; c < 32; ++c)
                s32[c] = c >= lo && c <= hi ? __float_as_uint(__uint_as_float(s32[c]) + seen) : 0xff800000u;
              tmem_st32(sbuf + c0, s32);
            }
            tmem_st_wait();
          }
          const float c20 = isnan(sc.x) ? 1.0f : fmaxf(c1 * sc.x, 1e-37f);   // positive: -inf stays -inf
          const float c21 = isnan(sc.y) ? 1.0f : fmaxf(c1 * sc.y, 1e-37f);
          const float ev0 = isnan(sc.z) ? 0.0f : pow2_log(sc.z), ev1 = isnan(sc.w) ? 0.0f : pow2_log(sc.w);
          ev_top = fmaxf(ev_top, fmaxf(ev0, ev1));
          // Pass 1: the row's maxima.  (Loops over the halves are rolled up: the
          // warps' loops share one instruction cache.)
          float s0 = 0.0f, s1 = 0.0f;
#pragma unroll 1
          for (int x = 0; x < 2; ++x) {
            uint32_t sv[64];
            tmem_ld64(sbuf + 64 * x, sv);
            s0 = s1;
            s1 = max64(sv) * (x ? c21 : c20);
          }
          const float pm = fmaxf(s0 + ev0, s1 + ev1);
          float f = 1.0f;
          if (pm > mt + kTopP) {
            f = mt == -INFINITY ? 1.0f : ex2_ftz(mt + kBaseP - pm);
            mt = pm - kBaseP;
          }
          // The slot's previous PV was issued before this tile's QK, whose
          // commit has arrived: O may be rescaled.
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
          const float top = fmaxf(ms, fmaxf(s0, s1));
          if (top > ms) {
            l *= ex2_ftz(ms - top);
            ms = top;
          }
          // A row that has seen no key: exp2(-inf - 0) = 0.
          const float nm = mt == -INFINITY ? 0.0f : -mt, ns = ms == -INFINITY ? 0.0f : -ms;
          float add = 0.0f;
          // Sum of the weights of half x where P may vanish beside another
          // block's but the sum must not.
          auto far_sum = [&](int x, float c2) {
#pragma unroll 1
            for (int c0 = 0; c0 < 64; c0 += 32) {
              uint32_t s32[32];
              tmem_ld32(sbuf + 64 * x + c0, s32);
#pragma unroll
              for (int c = 0; c < 32; ++c) add += ex2_ftz(fmaf(__uint_as_float(s32[c]), c2, ns));
            }
          };
          const bool far0 = ev_top - ev0 > 90.0f, far1 = ev_top - ev1 > 90.0f;
          if (far1) far_sum(1, c21);
          if (far0) far_sum(0, c20);
          // Pass 2: 32 scores as 16 pairs of P, over columns of S that have been
          // read.
          auto weights = [&](const uint32_t* v, uint64_t c22, uint64_t off, uint32_t to, uint64_t& sum0, uint64_t& sum1) {
            uint32_t pk[16];
#pragma unroll
            for (int c = 0; c < 32; c += 4) {
              float p0, p1, p2, p3;
              unpack2(fma2(pack2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), c22, off), p0, p1);
              unpack2(fma2(pack2(__uint_as_float(v[c + 2]), __uint_as_float(v[c + 3])), c22, off), p2, p3);
              p0 = ex2_ftz(p0);
              p1 = ex2_ftz(p1);
              p2 = ex2_ftz(p2);
              p3 = ex2_ftz(p3);
              pk[c / 2] = pack_f16x2(p0, p1);
              pk[c / 2 + 1] = pack_f16x2(p2, p3);
              sum0 = add2(sum0, pack2(p0, p1));
              sum1 = add2(sum1, pack2(p2, p3));
            }
            tmem_st16(to, pk);
          };
          // P of a half is in TMEM: its PV may start.
          auto hand_over = [&](uint32_t to) {
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(to);
          };
          // The two slots' warps of one scheduler take turns at the
          // exponentials: 128 of them are 1024 cycles of its unit, and a warp
          // that has them alone hands its P over while the other one's
          // products run, instead of both at half the speed.
          if (paired) {
            if ((slot == 1 || turns > 0) &&
                !__all_sync(0xffffffffu, mbar_wait_poll(turn(warp), (turns - (1 - slot)) & 1u, wait_ns, abort_flag))) {
              ok = false;
              break;
            }
            ++turns;
          }
          uint32_t sa[32], sb[32];
          tmem_ld32_async(sbuf, sa);
#pragma unroll 1
          for (int x = 0; x < 2; ++x) {
            const float c2 = x ? c21 : c20, ev = x ? ev1 : ev0;
            const uint64_t c22 = pack2(c2, c2), off = pack2(nm + ev, nm + ev);
            uint64_t sum0 = 0, sum1 = 0;
            tmem_arrived();
            pin32(sa);
            tmem_ld32_async(sbuf + 64 * x + 32, sb);
            weights(sa, c22, off, sbuf + 32 * x, sum0, sum1);
            tmem_arrived();
            pin32(sb);
            if (x == 0) tmem_ld32_async(sbuf + 64, sa);
            weights(sb, c22, off, sbuf + 32 * x + 16, sum0, sum1);
            if (x == 1 && paired && lane == 0) mbar_arrive(turn(warp ^ 4));
            hand_over(x ? p_full(slot) : p_half(slot));
            // The sum is not on the way to the next product.
            float u0, u1;
            unpack2(add2(sum0, sum1), u0, u1);
            if (!(x ? far1 : far0)) add = fmaf(u0 + u1, ex2_ftz(ns - nm - ev), add);
          }
          l += add;
        }
        if (!ok) break;
        // Every QK of the part has run: the next part's Q, while its last PV does.
        if (!__all_sync(0xffffffffu, mbar_wait_poll(q_free(slot), parts & 1u, wait_ns, abort_flag))) {
          ok = false;
          break;
        }
        ++parts;
        const Seg g = kept_seg();
        const CacheRow row = row_of(g);
        const Seg ng = seg_next(P, g);
        keep_seg(ng);
        start(ng);
        if (!__all_sync(0xffffffffu, mbar_wait_poll(o_done(slot), (parts - 1) & 1u, wait_ns, abort_flag))) {
          ok = false;
          break;
        }
        tc_fence_after();
        // ---- output: O is in units of 2^mt, the sum of 2^ms
        const bool whole = g.t0 == 0 && g.t1 == g.all.n;
        const bool odd = odd_seg[part_no % 8] == part_no + 1;
        const float unit = mt == -INFINITY ? 1.0f : ex2_ftz(mt - ms);
        // Means, of parts too: sums of large values need not be a float.
        const float inv = weight_inv(l);
        char* orow = P.o + g.b * P.ob + row.head * P.oh + row.n * P.on;
        const long long part = 2ll * blockIdx.x + (g.first ? 0 : 1);
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
          uint32_t o32[32];
          tmem_ld32(obuf + c0, o32);
          float v[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = vbad ? __int_as_float(0x7fffffff) : __uint_as_float(o32[e]) * inv * unit;
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
                  make_uint4(pack_bf16x2(v[e], v[e + 1]), pack_bf16x2(v[e + 2], v[e + 3]),
                             pack_bf16x2(v[e + 4], v[e + 5]), pack_bf16x2(v[e + 6], v[e + 7]));
          } else if (row.valid) {
            // [part][channel][row]: a warp's rows side by side.
            float* to = P.part_o + (part * D + c0) * kRows + slot * 128 + r;
#pragma unroll
            for (int e = 0; e < 32; ++e) to[e * kRows] = v[e];
          }
        }
        if (row.valid && whole && P.lse != nullptr)
          P.lse[(static_cast<long long>(g.b) * P.Hq + row.head) * P.N + row.n] = (ms + log2f(l)) * 0.6931471805599453f;
        if (row.valid && !whole) P.part_ml[part * kRows + slot * 128 + r] = make_float2(ms, l);
        tc_fence_before();
      } else {
        // No rows in this item: its slot's Q buffer is idle.
        const Seg ng = seg_next(P, kept_seg());
        keep_seg(ng);
        start(ng);
      }
      tile_no += n;
      ++part_no;
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

// Merges the parts of the items that more than one CTA worked on: a CTA for
// each CTA whose run begins inside an item, and 32 rows; a row per lane.  An
// item of n parts has n - 1 such CTAs.  The first S of them (8, 4 or, with up
// to four parts, 1) take a slice of the channels each; a warp has an eighth of
// the channels and every S-th part.  (With the parts one after the other 147 rows of 2 sequences
// on 20000 and 11000 keys, d = 64, 79 and 44 parts, took 97 us in all: 35 this
// way; few parts leave from the registers, since the exchange took 10 us of
// issue where every SM has eight such CTAs.)
template <int D>
__global__ void __launch_bounds__(256) cache_tc_merge_kernel(const __grid_constant__ TcParams T, int grid) {
  const CacheAttnParams& P = T.a;
  constexpr int C = D / 8, PAD = 33;
  __shared__ float os[8][C][PAD];
  __shared__ float2 mls[8][32];
  const int cta = blockIdx.x / (kRows / 32), r0 = blockIdx.x % (kRows / 32) * 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long long total = T.seq_prefix[P.c.B];
  const long long ctas = work_ctas(total, grid);
  const Inside in = T.inside[cta];
  if (cta == 0 || cta >= ctas) return;
  // (Beyond `tile < 0`: a launch that refused to run has noted nothing.)
  if (in.tile < 0 || in.tile >= P.tiles || in.b < 0 || in.b >= P.c.B || in.h < 0 || in.h >= P.c.H || in.n < 1 ||
      in.start < 0 || in.start + in.n > total)
    return;
  // CTA c holds tiles [total c / ctas, total (c + 1) / ctas).
  const int c0 = static_cast<int>(((in.start + 1) * ctas + total - 1) / total) - 1;
  const int c1 = static_cast<int>(((in.start + in.n) * ctas + total - 1) / total) - 1;
  const int split = c1 - c0 >= 8 ? 8 : (c1 - c0 >= 4 ? 4 : 1);
  const int slice = cta - c0 - 1;
  if (slice >= split) return;
  bool bad = false;
  const SeqInfo s = seq_info(P, in.b, &bad);
  if (in.tile * kRows + r0 >= s.count * P.group) return;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int groups = 8 / split;        // of channels, in this CTA
  const int ch0 = slice * groups * C, ch = ch0 + warp % groups * C, c_first = c0 + warp / groups;
  // The item is the first part of every CTA but, perhaps, its first one's.
  const int first_part = total * c0 / ctas >= in.start ? 0 : 1;
  auto part_of = [&](int c) { return 2ll * c + (c == c0 ? first_part : 0); };
  float m = -INFINITY;
#pragma unroll 4
  for (int c = c_first; c <= c1; c += split) m = fmaxf(m, P.part_ml[part_of(c) * kRows + r0 + lane].x);
  float l = 0.0f, acc[C] = {};
#pragma unroll 4
  for (int c = c_first; c <= c1; c += split) l += part_weight(P.part_ml[part_of(c) * kRows + r0 + lane], m);
  const float inv = weight_inv(l);
#pragma unroll 2
  for (int c = c_first; c <= c1; c += split) {
    const float f = part_weight(P.part_ml[part_of(c) * kRows + r0 + lane], m) * inv;
    const float* from = P.part_o + (part_of(c) * D + ch) * kRows + r0 + lane;
#pragma unroll
    for (int e = 0; e < C; ++e) acc[e] = fmaf(from[e * kRows], f, acc[e]);
  }
  if (split == 1) {
    // The row's sums are all here.
    const CacheRow row = cache_row(P, in.tile * kRows + r0 + lane, in.h, s.len, s.count);
    if (!row.valid) return;
    char* to = P.o + in.b * P.ob + row.head * P.oh + row.n * P.on + 2 * ch;
#pragma unroll
    for (int e = 0; e < C; e += 8)
      *reinterpret_cast<uint4*>(to + 2 * e) =
          make_uint4(pack_bf16x2(acc[e], acc[e + 1]), pack_bf16x2(acc[e + 2], acc[e + 3]),
                     pack_bf16x2(acc[e + 4], acc[e + 5]), pack_bf16x2(acc[e + 6], acc[e + 7]));
    if (ch == 0 && P.lse != nullptr)
      P.lse[(static_cast<long long>(in.b) * P.Hq + row.head) * P.N + row.n] = (m + log2f(l)) * 0.6931471805599453f;
    return;
  }
#pragma unroll
  for (int e = 0; e < C; ++e) os[warp][e][lane] = acc[e];
  mls[warp][lane] = make_float2(m, l);
  __syncthreads();
  // Two channels of a row at a time, a row's side by side.
  const int pairs = groups * C / 2, log_pairs = __ffs(pairs) - 1;
  for (int x = threadIdx.x; x < 32 * pairs; x += 256) {
    const int pair = x & (pairs - 1), i = x >> log_pairs, g = pair / (C / 2), e = pair % (C / 2) * 2;
    const CacheRow row = cache_row(P, in.tile * kRows + r0 + i, in.h, s.len, s.count);
    if (!row.valid) continue;
    float top = -INFINITY, sum = 0.0f, a0 = 0.0f, a1 = 0.0f;
    for (int k = g; k < 8; k += groups) top = fmaxf(top, mls[k][i].x);
    for (int k = g; k < 8; k += groups) sum += part_weight(mls[k][i], top);
    const float all = weight_inv(sum);
    for (int k = g; k < 8; k += groups) {
      const float f = part_weight(mls[k][i], top) * all;
      a0 = fmaf(os[k][e][i], f, a0);
      a1 = fmaf(os[k][e + 1][i], f, a1);
    }
    *reinterpret_cast<uint32_t*>(P.o + in.b * P.ob + row.head * P.oh + row.n * P.on + 2 * (ch0 + g * C + e)) =
        pack_bf16x2(a0, a1);
    if (ch0 == 0 && pair == 0 && P.lse != nullptr)
      P.lse[(static_cast<long long>(in.b) * P.Hq + row.head) * P.N + row.n] = (top + log2f(sum)) * 0.6931471805599453f;
  }
}

struct Layout {
  int tiles;
  size_t part_o, part_ml, tile_prefix, seq_prefix, inside, total;
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
  L.inside = take(num_sms * sizeof(Inside));
  L.total = off;
  return L;
}

template <int D>
cudaError_t launch_d(const Ctx& c, const TcParams& T) {
  const cudaError_t e = cudaFuncSetAttribute(cache_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, CT<D>::kSmem);
  if (e != cudaSuccess) return e;
  cache_plan_kernel<<<1, 1024, 0, c.stream>>>(T);
  // Each launched while the one before it runs; they wait for its end before
  // they read what it wrote.
  cudaLaunchAttribute early = {};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(c.num_sms);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = CT<D>::kSmem;
  cfg.stream = c.stream;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  const cudaError_t ran = cudaLaunchKernelEx(&cfg, cache_tc_kernel<D>, T);
  if (ran != cudaSuccess) return ran;
  cfg.gridDim = dim3(c.num_sms * (kRows / 32));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, cache_tc_merge_kernel<D>, T, c.num_sms);
}

}  // namespace

size_t cache_attn_tc_ws_bytes(const CacheAttnArgs& a, int num_sms) { return layout_of(a, num_sms).total; }

cudaError_t launch_cache_attn_tc(const Ctx& c, const CacheAttnArgs& a, CacheAttnParams P) {
  const Layout L = layout_of(a, c.num_sms);
  char* ws = static_cast<char*>(a.workspace);
  TcParams T;
  P.tiles = L.tiles;
  P.part_o = reinterpret_cast<float*>(ws + L.part_o);
  P.part_ml = reinterpret_cast<float2*>(ws + L.part_ml);
  T.a = P;
  T.tile_prefix = reinterpret_cast<int*>(ws + L.tile_prefix);
  T.seq_prefix = reinterpret_cast<long long*>(ws + L.seq_prefix);
  T.inside = reinterpret_cast<Inside*>(ws + L.inside);
  return a.cache.d == 128 ? launch_d<128>(c, T) : launch_d<64>(c, T);
}

}  // namespace salad
