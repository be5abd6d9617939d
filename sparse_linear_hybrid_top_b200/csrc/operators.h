// operators.h -- parameters and launchers of the rotary and cache operators.
#pragma once

#include "internal.h"
#include "rope.cuh"

namespace salad {

// A device error bit beside kErrTimeout and kErrLayout: a cache operator
// skipped a page, length, slot or count out of range.
constexpr unsigned kErrRange = 4u;

// Half pages of an e4m3 pool [slabs][64][d]: box d x 32 x 1, swizzled over its
// rows (128-byte at d = 128, 64-byte at d = 64).
bool make_tmap_codes(CUtensorMap* map, const void* base, long long slabs, int d);

// ---- rotary positions (rope.cu)
// y = x with every channel pair turned by position * rate (inverse: by the
// negative angle).  Strides (batch, head, token) in elements; k may be null
// with Hk = 0.
struct RopeArgs {
  const void* q;
  void* q_out;
  const void* k;
  void* k_out;
  long long q_st[3], qo_st[3], k_st[3], ko_st[3];
  int dtype;                  // 0 bf16, 1 fp16, 2 fp32
  int B, Hq, Hk, N, d;
  RopeWhere where;
  int split[3];
  float base;
  int pairing;                // 0 adjacent, 1 halves
  int inverse;
};
cudaError_t launch_rope(const Ctx& c, const RopeArgs& a);

// ---- 8-bit block cache (cache_append.cu)
struct CacheView {
  unsigned char* k_pages;     // e4m3 [pages, H, 64, d]
  unsigned char* v_pages;
  float* k_scale;             // [pages, H]
  float* v_scale;
  void* k_tail;               // bf16 [B, 2, H, 64, d]
  void* v_tail;
  const int32_t* page_table;  // [B, blocks]
  int B, H, d, pages, blocks;
};
struct CacheAppendArgs {
  CacheView cache;
  const int32_t* seq;         // [B, 2]: tokens held, tail slot
  int32_t* seq_out;           // null, seq (advanced by a second launch) or apart
  const void* k;
  const void* v;
  long long k_st[3], v_st[3]; // elements (batch, head, token)
  int N;
  const int32_t* counts;
  int rotate;
  RopeWhere where;
  int split[3];
  float base;
  int pairing;
};
cudaError_t launch_cache_append(const Ctx& c, const CacheAppendArgs& a);

// ---- attention over the cache (cache_attn.cu)
struct CacheAttnArgs {
  CacheView cache;
  const int32_t* seq;
  const void* q;
  void* o;
  long long q_st[3], o_st[3]; // elements (batch, head, token)
  float* lse;                 // [B, Hq, N] or null
  int Hq, N;
  const int32_t* counts;
  int frame, window;
  float scale;
  void* workspace;            // cache_attn_ws_bytes() bytes
};
size_t cache_attn_ws_bytes(const CacheAttnArgs& a, int num_sms);
cudaError_t launch_cache_attn(const Ctx& c, const CacheAttnArgs& a);

}  // namespace salad
