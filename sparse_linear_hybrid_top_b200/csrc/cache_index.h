// cache_index.h -- where the tokens of a block cache are: the arithmetic of
// lengths, blocks, slots, pages and masks that the append and the attention
// share.  Plain C++ (it compiles for the host too, where it is tested).
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define SALAD_HD __host__ __device__ __forceinline__
#else
#define SALAD_HD inline
#endif

namespace salad {

constexpr int kCacheBlock = 64;

// Most tokens that a table of `blocks` pages and an open block hold.
SALAD_HD int cache_room(int blocks) { return blocks * kCacheBlock + kCacheBlock - 1; }

// A sequence's state: tokens held and tail slot, forced into range.  *bad is
// set where it was not.
struct CacheSeq {
  int len, slot;
};
SALAD_HD CacheSeq cache_seq(int len, int slot, int blocks, bool* bad) {
  CacheSeq s{len, slot};
  if (s.len < 0) { s.len = 0; *bad = true; }
  if (s.len > cache_room(blocks)) { s.len = cache_room(blocks); *bad = true; }
  if (s.slot != 0 && s.slot != 1) { s.slot &= 1; *bad = true; }
  return s;
}

// Valid rows of a batch of N, forced into [0, N].
SALAD_HD int cache_count(int count, int N, bool* bad) {
  if (count >= 0 && count <= N) return count;
  *bad = true;
  return count < 0 ? 0 : N;
}

// What an append of n tokens to s does: blocks [first, last) close, the rows
// behind stay open in slot_out.  n is cut to the table's room.
struct CacheAppend {
  int n, first, last, slot_out;
};
SALAD_HD CacheAppend cache_append_plan(CacheSeq s, int n, int blocks, bool* bad) {
  CacheAppend a;
  if (n > cache_room(blocks) - s.len) { n = cache_room(blocks) - s.len; *bad = true; }
  a.n = n;
  a.first = s.len / kCacheBlock;
  a.last = (s.len + n) / kCacheBlock;
  // A chunk that closes the open block leaves its rows where they are and
  // opens the next block in the other slot: the append can be repeated.
  a.slot_out = a.first == a.last ? s.slot : 1 - s.slot;
  return a;
}

// The page of block j (j in [0, blocks)), or -1 where the table's entry is no page.
SALAD_HD int cache_page(int entry, int pages) { return entry >= 0 && entry < pages ? entry : -1; }

// Keys [lo, end) that the query at position p sees, of `len` held tokens; the
// n queries are the last ones.  lo >= end: none.
struct CacheSpan {
  int lo, end;
};
SALAD_HD CacheSpan cache_visible(int p, int len, int n, int frame, int window) {
  CacheSpan v;
  int group;
  if (frame > 0) {
    // floor(p / frame) * frame, p of either sign (|p| < 2^31 - frame is not
    // needed: a negative p only has to give an end <= 0).
    if (p < 0) return CacheSpan{0, 0};
    group = p / frame * frame;
    v.end = len - group > frame ? group + frame : len;
  } else {
    group = len - n;
    v.end = len;
  }
  v.lo = window >= 0 && group > window ? group - window : 0;
  return v;
}

}  // namespace salad
