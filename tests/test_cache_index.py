"""The block cache's index arithmetic (lengths, blocks, slots, pages, masks) on
the host: csrc/cache_index.h is compiled with g++ and compared with plain
Python, at the ends of every range and past them."""
import ctypes
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = r'''
#include "cache_index.h"
using namespace salad;
extern "C" int append(int len, int slot, int count, int N, int blocks, int* out) {
  bool bad = false;
  CacheSeq s = cache_seq(len, slot, blocks, &bad);
  int n = cache_count(count, N, &bad);
  CacheAppend a = cache_append_plan(s, n, blocks, &bad);
  out[0] = s.len; out[1] = s.slot; out[2] = a.n; out[3] = a.first; out[4] = a.last; out[5] = a.slot_out;
  return bad;
}
extern "C" int page(int entry, int pages) { return cache_page(entry, pages); }
extern "C" void visible(int p, int len, int n, int frame, int window, int* out) {
  CacheSpan v = cache_visible(p, len, n, frame, window);
  out[0] = v.lo; out[1] = v.end;
}
'''
BIG = 2 ** 31 - 1


@pytest.fixture(scope="module")
def index(tmp_path_factory):
    at = tmp_path_factory.mktemp("index")
    src, so = at / "index.cpp", at / "index.so"
    src.write_text(SRC)
    inc = os.path.join(ROOT, "sparse_linear_hybrid_top_b200", "csrc")
    # Overflow in the arithmetic would trap.
    subprocess.run(["g++", "-std=c++17", "-O1", "-ftrapv", "-shared", "-fPIC", "-I", inc, str(src), "-o", str(so)], check=True)
    return ctypes.CDLL(str(so))


def _append(index, *a):
    out = (ctypes.c_int * 6)()
    bad = index.append(*a, out)
    return bool(bad), list(out)


@pytest.mark.parametrize("blocks", [1, 2, 7, 1 << 24])
def test_append_plan(index, blocks):
    rng = random.Random(blocks)
    room = blocks * 64 + 63
    lens = [0, 1, 63, 64, 65, room - 64, room - 1, room, room + 1, -1, BIG, -BIG - 1] + [rng.randint(0, room) for _ in range(50)]
    for length in lens:
        for slot in (0, 1, 2, -1):
            for N in (1, 2, 63, 64, 65, 262144):
                for count in (0, 1, N // 2, N, N + 1, -1, BIG, -BIG - 1):
                    bad, (ln, sl, n, first, last, out) = _append(index, length, slot, count, N, blocks)
                    want_len = min(max(length, 0), room)
                    want_n = min(max(count, 0), N)
                    cut = min(want_n, room - want_len)
                    assert (ln, n) == (want_len, cut)
                    assert bad == (want_len != length or slot not in (0, 1) or want_n != count or cut != want_n)
                    assert sl in (0, 1) and (slot not in (0, 1) or sl == slot)
                    assert (first, last) == (want_len // 64, (want_len + cut) // 64)
                    assert out == (sl if first == last else 1 - sl)
                    assert last <= blocks      # closed blocks are inside the table


def test_page(index):
    for pages in (1, 5, BIG):
        for entry in (-BIG - 1, -1, 0, pages - 1, pages, BIG):
            assert index.page(ctypes.c_int(entry), ctypes.c_int(pages)) == (entry if 0 <= entry < pages else -1)


def test_visible_keys(index):
    rng = random.Random(3)
    out = (ctypes.c_int * 2)()
    top = (1 << 30) + 63
    for _ in range(20000):
        length = rng.choice([0, 1, 5, 64, 1000, top, rng.randint(0, top)])
        n = rng.choice([1, 2, 100, 262144, rng.randint(1, 262144)])
        i = rng.randint(0, n - 1)
        frame = rng.choice([0, 1, 2, 7, 1560, BIG])
        window = rng.choice([-1, 0, 1, 100, BIG, -BIG - 1])
        p = length - n + i
        index.visible(p, length, n, frame, window, out)
        if frame == 0:
            group, end = length - n, length
        else:
            group = p // frame * frame
            end = min(length, group + frame)
        low = max(0, group - window) if window >= 0 else 0
        keys = range(low, max(low, end))
        got = range(out[0], max(out[0], out[1]))
        assert (len(keys) == 0 and len(got) == 0) or keys == got, (p, length, n, frame, window)
        assert out[0] >= 0 and out[1] <= length
