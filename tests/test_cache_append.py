"""Appending to the 8-bit block cache: argument checks (no GPU) and GPU parity.

The cache's contents are compared bit for bit: the codes and scales against a
numpy implementation of their definition, from the bf16 rows (the keys as
salad.rope turns them, which test_rope.py holds to float64).
"""
import ctypes
import math

import numpy as np
import pytest
import torch

import sparse_linear_hybrid_top_b200 as salad
from sparse_linear_hybrid_top_b200 import Cache, CacheAppendArgs, Strides, lib

INVALID, UNSUP = -1, -2
A = 0x100000         # a 256-aligned fake device address (never dereferenced)
M = 1 << 30


def _cache(**kw):
    c = Cache(A, A + M, A + 2 * M, A + 3 * M, A + 4 * M, A + 5 * M, A + 6 * M, 2, 3, 64, 10, 5)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _status(cache=None, **kw):
    a = CacheAppendArgs()
    a.cache = _cache(**(cache or {}))
    a.seq, a.seq_out, a.k, a.v = A + 7 * M, A + 7 * M + 256, A + 8 * M, A + 9 * M
    a.k_st = a.v_st = Strides(3 * 100 * 64, 100 * 64, 64)
    a.N, a.rotate, a.Hh, a.Wh, a.base = 100, 1, 4, 5, 10000.0
    a.split = (ctypes.c_int * 3)(24, 20, 20)
    for k, v in kw.items():
        setattr(a, k, v)
    return lib.salad_cache_append(ctypes.byref(a), None)


def test_append_argument_checks():
    assert lib.salad_cache_append(None, None) == INVALID
    for kw in (dict(k_pages=None), dict(v_pages=A + 8), dict(k_scale=None), dict(v_scale=A + 2), dict(k_tail=A + 8),
               dict(v_tail=None), dict(page_table=None), dict(B=0), dict(H=0), dict(H=257), dict(B=40000), dict(pages=0),
               dict(blocks=0), dict(blocks=(1 << 24) + 1)):
        assert _status(cache=kw) == INVALID, kw
    for d in (32, 96, 256):
        assert _status(cache=dict(d=d)) == UNSUP
    for kw in (dict(seq=None), dict(seq_out=A + 7 * M + 8), dict(seq_out=A + 7 * M + 2), dict(k=None), dict(v=A + 8),
               dict(N=0), dict(N=262145), dict(counts=A + 1), dict(rotate=2), dict(positions=A + 1), dict(positions_batched=3),
               dict(Hh=0), dict(base=0.5), dict(pairing=7), dict(split=(ctypes.c_int * 3)(24, 20, 18)),
               dict(k_st=Strides(19200, 6400, 60)), dict(v_st=Strides(19200, 6400, -64)),
               dict(k=A), dict(v=A + 4 * M)):           # the new tokens inside the cache
        assert _status(**kw) == INVALID, kw


def test_append_accepts_valid_calls():
    if torch.cuda.is_available():
        pytest.skip("fake addresses must not reach a launch")
    for kw in (dict(), dict(seq_out=None), dict(seq_out=A + 7 * M), dict(rotate=0, Hh=0, base=0.0), dict(positions=A, Hh=0),
               dict(k_st=Strides(0, 0, 0))):
        assert _status(**kw) in (UNSUP, -3), kw


# ------------------------------------------------------------------- GPU ---
def _f64(t):
    return t.detach().float().cpu().double().numpy()


def _encode(x):
    """x float64 [64, d] (bf16 values): e4m3 values and the scale, by definition."""
    if not np.all(np.isfinite(x)):
        return np.full_like(x, np.nan), np.nan
    top, e = float(np.abs(x).max()), -100
    while top > 448.0 * 2.0 ** e:
        e += 1
    y = x / 2.0 ** e
    step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6))) - 3)
    return np.round(y / step) * step, 2.0 ** e      # np.round: ties to even


def _fill(cache, seed):
    """Recognisable contents everywhere, so that a stray write shows."""
    g = torch.Generator().manual_seed(seed)
    for t in (cache.k_pages, cache.v_pages):
        t.view(torch.uint8).copy_(torch.randint(0, 126, t.shape, generator=g, dtype=torch.uint8))
    for t in (cache.k_scale, cache.v_scale):
        t.copy_(torch.exp2(torch.randint(-3, 3, t.shape, generator=g).float()))
    for t in (cache.k_tail, cache.v_tail):
        t.copy_(torch.randn(t.shape, generator=g))


def _state(cache):
    return {n: _f64(getattr(cache, n)) for n in ("k_pages", "v_pages", "k_scale", "v_scale", "k_tail", "v_tail")}


def _expect(before, cache, turned, v, seq, counts):
    """The cache after the append, from its state before it."""
    want = {n: x.copy() for n, x in before.items()}
    table = cache.page_table.cpu().numpy()
    out = []
    for b, ((L, slot), n) in enumerate(zip(seq, counts)):
        first, last = L // 64, (L + n) // 64
        to = slot if first == last else 1 - slot
        out.append((L + n, to))
        for name, new in (("k", turned), ("v", v)):
            rows = np.concatenate([before[name + "_tail"][b, slot, :, :L % 64], _f64(new)[b, :, :n]], axis=1)
            for j in range(first, last):
                for h in range(cache.H):
                    y, scale = _encode(rows[h, (j - first) * 64:(j - first + 1) * 64])
                    want[name + "_pages"][table[b, j], h] = y
                    want[name + "_scale"][table[b, j], h] = scale
            lo, hi = (0 if last > first else L % 64), (L + n) % 64
            if hi > lo:
                at = (last - first) * 64
                want[name + "_tail"][b, to, :, lo:hi] = rows[:, at + lo:at + hi]
    return want, out


def _make(B, H, d, blocks, extra=3, seed=0):
    cache = salad.BlockCache.allocate(B, H, d, blocks, pages=B * blocks + extra)
    g = torch.Generator().manual_seed(seed)
    cache.page_table.copy_(torch.randperm(B * blocks + extra, generator=g)[:B * blocks].reshape(B, blocks))
    _fill(cache, seed + 1)
    return cache


def _tokens(B, H, N, d, seed):
    g = torch.Generator().manual_seed(seed)
    size = torch.exp2(torch.randint(-6, 6, (1, H, 1, d), generator=g).float())
    return [(torch.randn(B, H, N, d, generator=g) * size).to(torch.bfloat16).cuda() for _ in range(2)]


def _run(cache, k, v, seq, counts=None, turned=None, **kw):
    before = _state(cache)
    n = [k.shape[2]] * cache.B if counts is None else counts
    got = salad.cache_append(cache, k, v, torch.tensor(seq, dtype=torch.int32).cuda(),
                             counts=None if counts is None else torch.tensor(counts, dtype=torch.int32).cuda(), **kw)
    want, out = _expect(before, cache, k if turned is None else turned, v, seq, n)
    assert got.cpu().tolist() == [list(x) for x in out]
    after = _state(cache)
    for name in want:
        np.testing.assert_array_equal(after[name], want[name], err_msg=name)
    salad.check_error()


needs_gpu = pytest.mark.gpu


@needs_gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,lens,counts", [
    (1, [0, 5, 63], None),                 # single tokens; the last one closes its block
    (1, [64, 127, 128], [1, 0, 1]),        # and an empty row of the batch
    (64, [0, 1, 63], None),                # whole blocks, aligned and not
    (65, [0, 64, 130], [65, 64, 63]),
    (130, [10, 126, 190], [130, 2, 0]),    # the open block closes and another opens, same parity
    (200, [0, 33, 120], [200, 31, 199]),
], ids=str)
def test_append_without_rotation(d, N, lens, counts):
    cache = _make(3, 2, d, 7, seed=N)
    k, v = _tokens(3, 2, N, d, N + 1)
    _run(cache, k, v, list(zip(lens, [0, 1, 0])), counts)


@needs_gpu
@pytest.mark.parametrize("pairing", ["adjacent", "halves"])
@pytest.mark.parametrize("d,H", [(64, 1), (128, 5)])
def test_append_turns_keys(d, H, pairing):
    B, N, lens = 2, 150, [37, 128]
    cache = _make(B, H, d, 5, seed=2)
    k, v = _tokens(B, H, N, d, 3)
    # The grid position of a token is its place in the cache.
    turned = torch.cat([salad.rope(k[b:b + 1], grid=(3, 7), offset=lens[b], pairing=pairing) for b in range(B)])
    _run(cache, k, v, [(37, 1), (128, 0)], [150, 101], turned=turned, grid=(3, 7), pairing=pairing)
    at = torch.randint(-1000, 1 << 20, (B, N, 3), dtype=torch.int32).cuda()
    split = (0, d // 2, d // 2)
    for pos in (at, at[1].contiguous()):
        turned = salad.rope(k, positions=pos, pairing=pairing, split=split)
        _run(cache, k, v, [(37, 1), (128, 0)], turned=turned, positions=pos, pairing=pairing, split=split)


@needs_gpu
def test_append_many_heads_share_a_cta():
    """More blocks than four CTAs an SM would be: heads share a CTA."""
    cache = _make(2, 40, 64, 30, seed=4)
    k, v = _tokens(2, 40, 1500, 64, 5)
    turned = torch.cat([salad.rope(k[b:b + 1], grid=(9, 16), offset=L) for b, L in ((0, 77), (1, 300))])
    _run(cache, k, v, [(77, 0), (300, 1)], turned=turned, grid=(9, 16))


@needs_gpu
def test_append_strided_tokens():
    B, H, N, d = 2, 3, 70, 64
    g = torch.Generator().manual_seed(6)
    qkv = torch.randn(B, N, 3, H, d, generator=g).to(torch.bfloat16).cuda()
    k, v = qkv[:, :, 1].transpose(1, 2), qkv[:, :, 2].transpose(1, 2)
    _run(_make(B, H, d, 3, seed=7), k, v, [(0, 0), (50, 1)])
    one = torch.randn(1, 1, N, d, generator=g).to(torch.bfloat16).cuda().expand(B, H, N, d)
    _run(_make(B, H, d, 3, seed=8), one, v, [(0, 0), (50, 1)])


@needs_gpu
def test_append_can_be_repeated_and_continued():
    """A chunk written twice at one place is the last one written; chunks of
    any size leave the same cache as one append of them all."""
    B, H, N, d = 1, 2, 300, 128
    k, v = _tokens(B, H, N, d, 9)
    whole = _make(B, H, d, 6, extra=0, seed=10)
    parts = _make(B, H, d, 6, extra=0, seed=10)
    seq = whole.new_seq()
    end = salad.cache_append(whole, k, v, seq, grid=(4, 9))
    at, i = parts.new_seq(), 0
    for n in (1, 62, 1, 5, 130, 64, 37):
        noise = _tokens(B, H, n, d, n)
        salad.cache_append(parts, *noise, at, grid=(4, 9))          # an earlier denoising step
        at = salad.cache_append(parts, k[:, :, i:i + n], v[:, :, i:i + n], at, grid=(4, 9))
        i += n
    assert i == N and int(end[0, 0]) == int(at[0, 0]) == N
    a, b = _state(whole), _state(parts)
    pages = whole.page_table[0, :N // 64].cpu().numpy()
    for name in ("k_pages", "v_pages", "k_scale", "v_scale"):
        np.testing.assert_array_equal(a[name][pages], b[name][pages])
    for name in ("k_tail", "v_tail"):
        np.testing.assert_array_equal(a[name][0, int(end[0, 1]), :, :N % 64], b[name][0, int(at[0, 1]), :, :N % 64])


@needs_gpu
def test_append_extreme_blocks():
    """Zeros, the scale's borders, tiny and huge values, infinities and NaN."""
    d, H = 64, 9
    cache = _make(1, H, d, 2, seed=11)
    k = torch.zeros(1, H, 64, d, dtype=torch.bfloat16)
    k[0, 1, 3, 5] = 448.0
    k[0, 2, 3, 5] = 450.0                       # the next bf16 value: the scale doubles
    k[0, 3, :, :] = -1.75 * 2.0 ** -20
    k[0, 4, 63, 63] = 2.0 ** -133               # a bf16 subnormal: below the smallest scale
    k[0, 5, 0, 0] = 3.0e38
    k[0, 6, 1, 1] = math.inf
    k[0, 7, 2, 2] = math.nan
    k[0, 8] = torch.linspace(-3, 3, 64 * d).reshape(64, d).to(torch.bfloat16)
    k = k.cuda()
    _run(cache, k, -k, [(0, 0)])
    assert torch.isnan(cache.k_scale[cache.page_table[0, 0].long(), 6])


@needs_gpu
def test_append_advances_seq_in_place_and_in_a_graph():
    B, H, d = 2, 2, 64
    cache, ref = _make(B, H, d, 3, seed=12), _make(B, H, d, 3, seed=12)
    k, v = _tokens(B, H, 1, d, 13)
    seq, counts = cache.new_seq(), torch.tensor([1, 0], dtype=torch.int32).cuda()
    seq[:, 0] = 62
    salad.cache_append(cache, k, v, seq, grid=(2, 2), counts=counts, seq_out=seq)     # 63
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = salad.cache_append(cache, k, v, seq, grid=(2, 2), counts=counts, seq_out=seq)
    assert out is seq
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert seq.cpu().tolist() == [[66, 1], [62, 0]]
    at = ref.new_seq()
    at[:, 0] = 62
    for _ in range(4):
        at = salad.cache_append(ref, k, v, at, grid=(2, 2), counts=counts)
    for name, x in _state(ref).items():
        np.testing.assert_array_equal(_state(cache)[name], x)


@needs_gpu
def test_append_reports_what_is_out_of_range():
    B, H, d = 2, 1, 64
    k, v = _tokens(B, H, 70, d, 14)

    def call(seq, counts=None, table=None):
        cache = _make(B, H, d, 2, seed=15)
        if table is not None:
            cache.page_table.copy_(torch.tensor(table, dtype=torch.int32))
        before = _state(cache)
        out = salad.cache_append(cache, k, v, torch.tensor(seq, dtype=torch.int32).cuda(),
                                 counts=None if counts is None else torch.tensor(counts, dtype=torch.int32).cuda())
        with pytest.raises(salad.SaladError) as e:
            salad.check_error()
        assert e.value.code == INVALID
        salad.check_error()
        return before, _state(cache), out.cpu().tolist()

    # Bad pages: nothing is written for those blocks, the open block is.
    before, after, out = call([[0, 0], [0, 0]], table=[[-1, 0], [5000, 1]])
    assert out == [[70, 1], [70, 1]]
    for name in ("k_pages", "v_pages", "k_scale", "v_scale"):
        np.testing.assert_array_equal(before[name], after[name])
    # A full table: 191 tokens are the most it holds.
    assert call([[150, 0], [0, 0]])[2] == [[191, 0], [70, 1]]
    # Lengths, slots and counts out of range are forced into it.
    assert call([[-3, 0], [0, 2]], counts=[1, 1])[2] == [[1, 0], [1, 0]]
    assert call([[0, 0], [0, 0]], counts=[71, -1])[2] == [[70, 1], [0, 0]]


@needs_gpu
def test_append_refusals_on_the_device():
    cache = _make(1, 2, 64, 2, seed=16)
    k, v = _tokens(1, 2, 4, 64, 17)
    seq = cache.new_seq()
    for bad in (dict(k=k[:, :1]), dict(k=k.float()), dict(v=v[:, :, :3]), dict(seq=seq[:, :1]), dict(seq=seq.long()),
                dict(seq=seq.cpu()), dict(counts=torch.zeros(2, dtype=torch.int32, device="cuda")),
                dict(seq_out=seq.long()), dict(cache=None), dict(grid=(2, 2), pairing="x")):
        with pytest.raises(ValueError):
            salad.cache_append(**{**dict(cache=cache, k=k, v=v, seq=seq), **bad})
    with pytest.raises(ValueError):
        salad.BlockCache(cache.k_pages, cache.v_pages, cache.k_scale, cache.v_scale, cache.k_tail[:, :1], cache.v_tail,
                         cache.page_table)
    with pytest.raises(ValueError):
        salad.BlockCache(cache.k_pages.view(torch.uint8), cache.v_pages, cache.k_scale, cache.v_scale, cache.k_tail,
                         cache.v_tail, cache.page_table)


def test_seq_out_apart_from_inputs():
    """seq_out may be seq; it may not lie in counts, positions, the cache, k or v."""
    at = A + 7 * M + 256
    for kw in (dict(k=at), dict(v=at), dict(counts=at), dict(positions=at), dict(seq_out=A), dict(seq_out=A + 3 * M),
               dict(seq_out=A + 4 * M), dict(seq_out=A + 6 * M)):
        assert _status(**kw) == INVALID, kw
