"""Attention over the 8-bit block cache: argument checks (no GPU) and GPU
parity with a float64 implementation that reads the cache's own contents.

Tolerances.  Scores are sums of d exact bf16 products in float32: off by at
most D = d 2^-22 * scale * max_j sum_c |q_c k_jc| (2^-22 allows for the tensor
core's truncated additions), which moves every weight by a factor within 1 +-
D, so the output by at most 2 D A, where A = sum_j p_j |v_j| / sum_j p_j.  P is
rounded to bf16 (2^-8 of each weight, so 2^-8 A) by the kernel of few rows.
The one of many rows multiplies c_j = v_j / s_j, s_j the power-of-two scale of
the key's block, by P_j = p_j s_j / max_i(p_i s_i), rounded to fp16: by 2^-11
of it, or by half of fp16's smallest step, 2^-25, where that is more.  The
latter adds at most F = 2^-25 max_i(p_i s_i) sum_j |c_j| / sum_j p_j.  The sums
of weights and of products are float32 (n 2^-23 A each for n keys: the longest
sequence's), and the output is rounded to bf16 (2^-8 |o|).  lse moves by D and
n 2^-23.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

import sparse_linear_hybrid_top_b200 as salad
from sparse_linear_hybrid_top_b200 import Cache, CacheAttnArgs, Strides, lib

INVALID, UNSUP, WS = -1, -2, -5
A = 0x100000         # a 256-aligned fake device address (never dereferenced)
M = 1 << 30


def _fake(cache=None, **kw):
    a = CacheAttnArgs()
    a.cache = Cache(A, A + M, A + 2 * M, A + 3 * M, A + 4 * M, A + 5 * M, A + 6 * M, 2, 3, 64, 1000, 500)
    for k, v in (cache or {}).items():
        setattr(a.cache, k, v)
    a.seq, a.q, a.o, a.lse = A + 7 * M, A + 8 * M, A + 9 * M, A + 10 * M
    a.q_st = a.o_st = Strides(6 * 4 * 64, 4 * 64, 64)
    a.Hq, a.N, a.frame, a.window, a.scale = 6, 4, 1, -1, 0.125
    a.workspace, a.workspace_bytes = A + 11 * M, 1 << 28
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _status(**kw):
    return lib.salad_cache_attn(ctypes.byref(_fake(**kw)), None)


def test_attn_argument_checks():
    assert lib.salad_cache_attn(None, None) == INVALID
    assert lib.salad_cache_attn_workspace_bytes(None) == 0
    for kw in (dict(cache=dict(k_pages=A + 8)), dict(cache=dict(H=4)), dict(cache=dict(blocks=0)), dict(Hq=0), dict(Hq=7),
               dict(Hq=258), dict(N=0), dict(N=262145), dict(seq=None), dict(counts=A + 2), dict(lse=A + 1), dict(frame=-1),
               dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(q=None), dict(o=A + 8),
               dict(q_st=Strides(1536, 256, 60)), dict(o_st=Strides(1536, 0, 64)), dict(o=A + 8 * M),
               dict(o=A + 8 * M + 128), dict(o=A), dict(lse=A + 8 * M), dict(lse=A + 9 * M)):
        assert _status(**kw) == INVALID, kw
        assert lib.salad_cache_attn_workspace_bytes(ctypes.byref(_fake(**kw))) == 0, kw
    assert _status(cache=dict(d=96)) == UNSUP


def test_attn_workspace():
    need = lib.salad_cache_attn_workspace_bytes(ctypes.byref(_fake()))
    assert need > 0 and need % 256 == 0
    assert _status(workspace=None) == WS
    assert _status(workspace_bytes=need - 1) == WS
    assert _status(workspace=A + 11 * M + 16) == WS
    if not torch.cuda.is_available():
        assert _status(workspace_bytes=need) in (UNSUP, -3)
        assert _status(workspace_bytes=need, lse=None, counts=A, q_st=Strides(0, 0, 0), window=7, frame=0) in (UNSUP, -3)


# ------------------------------------------------------------------- GPU ---
def _make(B, H, d, lens, blocks=None, seed=0, extra=3):
    """A cache whose first `lens` tokens are random and the rest of whose
    buffers (pages behind a sequence, tail rows behind it, the other slot) is NaN."""
    blocks = max(1, max(lens) // 64 + 1) if blocks is None else blocks
    cache = salad.BlockCache.allocate(B, H, d, blocks, pages=B * blocks + extra)
    g = torch.Generator().manual_seed(seed)
    table = torch.randperm(B * blocks + extra, generator=g)[:B * blocks].reshape(B, blocks).to(torch.int32)
    codes = torch.randint(0, 256, (2, *cache.k_pages.shape), generator=g, dtype=torch.uint8)
    codes[(codes & 127) == 127] = 1
    scale = torch.exp2(torch.randint(-9, -5, (2, *cache.k_scale.shape), generator=g).float())
    tail = torch.randn(2, *cache.k_tail.shape, generator=g).to(torch.bfloat16)
    slots = torch.randint(0, 2, (B,), generator=g)
    used = torch.zeros(len(codes[0]), dtype=torch.bool)
    for b, n in enumerate(lens):
        used[table[b, :n // 64].long()] = True
        table[b, n // 64:] = 10 ** 6 if b % 2 else -7
        tail[:, b, slots[b], :, n % 64:] = math.nan
        tail[:, b, 1 - slots[b]] = math.inf
    codes[:, ~used] = 127
    scale[:, ~used] = math.nan
    cache.k_pages.view(torch.uint8).copy_(codes[0])
    cache.v_pages.view(torch.uint8).copy_(codes[1])
    cache.k_scale.copy_(scale[0])
    cache.v_scale.copy_(scale[1])
    cache.k_tail.copy_(tail[0])
    cache.v_tail.copy_(tail[1])
    cache.page_table.copy_(table)
    return cache, torch.stack([torch.tensor(lens), slots], 1).to(torch.int32).cuda()


def _tail_scale(x):
    """The scale of an open block's rows [H, n, d]: that of a closed block."""
    top = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax(dim=(1, 2))
    part, e = torch.frexp(top / 448.0)
    return torch.ldexp(torch.ones_like(top), (e - (part == 0.5).int()).clamp(min=-100))


def _held(cache, seq, b):
    """Keys and values of sequence b as float64 [H, len, d], and the values' scales [H, len]."""
    n, slot = (int(x) for x in seq[b].cpu())
    out = []
    pages = cache.page_table[b, :n // 64].long().cpu()
    for name in ("k", "v"):
        x = getattr(cache, name + "_pages").cpu().double()[pages] * getattr(cache, name + "_scale").cpu().double()[pages][..., None, None]
        x = x.transpose(0, 1).reshape(cache.H, -1, cache.d)
        out.append(torch.cat([x, getattr(cache, name + "_tail").cpu().double()[b, slot, :, :n % 64]], 1))
    scale = cache.v_scale.cpu().double()[pages].T.repeat_interleave(64, 1)
    if n % 64:
        scale = torch.cat([scale, _tail_scale(out[1][:, n - n % 64:])[:, None].expand(-1, n % 64)], 1)
    return out[0], out[1], scale


def _reference(cache, q, seq, counts=None, frame=0, window=-1, scale=None):
    B, Hq, N, d = q.shape
    scale = 1 / math.sqrt(d) if scale is None else scale
    o = torch.zeros(B, Hq, N, d, dtype=torch.float64)
    mean_abs, flush = torch.zeros_like(o), torch.zeros_like(o)
    spread = torch.zeros(B, Hq, N, 1, dtype=torch.float64)
    lse = torch.full((B, Hq, N), -math.inf, dtype=torch.float64)
    q64 = q.cpu().double()
    for b in range(B):
        k, v, vs = _held(cache, seq, b)
        L, n = k.shape[1], N if counts is None else counts[b]
        for h in range(Hq):
            kh, vh = k[h // (Hq // cache.H)], v[h // (Hq // cache.H)]
            for i in range(n):
                p = L - n + i
                group = p // frame * frame if frame else L - n
                end = min(L, group + frame) if frame else L
                lo = max(0, group - window) if window >= 0 else 0
                if lo >= end:
                    continue
                x = kh[lo:end] @ q64[b, h, i] * scale
                spread[b, h, i] = (kh[lo:end].abs() @ q64[b, h, i].abs()).max() * scale
                w = torch.softmax(x, 0)
                lse[b, h, i] = torch.logsumexp(x, 0)
                o[b, h, i] = w @ vh[lo:end]
                mean_abs[b, h, i] = w @ vh[lo:end].abs()
                sc = vs[h // (Hq // cache.H), lo:end]
                flush[b, h, i] = 2.0 ** -25 * (w * sc).max() * (vh[lo:end].abs() / sc[:, None]).sum(0)
    return o, lse, mean_abs, flush, spread


def _check(cache, q, seq, counts=None, **kw):
    B, Hq, N, d = q.shape
    o = torch.full((B, Hq, N, d), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, Hq, N), 5.0, device="cuda")
    c = None if counts is None else torch.tensor(counts, dtype=torch.int32).cuda()
    got = salad.cache_attn(cache, q, seq, counts=c, o=o, lse=lse, **kw)
    assert got is o
    salad.check_error()
    want, wlse, mean_abs, flush, spread = _reference(cache, q, seq, counts, **kw)
    o, lse = o.cpu().double(), lse.cpu().double()
    D = d * 2.0 ** -22 * spread
    n = int(seq[:, 0].max()) * 2.0 ** -23
    for b in range(B):
        m = N if counts is None else counts[b]
        assert torch.all(o[b, :, m:] == 5.0) and torch.all(lse[b, :, m:] == 5.0)     # rows behind a count
        err = (o[b, :, :m] - want[b, :, :m]).abs()
        bound = (2.0 ** -8 + 2 * D[b, :, :m] + 2 * n) * mean_abs[b, :, :m] + flush[b, :, :m] + 2.0 ** -8 * want[b, :, :m].abs() * 1.01
        assert torch.all(err <= bound), float((err - bound).max())
        empty = torch.isinf(wlse[b, :, :m])
        assert torch.equal(torch.isinf(lse[b, :, :m]) & (lse[b, :, :m] < 0), empty)
        assert torch.all(o[b, :, :m][empty] == 0)
        gap = (lse[b, :, :m] - wlse[b, :, :m]).abs()[~empty]
        assert torch.all(gap <= (D[b, :, :m, 0] + n + 4e-6 * (1 + wlse[b, :, :m].abs()))[~empty])


def _q(B, H, N, d, seed):
    g = torch.Generator().manual_seed(seed)
    return (1.5 * torch.randn(B, H, N, d, generator=g)).to(torch.bfloat16).cuda()


needs_gpu = pytest.mark.gpu
LENS = [0, 1, 31, 33, 63, 64, 65, 128, 200, 517]


@needs_gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("frame,window", [(0, -1), (1, -1), (1, 40), (7, 0), (0, 33), (64, 100)])
def test_single_tokens_of_every_length(d, frame, window):
    cache, seq = _make(len(LENS), 2, d, LENS, seed=d + frame)
    _check(cache, _q(len(LENS), 2, 1, d, 1), seq, frame=frame, window=window)


@needs_gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,Hq,H", [(3, 2, 2), (16, 4, 2), (17, 3, 3), (5, 6, 1), (40, 2, 1), (70, 2, 2), (130, 3, 1), (300, 1, 1)])
@pytest.mark.parametrize("frame,window", [(0, -1), (1, 50), (13, -1)])
def test_chunks(d, N, Hq, H, frame, window):
    """Rows of every tile height, sequences shorter than the chunk among them
    (rows before the first token see nothing), and padded batches."""
    lens = [0, N // 2, N, 64 * ((N + 63) // 64), N + 517]
    counts = [N, N, max(1, N - 1), 0, N]
    cache, seq = _make(len(lens), H, d, lens, seed=N + Hq)
    _check(cache, _q(len(lens), Hq, N, d, 2), seq, counts, frame=frame, window=window)


@needs_gpu
@pytest.mark.parametrize("N,Hq,H,length", [(1, 1, 1, 2100), (1, 8, 2, 2111), (4, 12, 3, 1984), (200, 2, 1, 2150), (513, 1, 1, 2049)])
def test_long_sequences(N, Hq, H, length):
    for d in (64, 128):
        cache, seq = _make(1, H, d, [length], seed=length)
        _check(cache, _q(1, Hq, N, d, 3), seq, frame=1)
        _check(cache, _q(1, Hq, N, d, 4), seq, frame=0, scale=0.3)


@needs_gpu
def test_table_much_wider_than_the_sequences():
    cache, seq = _make(2, 2, 128, [70, 3], blocks=4000, seed=5, extra=0)
    _check(cache, _q(2, 2, 1, 128, 6), seq, frame=1)
    _check(cache, _q(2, 2, 3, 128, 6), seq, frame=1)


@needs_gpu
def test_strided_queries_and_outputs():
    B, Hq, N, d = 2, 4, 5, 64
    cache, seq = _make(B, 2, d, [90, 130], seed=6)
    q = _q(B, N, Hq, d, 7).transpose(1, 2)                     # token-major
    out = torch.full((B, N, Hq + 1, 2 * d), 3.0, dtype=torch.bfloat16, device="cuda")
    o = out[:, :, :Hq, d:].transpose(1, 2)
    salad.cache_attn(cache, q, seq, frame=1, o=o)
    assert torch.equal(o, salad.cache_attn(cache, q.contiguous(), seq, frame=1))
    o.fill_(3.0)
    assert torch.all(out == 3.0)
    one = _q(1, 1, N, d, 8).expand(B, Hq, N, d)                # a broadcast input
    assert torch.equal(salad.cache_attn(cache, one, seq), salad.cache_attn(cache, one.contiguous(), seq))


@needs_gpu
@pytest.mark.parametrize("N", [1, 100])
def test_infinities_and_nan_reach_only_the_rows_that_see_them(N):
    """In the open block (per value) and in closed blocks (the whole block and head)."""
    d, L = 64, 300
    q = _q(1, 2, N, d, 9)

    def call(change, **kw):
        cache, seq = _make(1, 2, d, [L], seed=9)
        change(cache, int(seq[0, 1]))
        o = salad.cache_attn(cache, q, seq, **kw)
        salad.check_error()
        return o.float()

    kw = dict(frame=1, window=20)
    clean = call(lambda c, s: None, **kw)
    p = torch.arange(L - N, L)

    def sees(lo, hi):                                          # rows that see a key in [lo, hi)
        return ((p >= lo) & (p - 20 < hi)).cuda()

    def tail_v(c, s):
        c.v_tail[0, s, 1, 5, 7] = math.inf                     # token 261, head 1

    o, rows = call(tail_v, **kw), sees(261, 262)
    assert torch.all(torch.isinf(o[0, 1, rows, 7])) and torch.equal(o[0, 0], clean[0, 0])
    o[0, 1, rows, 7] = clean[0, 1, rows, 7]
    assert torch.equal(o, clean)

    def tail_k(c, s):
        c.k_tail[0, s, 0, 5, 7] = math.nan

    o = call(tail_k, **kw)
    assert torch.all(torch.isnan(o[0, 0, rows])) and torch.equal(o[0, 0, ~rows], clean[0, 0, ~rows])
    assert torch.equal(o[0, 1], clean[0, 1])
    for name in ("k", "v"):
        def block(c, s, name=name):                            # block 3, head 0: tokens 192 to 255
            at = int(c.page_table[0, 3])
            getattr(c, name + "_scale")[at, 0] = math.nan
            getattr(c, name + "_pages").view(torch.uint8)[at, 0] = 127
        o, rows = call(block, **kw), sees(192, 256)
        assert torch.all(torch.isnan(o[0, 0, rows])) and torch.equal(o[0, 0, ~rows], clean[0, 0, ~rows])
        assert torch.equal(o[0, 1], clean[0, 1])


@needs_gpu
@pytest.mark.parametrize("N", [1, 100])
def test_scales_far_apart(N):
    """Value blocks of very different size: the weights do not depend on it."""
    d, L = 64, 64 * 9 + 5
    cache, seq = _make(1, 1, d, [L], seed=10)
    for j, e in enumerate((0, -100, 90, -60, 3, -100, 20, 0, -3)):
        cache.v_scale[int(cache.page_table[0, j])] = 2.0 ** e
    for j, e in enumerate((-6, -8, -7, -100, -30, -6, -9, -5, -6)):
        cache.k_scale[int(cache.page_table[0, j])] = 2.0 ** e
    _check(cache, _q(1, 1, N, d, 11), seq, frame=1)


@needs_gpu
@pytest.mark.parametrize("N", [1, 100])
def test_out_of_range_is_reported(N):
    d = 64
    q = _q(1, 1, N, d, 12)

    def code(call):
        o = call()
        torch.cuda.synchronize()
        with pytest.raises(salad.SaladError) as e:
            salad.check_error()
        assert e.value.code == INVALID
        salad.check_error()
        return o

    cache, seq = _make(1, 1, d, [300], seed=12)
    for entry in (-1, 10 ** 7):                       # the block is left out
        cache.page_table[0, 2] = entry
        o = code(lambda: salad.cache_attn(cache, q, seq))
        assert torch.all(torch.isfinite(o))
    bad = seq.clone()
    bad[0, 0] = -5
    cache, seq = _make(1, 1, d, [300], seed=12)
    assert torch.all(code(lambda: salad.cache_attn(cache, q, bad)) == 0)
    counts = torch.tensor([N + 1], dtype=torch.int32).cuda()
    assert torch.equal(code(lambda: salad.cache_attn(cache, q, seq, counts=counts)), salad.cache_attn(cache, q, seq))


@needs_gpu
@pytest.mark.parametrize("N", [1, 90])
def test_captured_and_on_another_stream(N):
    d = 128
    cache, seq = _make(2, 2, d, [700, 333], seed=13)
    q = _q(2, 4, N, d, 14)
    want = salad.cache_attn(cache, q, seq, frame=1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = salad.cache_attn(cache, q, seq, frame=1, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    o = torch.empty_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        salad.cache_attn(cache, q, seq, frame=1, o=o)
    q2 = _q(2, 4, N, d, 15)
    q.copy_(q2)
    seq[:, 0] -= 64                                   # the graph reads the lengths on the device
    seq[0, 0] = 640
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, salad.cache_attn(cache, q2, seq, frame=1))
    # Two calls at once, each with its own workspace.
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (a, b):
        s.wait_stream(torch.cuda.current_stream())
    outs = [salad.cache_attn(cache, q2, seq, frame=1, stream=s) for s in (a, b) for _ in range(10)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, o) for x in outs)
    salad.check_error()


@needs_gpu
def test_chunk_by_chunk_generation():
    """Chunks appended and attended as a video is generated, against dense
    attention over everything so far: the cache's rounding (e4m3, 2^-4 of a
    value) is the difference, and none of it is there before a block closes."""
    B, H, d, Hh, Wh, F = 1, 3, 128, 4, 5, 12
    plane = Hh * Wh
    cache = salad.BlockCache.allocate(B, H, d, (F * plane + 63) // 64)
    seq = cache.new_seq()
    g = torch.Generator().manual_seed(16)
    q, k, v = (torch.randn(B, H, F * plane, d, generator=g).to(torch.bfloat16).cuda() for _ in range(3))
    for f in range(0, F, 3):
        part = slice(f * plane, (f + 3) * plane)
        qr = salad.rope(q[:, :, part], grid=(Hh, Wh), offset=f * plane)
        for _ in range(2):                            # two denoising steps write the same place
            nxt = salad.cache_append(cache, k[:, :, part], v[:, :, part], seq, grid=(Hh, Wh))
        o = salad.cache_attn(cache, qr, nxt)
        seq = nxt
        kr = salad.rope(k[:, :, :part.stop], grid=(Hh, Wh))
        x = qr.double() @ kr.double().transpose(-1, -2) / math.sqrt(d)
        want = torch.softmax(x, -1) @ v[:, :, :part.stop].double()
        if part.stop < 64:                            # all tokens still in bf16
            assert float((o.double() - want).abs().max()) <= 2.0 ** -7 * float(v.double().abs().max())
        # Values are off by 2^-4 |v| at most and weights by a factor within
        # exp(+-2 max|score error|); in the mean, rounding errors of independent
        # sign: the bars below are the worst case over the batch.
        ds = float((2.0 ** -4 * (qr.double().abs() @ kr.double().abs().transpose(-1, -2)) / math.sqrt(d)).max())
        top = float(v.double().abs().max())
        assert float((o.double() - want).abs().max()) <= (math.exp(min(2 * ds, 20.0)) - 1 + 2.0 ** -4 + 2.0 ** -7) * top
        ref, _, mean_abs, flush, spread = _reference(cache, qr, nxt)
        bound = (2.0 ** -8 + 2 * d * 2.0 ** -22 * spread + 2 * 240 * 2.0 ** -23) * mean_abs + flush + 2.0 ** -8 * ref.abs() * 1.01
        assert torch.all((o.cpu().double() - ref).abs() <= bound)
    assert int(seq[0, 0]) == F * plane
    salad.check_error()


@needs_gpu
def test_single_token_generation_in_one_graph():
    """rope, append (seq advanced in place) and attention captured once and
    replayed for every token, against the same calls made one by one."""
    B, H, Hq, d, T = 2, 2, 4, 64, 70
    g = torch.Generator().manual_seed(17)
    toks = [[torch.randn(B, h, 1, d, generator=g).to(torch.bfloat16).cuda() for h in (Hq, H, H)] for _ in range(T)]
    pos = torch.zeros(B, 1, 3, dtype=torch.int32, device="cuda")

    def step(cache, seq, q, k, v):
        qr = salad.rope(q, positions=pos)
        salad.cache_append(cache, k, v, seq, positions=pos, seq_out=seq)
        return salad.cache_attn(cache, qr, seq, frame=1)

    one, two = (salad.BlockCache.allocate(B, H, d, 2) for _ in range(2))
    s1, s2 = one.new_seq(), two.new_seq()
    q, k, v = (t.clone() for t in toks[0])
    step(two, s2, q, k, v)                            # warm up, then start again
    s2.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(two, s2, q, k, v)
    s2.zero_()
    for i, (a, b, c) in enumerate(toks):
        pos.fill_(i)
        want = step(one, s1, a, b, c)
        for x, y in ((q, a), (k, b), (v, c)):
            x.copy_(y)
        graph.replay()
        assert torch.equal(out, want), i
    assert s1.cpu().tolist() == s2.cpu().tolist() == [[T, 1], [T, 1]]
    salad.check_error()


@needs_gpu
def test_attn_refusals_on_the_device():
    cache, seq = _make(1, 2, 64, [10], blocks=300, seed=18)
    q = _q(1, 2, 3, 64, 19)
    for bad in (dict(q=q.half()), dict(q=q[0]), dict(q=q[..., :32]), dict(q=q.cpu()), dict(seq=seq.long()),
                dict(seq=seq[0]), dict(counts=seq[0]), dict(o=q[:, :1]), dict(lse=torch.zeros(1, 2, 3).cuda().half()),
                dict(lse=torch.zeros(1, 2, 4).cuda()), dict(cache=0), dict(workspace=torch.zeros(16, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            salad.cache_attn(**{**dict(cache=cache, q=q, seq=seq), **bad})
    for bad in (dict(o=q), dict(frame=-1), dict(scale=-1.0), dict(q=_q(1, 3, 3, 64, 20))):
        with pytest.raises(salad.SaladError) as e:
            salad.cache_attn(**{**dict(cache=cache, q=q, seq=seq), **bad})
        assert e.value.code == INVALID


def test_outputs_apart_from_inputs():
    """o and lse may not lie in the cache, in seq or in counts."""
    for at in (A + 2 * M, A + 4 * M, A + 6 * M, A + 7 * M):
        assert _status(lse=at) == INVALID and _status(o=at) == INVALID
    assert _status(counts=A + 10 * M) == INVALID
    assert _status(counts=A + 9 * M) == INVALID
    # Key tiles of the rows of one key head beyond 31 bits.
    wide = dict(N=262144, Hq=3, lse=None, workspace=None, q_st=Strides(3 << 24, 1 << 24, 64), o_st=Strides(3 << 24, 1 << 24, 64))
    assert _status(cache=dict(blocks=1 << 23), **wide) == UNSUP
    assert _status(cache=dict(blocks=1 << 21), **wide) == WS


@needs_gpu
@pytest.mark.parametrize("N,Hq,H", [(1, 5, 1), (2, 4, 2), (65, 1, 1), (40, 8, 2)])
@pytest.mark.parametrize("lens", [
    [2111 - 131 * i for i in range(16)],
    [0, 5000, 0, 0, 64, 1, 3000, 0, 63, 128, 0],
    [1, 2, 3, 4, 5, 6, 7, 4001],
])
def test_unequal_sequences(N, Hq, H, lens):
    """Runs of work that begin and end inside sequences, between them, and skip
    empty ones; every other sequence has fewer rows, some none.  (Sums of up to
    5000 keys: the bound takes n from the longest.)"""
    cache, seq = _make(len(lens), H, 64, lens, seed=N)
    counts = [(N, max(1, N // 2), 0)[i % 3] for i in range(len(lens))]
    q = _q(len(lens), Hq, N, 64, 7 * N)
    _check(cache, q, seq, frame=1)
    _check(cache, q, seq, counts)


@needs_gpu
@pytest.mark.parametrize("B,N", [(512, 1), (513, 1), (513, 70)])
def test_many_sequences(B, N):
    """As many sequences as a CTA sums (512), and more."""
    lens = [(i * 37) % 150 for i in range(B)]
    cache, seq = _make(B, 1, 64, lens, seed=B)
    counts = [N if i % 3 else i % 2 for i in range(B)]
    _check(cache, _q(B, 1, N, 64, B), seq, counts, frame=1)


@needs_gpu
@pytest.mark.parametrize("Hq,N", [(1, 1), (3, 2), (1, 20), (2, 40)])
def test_one_key_head_over_many_ctas(Hq, N):
    """More than 128 parts of a row, of a sequence longer than its pool: many
    blocks are the same page.  (60001 keys: n 2^-23 is 0.7%, which the bound has.)"""
    n = 60001
    cache, seq = _make(1, 1, 64, [2111], blocks=n // 64, seed=3)
    cache.page_table[0] = cache.page_table[0, torch.arange(n // 64) % 32]
    seq[0, 0] = n
    cache.k_tail.copy_(torch.randn(cache.k_tail.shape).bfloat16())
    cache.v_tail.copy_(torch.randn(cache.v_tail.shape).bfloat16())
    _check(cache, _q(1, Hq, N, 64, N), seq, frame=1)


@needs_gpu
def test_sequences_share_pages():
    """Two sequences with a common prefix name the same pages."""
    cache, seq = _make(2, 2, 128, [700, 900], seed=11)
    cache.page_table[1, :10] = cache.page_table[0, :10]
    for N in (1, 70):
        _check(cache, _q(2, 4, N, 128, N), seq, frame=1)


@needs_gpu
@pytest.mark.parametrize("N", [1, 100])
def test_calls_at_the_same_time_on_two_streams(N):
    """Two calls that overlap, each with a workspace of its own."""
    cache, seq = _make(2, 4, 128, [2100, 777], seed=5)
    q = [_q(2, 8, N, 128, s) for s in (1, 2)]
    want = [salad.cache_attn(cache, x, seq, frame=1) for x in q]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            got[i].append(salad.cache_attn(cache, q[i], seq, frame=1, stream=s))
    torch.cuda.synchronize()
    salad.check_error()
    for i in range(2):
        for o in got[i]:
            assert torch.equal(o, want[i])       # the split does not depend on timing


@needs_gpu
@pytest.mark.parametrize("N,Hq", [(33, 2), (64, 2), (11, 10)])
def test_rows_at_the_border_of_two_kernels(N, Hq):
    """33 to 64 rows of a key head: another kernel where the tables have room for
    much work."""
    for blocks in (20, 1600):
        cache, seq = _make(2, 2, 64, [700, 1200], blocks=blocks, seed=blocks)
        _check(cache, _q(2, Hq, N, 64, N), seq, frame=1)
        _check(cache, _q(2, Hq, N, 64, N), seq, [N, 5], window=100)


@needs_gpu
def test_no_gradient_is_lost():
    """Neither cache call has a backward pass: under grad mode it refuses inputs that ask for one."""
    cache, seq = _make(1, 2, 64, [100])
    x = torch.randn(1, 2, 3, 64, device="cuda", dtype=torch.bfloat16)
    g = x.clone().requires_grad_()
    for call in (lambda: salad.cache_attn(cache, g, seq), lambda: salad.cache_append(cache, g, x, seq),
                 lambda: salad.cache_append(cache, x, g, seq)):
        with pytest.raises(ValueError, match="backward"):
            call()
    with torch.no_grad():
        assert torch.equal(salad.cache_attn(cache, g, seq), salad.cache_attn(cache, x, seq))


@needs_gpu
def test_pages_behind_four_gigabytes():
    """A pool of more than 2^32 bytes, the sequence in its last pages: the same
    bits as in a small pool, from the append and from both attention kernels."""
    B, H, d, n = 1, 8, 128, 700
    g = torch.Generator().manual_seed(2)
    k, v = (torch.randn(B, H, n, d, generator=g).bfloat16().cuda() for _ in range(2))
    small = salad.BlockCache.allocate(B, H, d, 11)
    big = salad.BlockCache.allocate(B, H, d, 11, pages=68000)
    assert big.k_pages.numel() > 1 << 32
    big.page_table.copy_(67989 + torch.arange(11))
    after = [salad.cache_append(c, k, v, c.new_seq(), grid=(4, 5)) for c in (small, big)]
    assert torch.equal(after[0], after[1])
    for name in ("k_pages", "v_pages"):
        x, y = getattr(small, name).view(torch.uint8), getattr(big, name).view(torch.uint8)
        assert torch.equal(x[:10], y[67989:67999])
    assert torch.equal(small.k_scale[:10], big.k_scale[67989:67999])
    for N in (1, 70):
        q = _q(B, H, N, d, N)
        assert torch.equal(salad.cache_attn(small, q, after[0], frame=1), salad.cache_attn(big, q, after[1], frame=1))
    salad.check_error()
