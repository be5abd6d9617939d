"""How many bits the attention over the 8-bit block cache keeps, against
float64 on the cache's own contents.

D, A and n are those of the tests of that call (a score's error, the mean of
|v| under the weights, the number of keys), with A's shares A_c of the closed
blocks and A_o of the open one.  For a closed block's key P_j = p_j s_j /
max_i(p_i s_i), s_j the power-of-two scale of its values, is held in fp16 times
a power of two: it is rounded by 2^-11 of itself, or by half of fp16's smallest
step, 2^-25, where that is more.  With up to 64 rows of a key head the factor
is 2^15, and the latter 2^-40 of the row's largest product; the open block's P
is rounded to bf16, by 2^-8 of itself.  With more rows the factor is between
2^11 and 2^15, and the open block is multiplied like a closed one.
"""
import math

import pytest
import torch

import sparse_linear_hybrid_top_b200 as salad
from tests.test_cache_attn import _held, _make, _q

needs_gpu = pytest.mark.gpu
FEW = dict(log_top=15, open_error=2.0 ** -8)
MANY = dict(log_top=11, open_error=2.0 ** -11)


def _bounded(cache, q, seq, log_top, open_error, o=None, frame=0, scale=None, held=None):
    """Checks o (default: the call's output) against the bound, row by row.
    held: keys, values and the values' scales of every sequence, where they are
    known otherwise than from the cache."""
    B, Hq, N, d = q.shape
    if o is None:
        o = salad.cache_attn(cache, q, seq, frame=frame, scale=scale)
    salad.check_error()
    o, q64 = o.cpu().double(), q.cpu().double()
    scale = 1 / math.sqrt(d) if scale is None else scale
    want = torch.zeros_like(o)
    worst = 0.0
    for b in range(B):
        k, v, vs = _held(cache, seq, b) if held is None else held[b]
        L = k.shape[1]
        closed = torch.arange(L) < L // 64 * 64
        for h in range(Hq):
            kh, vh, sh = (x[h // (Hq // cache.H)] for x in (k, v, vs))
            x = q64[b, h] @ kh.T * scale                                    # [N, L]
            p = torch.arange(L - N, L)
            end = (p // frame * frame + frame).clamp(max=L) if frame else torch.full((N,), L)
            see = (torch.arange(L) < end[:, None]) & (p[:, None] >= 0 if frame else True)
            D = d * 2.0 ** -22 * scale * (q64[b, h].abs() @ kh.abs().T).masked_fill(~see, 0).amax(1, keepdim=True)
            rows = see.any(1)
            w = torch.softmax(x[rows].masked_fill(~see[rows], -math.inf), 1)
            want[b, h, rows] = w @ vh
            fp16 = closed if open_error > 2.0 ** -11 else torch.ones_like(closed)
            a_c, a_o = (w * fp16) @ vh.abs(), (w * ~fp16) @ vh.abs()
            top = (w * sh * fp16).amax(1, keepdim=True)
            flush = 2.0 ** (-25 - log_top) * top * ((see[rows] & fp16).double() @ (vh.abs() / sh[:, None]))
            bound = (2.0 ** -11 * a_c + open_error * a_o + (2 * D[rows] + 2 * L * 2.0 ** -23) * (a_c + a_o) + flush +
                     2.0 ** -8 * 1.01 * want[b, h, rows].abs())
            err = (o[b, h, rows] - want[b, h, rows]).abs()
            worst = max(worst, float((err / bound).nan_to_num(nan=0.0).max())) if rows.any() else worst
            assert torch.all(err <= bound), worst
    return o, want


def _sink(H, d, n, at):
    """n keys with scores near 0 and values near 1, and one, token `at`, whose
    score is 18 and whose value is 0; the same for every head."""
    g = torch.Generator().manual_seed(n + at)
    k = torch.zeros(1, 1, n, d)
    k[..., 1] = torch.randn(1, 1, n, generator=g)
    k[0, 0, at, :2] = torch.tensor([18.0, 0.0])
    v = 1 + 0.25 * torch.randn(1, 1, n, d, generator=g)
    v[0, 0, at] = 0
    cache = salad.BlockCache.allocate(1, H, d, n // 64 + 1)
    k, v = (x.bfloat16().cuda().expand(1, H, n, d) for x in (k, v))
    return cache, salad.cache_append(cache, k, v, cache.new_seq())


def _sink_queries(rows, d):
    q = torch.zeros(1, 1, rows, d)
    q[..., 0] = 1 + torch.arange(rows) % 3 / 16
    q[..., 1] = 0.25
    return q.bfloat16().cuda()


def _check_sink(d, n, rows, at, **kernel):
    """256 heads leave a head's keys to one CTA (fewer would spread them, and the
    sink would stand beside a part of them only)."""
    q = _sink_queries(rows, d)
    cache, seq = _sink(256, d, n, at)
    o = salad.cache_attn(cache, q.expand(1, 256, rows, d), seq, scale=1.0)
    cache, seq = _sink(1, d, n, at)
    for h in (0, 100, 255):
        got, want = _bounded(cache, q, seq, o=o[:, h:h + 1], scale=1.0, **kernel)
        assert torch.all((got - want).abs() <= 0.02 * want.abs())


@needs_gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [1, 16, 32])
@pytest.mark.parametrize("at", [70, 8001 - 5])
def test_many_small_weights_beside_one_large_few_rows(d, rows, at):
    """A key that takes nearly all of the softmax and has no value: the output
    is the sum of 8000 weights of 2^-26 of the largest."""
    _check_sink(d, 8001, rows, at, **FEW)


@needs_gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows,lens", [(1, [1, 31, 64, 100, 128, 2111]), (16, [40, 640, 703]), (33, [63, 128, 700])])
def test_weights_few_rows(d, rows, lens):
    cache, seq = _make(len(lens), 2, d, lens, seed=rows)
    for frame in (0, 1):
        _bounded(cache, _q(len(lens), 2, rows, d, rows), seq, frame=frame, **FEW)


@needs_gpu
@pytest.mark.parametrize("rows", [1, 20, 60])
def test_open_block_of_any_size_few_rows(rows):
    """Values of the open block far larger and far smaller than those of the
    closed ones; rows behind the sequence hold larger ones still."""
    for e in (-90, -30, 30, 100, 121):
        cache, seq = _make(1, 2, 64, [64 * 3 + 37], seed=rows)
        slot = int(seq[0, 1])
        cache.v_tail[0, slot] *= 2.0 ** e
        cache.v_tail[0, slot, :, 37:] = 2.0 ** 127
        _bounded(cache, _q(1, 4, rows, 64, rows + 1), seq, **FEW)


@needs_gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [70, 300])
@pytest.mark.parametrize("at", [70, 8001 - 5])
def test_many_small_weights_beside_one_large_many_rows(d, rows, at):
    _check_sink(d, 8001, rows, at, **MANY)


@needs_gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows,lens", [(70, [70, 128, 700]), (130, [190, 2111]), (300, [333, 1500])])
def test_weights_many_rows(d, rows, lens):
    cache, seq = _make(len(lens), 2, d, lens, seed=rows)
    for frame in (0, 1):
        _bounded(cache, _q(len(lens), 2, rows, d, rows), seq, frame=frame, **MANY)


@needs_gpu
@pytest.mark.parametrize("rows", [70, 300])
def test_maxima_that_grow(rows):
    """Scores that rise from block to block by less, and by more, than what a
    row's maximum is raised at a time by."""
    for step in (0.5, 2.0, 6.0, 20.0):
        L = 64 * 12 + 17
        g = torch.Generator().manual_seed(rows)
        k = 0.25 * torch.randn(1, 1, L, 64, generator=g)
        k[0, 0, :, 0] = (torch.arange(L) // 64) * step * math.log(2)
        v = 1 + 0.25 * torch.randn(1, 1, L, 64, generator=g)
        cache = salad.BlockCache.allocate(1, 1, 64, 13)
        seq = salad.cache_append(cache, k.bfloat16().cuda(), v.bfloat16().cuda(), cache.new_seq())
        q = torch.randn(1, 1, rows, 64, generator=g)
        q[..., 0] = 1
        _bounded(cache, q.bfloat16().cuda(), seq, scale=1.0, **MANY)


@needs_gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows,H", [(1, 1), (1, 40), (20, 2), (60, 2), (70, 1), (300, 2)])
def test_values_near_the_largest_and_the_smallest(d, rows, H):
    """Means of values up to 2^127, whose sums are not floats, and of values
    around 2^-95: in the open block alone, in one CTA and in many."""
    kernel = MANY if rows > 64 else FEW
    g = torch.Generator().manual_seed(d + rows)
    for L in (rows + 20, rows + 300, 3001):
        k = torch.randn(1, H, L, d, generator=g)
        v = 1 - torch.randint(0, 3, (1, H, L, d), generator=g) / 4
        q = _q(1, H, rows, d, L)
        for size in (2.0 ** 127, 2.0 ** -95):
            cache = salad.BlockCache.allocate(1, H, d, L // 64 + 1)
            seq = salad.cache_append(cache, k.bfloat16().cuda(), (v * size).bfloat16().cuda(), cache.new_seq())
            if H == 40:
                o = salad.cache_attn(cache, q, seq)
                assert torch.all((o.double() <= size) & (o.double() >= size / 2))
            else:
                _bounded(cache, q, seq, **kernel)


def _as_held(x):
    """What a cache holds of x (bf16 [H, n, d]) and its scales [H, n], from the
    rule alone: full blocks of 64 tokens in e4m3, times the smallest 2^e for which
    none of the head's values passes 448 * 2^e; the rest as it is."""
    x = x.cpu().double()
    H, n, d = x.shape
    out, scales = x.clone(), torch.ones(H, n, dtype=torch.float64)
    for j in range(0, n, 64):
        block = x[:, j:j + 64]
        e = torch.log2(block.abs().amax((1, 2)) / 448).ceil()
        e += (block.abs().amax((1, 2)) > 448 * torch.exp2(e)).double()
        scales[:, j:j + 64] = torch.exp2(e)[:, None]
        if block.shape[1] == 64:
            s = torch.exp2(e)[:, None, None]
            out[:, j:j + 64] = (block / s).float().to(torch.float8_e4m3fn).double() * s
    return out, scales


@needs_gpu
@pytest.mark.parametrize("Hh,Wh,kernel", [(4, 5, FEW), (8, 12, MANY)])
def test_chunk_by_chunk_generation_against_dense_attention(Hh, Wh, kernel):
    """Three frames at a time, appended twice and attended frame by frame, against
    dense attention over all keys and values so far, turned by salad_rope and
    rounded by the cache's rule, which never saw the cache.  The bound tells the
    blocks' places: it does not hold with the values of two exchanged, nor with
    two of different frames exchanged whole."""
    H, d, F, plane = 3, 128, 12, Hh * Wh
    cache = salad.BlockCache.allocate(1, H, d, (F * plane + 63) // 64)
    cache.page_table.copy_(cache.page_table.flip(1))
    seq = cache.new_seq()
    g = torch.Generator().manual_seed(plane)
    q, k, v = (torch.randn(1, H, F * plane, d, generator=g).to(torch.bfloat16).cuda() for _ in range(3))
    turned = salad.rope(k, grid=(Hh, Wh))
    for f in range(0, F, 3):
        part = slice(f * plane, (f + 3) * plane)
        qr = salad.rope(q[:, :, part], grid=(Hh, Wh), offset=f * plane)
        for _ in range(2):
            after = salad.cache_append(cache, k[:, :, part], v[:, :, part], seq, grid=(Hh, Wh))
        seq = after
        kh, _ = _as_held(turned[0, :, :part.stop])
        vh, vs = _as_held(v[0, :, :part.stop])
        o, _ = _bounded(cache, qr, seq, frame=plane, held=[(kh, vh, vs)], **kernel)

    def exchanged(x, i, j):
        x = x.clone()
        x[:, 64 * i:64 * i + 64], x[:, 64 * j:64 * j + 64] = x[:, 64 * j:64 * j + 64].clone(), x[:, 64 * i:64 * i + 64].clone()
        return x

    wrong = [(kh, exchanged(vh, 0, 1), exchanged(vs, 0, 1))]
    if plane > 64:
        wrong.append(tuple(exchanged(x, F * plane // 64 - 4, F * plane // 64 - 1) for x in (kh, vh, vs)))
    for held in wrong:
        with pytest.raises(AssertionError):
            _bounded(cache, qr, seq, o=o, frame=plane, held=[held], **kernel)
