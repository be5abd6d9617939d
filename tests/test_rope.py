"""Rotary positions with several axes: argument checks (no GPU) and GPU parity
with a float64 implementation.

Tolerances.  A result is rounded once to the tensors' type: half a step,
eps(type) / 2 relative.  Before that the kernel multiplies float32 values by a
cosine and a sine rounded once to float32 (2^-24 relative) from an angle of
which float64 leaves 2 * 2^-53 |pos| rad at far positions (the rate's and the
product's rounding); two products and a sum add 3 * 2^-24.  So, for a pair
(u, w) with |x| = max(|u|, |w|), the second part is at most
    |x| (2 * 2^-24 + 2 * 2 |pos| 2^-53 + 2 * 3 * 2^-24) < |x| (4.8e-7 + 4 |pos| 2^-53),
taken as 1.1e-6 |x| + 4 |pos| 2^-53 |x|.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle
import sparse_linear_hybrid_top_b200 as salad
from sparse_linear_hybrid_top_b200 import RopeArgs, Strides, lib

INVALID, UNSUP = -1, -2
A = 0x10000          # a 256-aligned fake device address (never dereferenced)
M = 1 << 26


def _args(**kw):
    """A valid call on q [1,2,100,64] and k [1,1,100,64] (fake addresses)."""
    a = RopeArgs()
    a.q, a.q_out, a.k, a.k_out = A, A + M, A + 2 * M, A + 3 * M
    a.q_st = a.qo_st = Strides(2 * 100 * 64, 100 * 64, 64)
    a.k_st = a.ko_st = Strides(100 * 64, 100 * 64, 64)
    a.B, a.Hq, a.Hk, a.N, a.d = 1, 2, 1, 100, 64
    a.Hh, a.Wh = 5, 10
    a.split = (ctypes.c_int * 3)(24, 20, 20)
    a.base = 10000.0
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _status(**kw):
    return lib.salad_rope(ctypes.byref(_args(**kw)), None)


def test_rope_argument_checks():
    ints = lambda *v: (ctypes.c_int * 3)(*v)  # noqa: E731
    assert lib.salad_rope(None, None) == INVALID
    for kw in (dict(q=None), dict(q=A + 8), dict(q_out=None), dict(k=None), dict(k_out=None), dict(Hk=0),
               dict(B=0), dict(N=0), dict(N=262145), dict(Hq=257), dict(Hq=0),
               dict(split=ints(24, 20, 18)), dict(split=ints(25, 19, 20)), dict(split=ints(-2, 46, 20)),
               dict(split=ints(64, 64, -64)), dict(base=1.0), dict(base=float("inf")), dict(base=float("nan")),
               dict(pairing=2), dict(inverse=2), dict(Hh=0), dict(Wh=0), dict(Hh=1 << 20, Wh=1 << 20),
               dict(offset=-1), dict(offset=0x7fffffff - 99), dict(positions=A + 2), dict(positions_batched=2),
               dict(q_st=Strides(12800, 6400, 60)),           # rows off 16 bytes
               dict(q_st=Strides(12800, -6400, 64)),
               dict(qo_st=Strides(12800, 0, 64)),             # two heads on one output row
               dict(qo_st=Strides(12800, 6400, 32)),          # rows overlap
               dict(q_out=A + 64), dict(q_out=A + 2 * M), dict(k_out=A + M), dict(k_out=A),
               dict(q_out=A, qo_st=Strides(12800, 64, 128)),  # in place with other strides
               dict(k=A, k_out=A, q_out=A)):                  # the same tensor twice
        assert _status(**kw) == INVALID, kw
    for kw in (dict(dtype=3), dict(d=8), dict(d=272), dict(d=72)):
        assert _status(**kw) == UNSUP, kw


def test_rope_accepts_valid_layouts():
    """Valid calls pass every check: without a device they stop at the device lookup."""
    if torch.cuda.is_available():
        pytest.skip("fake addresses must not reach a launch")
    row = 3 * 2 * 64   # [B, N, 3, H, d] slices
    for kw in (dict(), dict(q_out=A), dict(k=None, k_out=None, Hk=0), dict(positions=A, Hh=0, Wh=0),
               dict(q_st=Strides(0, 0, 64)), dict(offset=0x7fffffff - 100),
               dict(Hk=2, q=A, q_out=A, k=A + 256, k_out=A + 256, q_st=Strides(100 * row, 64, row),
                    qo_st=Strides(100 * row, 64, row), k_st=Strides(100 * row, 64, row), ko_st=Strides(100 * row, 64, row))):
        assert _status(**kw) in (UNSUP, -3), kw


def test_rope_binding_refuses_bad_tensors():
    q = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        salad.rope(q, grid=(2, 2))                       # a host tensor
    with pytest.raises(ValueError):
        salad.rope(q[0], grid=(2, 2))
    with pytest.raises(ValueError):
        salad.rope(q.double(), grid=(2, 2))


# ------------------------------------------------------------------- GPU ---
def _angles(pos, split, base):
    """[..., d/2] float64 angles of positions [..., 3]."""
    cols = []
    for axis, g in enumerate(split):
        for i in range(g // 2):
            cols.append(pos[..., axis] * base ** (-2.0 * i / g))
    return np.stack(cols, axis=-1)


def _rotate(x, angles, pairing, inverse=False):
    """x [B,H,N,d], angles [B,N,d/2]; and the largest magnitude of each element's pair."""
    c, s = np.cos(angles)[:, None], np.sin(angles)[:, None] * (-1 if inverse else 1)
    d = x.shape[-1]
    u = np.arange(0, d, 2) if pairing == "adjacent" else np.arange(d // 2)
    w = u + 1 if pairing == "adjacent" else u + d // 2
    out, big = np.empty_like(x), np.empty_like(x)
    out[..., u] = x[..., u] * c - x[..., w] * s
    out[..., w] = x[..., u] * s + x[..., w] * c
    big[..., u] = big[..., w] = np.maximum(np.abs(x[..., u]), np.abs(x[..., w]))
    return out, big


def _check(got, x, pos, split, pairing, base=10000.0, inverse=False):
    x64 = x.detach().cpu().double().numpy()
    want, big = _rotate(x64, _angles(pos.astype(np.float64), split, base), pairing, inverse)
    far = float(np.abs(pos).max())
    err = np.abs(got.cpu().double().numpy() - want)
    tiny = 2.0 ** -25 if x.dtype == torch.float16 else 0.0      # half a step of fp16's subnormals
    bound = torch.finfo(x.dtype).eps / 2 * np.abs(want) + (1.1e-6 + 4 * far * 2.0 ** -53) * big * \
        (1 + torch.finfo(x.dtype).eps) + tiny
    assert np.all(err <= bound), float((err - bound).max())


def _grid(N, Hh, Wh, offset=0):
    p = np.arange(N) + offset
    return np.stack([p // (Hh * Wh), p // Wh % Hh, p % Wh], axis=-1)[None]


def _draw(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype).cuda()


needs_gpu = pytest.mark.gpu


@needs_gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=str)
@pytest.mark.parametrize("pairing", ["adjacent", "halves"])
@pytest.mark.parametrize("B,Hq,Hk,N,d", [(1, 1, 0, 1, 64), (2, 3, 1, 37, 128), (1, 12, 12, 930, 128), (3, 5, 2, 65, 64),
                                         (1, 2, 7, 129, 96), (2, 1, 1, 33, 16), (1, 9, 0, 50, 256)])
def test_rope_on_a_grid(dtype, pairing, B, Hq, Hk, N, d):
    q = _draw((B, Hq, N, d), dtype, 1)
    k = _draw((B, Hk, N, d), dtype, 2) if Hk else None
    dy = 2 * (d // 6)
    split = (d - 2 * dy, dy, dy)
    pos = np.repeat(_grid(N, 5, 7, 3), B, 0)
    for inverse, call in ((False, salad.rope), (True, salad.rope_backward)):
        out = call(q, k, grid=(5, 7), offset=3, pairing=pairing)
        for got, x in zip(out if Hk else (out,), (q, k)):
            _check(got, x, pos, split, pairing, inverse=inverse)
    salad.check_error()


@needs_gpu
@pytest.mark.parametrize("split", [(44, 42, 42), (0, 64, 64), (128, 0, 0), (2, 0, 126)])
@pytest.mark.parametrize("far", [1, 4096, 1 << 24, 0x7fffffff])
def test_rope_with_given_positions(split, far):
    """Positions of either sign up to the ends of int32, per sample and shared."""
    B, H, N, d = 2, 3, 41, 128
    g = np.random.default_rng(far)
    pos = g.integers(-far, far + 1, size=(B, N, 3)).astype(np.int32)
    pos[0, 0] = far
    q = _draw((B, H, N, d), torch.float32, 5)
    at = torch.from_numpy(pos).cuda()
    _check(salad.rope(q, positions=at, split=split), q, pos, split, "adjacent")
    _check(salad.rope(q, positions=at[1].contiguous(), split=split, base=500000.0), q, np.repeat(pos[1:], B, 0), split,
           "adjacent", base=500000.0)


@needs_gpu
def test_rope_equals_the_linear_branch_encoding():
    """The default split and grid are the oracle's 3-D encoding."""
    F, Hh, Wh, d = 3, 4, 5, 128
    x = _draw((1, 1, F * Hh * Wh, d), torch.float32, 6)
    got = salad.rope(x, grid=(Hh, Wh))[0, 0].cpu().double().numpy()
    want = oracle.rope3d_rotate(x[0, 0].cpu(), oracle.rope3d_angles(F * Hh * Wh, d, F, Hh, Wh))
    np.testing.assert_allclose(got, want, rtol=0, atol=1.2e-6 * float(x.abs().max()))


@needs_gpu
def test_rope_strided_in_place_and_interleaved():
    B, H, N, d = 2, 3, 50, 64
    pos = np.repeat(_grid(N, 3, 4), B, 0)
    split = (24, 20, 20)
    # Token-major slices of one projection output, turned in place; the values stay.
    qkv = _draw((B, N, 3, H, d), torch.bfloat16, 7)
    before = qkv.clone()
    q, k, v = (qkv[:, :, i].transpose(1, 2) for i in range(3))
    x, y = q.clone(), k.clone()
    out = salad.rope(q, k, grid=(3, 4), q_out=q, k_out=k)
    assert out[0].data_ptr() == q.data_ptr()
    _check(q, x, pos, split, "adjacent")
    _check(k, y, pos, split, "adjacent")
    assert torch.equal(v, before[:, :, 2].transpose(1, 2))
    # A broadcast input, and an output inside a larger buffer whose rest stays.
    one = _draw((1, 1, N, d), torch.bfloat16, 8)
    big = torch.full((B, H, N + 5, 2 * d), 7.0, dtype=torch.bfloat16, device="cuda")
    salad.rope(one.expand(B, H, N, d), grid=(3, 4), q_out=big[:, :, 2:N + 2, :d])
    _check(big[:, :, 2:N + 2, :d], one.expand(B, H, N, d), pos, split, "adjacent")
    big[:, :, 2:N + 2, :d] = 7.0
    assert torch.all(big == 7.0)
    with pytest.raises(salad.SaladError):
        salad.rope(one, grid=(3, 4), q_out=one.as_strided(one.shape, (0, 0, d // 2, 1)))


@needs_gpu
def test_rope_is_orthogonal_and_backward_matches_differences():
    B, H, N, d = 1, 2, 9, 64
    at = torch.randint(-50, 50, (B, N, 3), dtype=torch.int32).cuda()
    x, dy = _draw((B, H, N, d), torch.float32, 9), _draw((B, H, N, d), torch.float32, 10)
    dx = salad.rope_backward(dy, positions=at)
    # <R x, dy> is linear in x: its difference along any direction is <x', R^T dy>.
    step = _draw((B, H, N, d), torch.float32, 11)
    f = lambda t: float((salad.rope(t, positions=at).double() * dy.double()).sum())  # noqa: E731
    num = (f(x + step) - f(x - step)) / 2
    ana = float((dx.double() * step.double()).sum())
    # Each of the 2 * 1152 terms is off by at most 1.1e-6 * |x||dy| (about 20).
    assert abs(num - ana) <= 2 * B * H * N * d * 1.1e-6 * 20
    back = salad.rope_backward(salad.rope(x, positions=at), positions=at)
    assert float((back - x).abs().max()) <= 2 * 1.1e-6 * math.sqrt(2) * float(x.abs().max()) * 1.01


@needs_gpu
def test_rope_keeps_infinities_and_nan_in_their_pairs():
    x = torch.ones(1, 1, 3, 64, device="cuda")
    x[0, 0, 1, 10], x[0, 0, 2, 21] = math.inf, math.nan
    y = salad.rope(x, grid=(1, 1), split=(64, 0, 0))
    bad = ~torch.isfinite(y[0, 0])
    assert bad.nonzero().tolist() == [[1, 10], [1, 11], [2, 20], [2, 21]]


@needs_gpu
def test_rope_refusals_on_the_device():
    q = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16, device="cuda")
    for bad in (dict(), dict(grid=(2, 2), positions=torch.zeros(4, 3, dtype=torch.int32, device="cuda")),
                dict(positions=torch.zeros(3, 3, dtype=torch.int32, device="cuda")),
                dict(positions=torch.zeros(4, 3, dtype=torch.int64, device="cuda")),
                dict(grid=(2, 2), pairing="other"), dict(grid=(2, 2), q_out=q[:, :1])):
        with pytest.raises(ValueError):
            salad.rope(q, **bad)
    with pytest.raises(ValueError):
        salad.rope(q.transpose(2, 3).contiguous().transpose(2, 3), grid=(2, 2))
    with pytest.raises(ValueError):
        salad.rope(q.float().requires_grad_(), grid=(2, 2))
    with pytest.raises(salad.SaladError) as e:
        salad.rope(q, q, grid=(2, 2), q_out=q, k_out=q)
    assert e.value.code == INVALID


@needs_gpu
def test_rope_captured_and_on_another_stream():
    q = _draw((2, 4, 100, 128), torch.bfloat16, 12)
    want = salad.rope(q, grid=(3, 5))
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    salad.rope(q, grid=(3, 5), q_out=out, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    out.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        salad.rope(q, grid=(3, 5), q_out=out)
    new = _draw((2, 4, 100, 128), torch.bfloat16, 13)
    q.copy_(new)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, salad.rope(new, grid=(3, 5)))


def test_rope_outputs_apart_from_positions():
    for kw in (dict(positions=A + M), dict(positions=A + 3 * M + 64), dict(positions=A + M - 4)):
        assert _status(Hh=0, Wh=0, **kw) == INVALID, kw
