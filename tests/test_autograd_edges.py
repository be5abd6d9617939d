"""What autograd must learn of calls that it does not record: they refuse
tensors whose gradient or tangent would be lost, and what they write counts as
changed."""
import pytest
import torch
from torch.autograd import forward_ad

import sparse_linear_hybrid_top_b200 as salad

needs_gpu = pytest.mark.gpu
GRID = dict(grid=(2, 3))


@pytest.fixture
def x():
    g = torch.Generator().manual_seed(1)
    return [torch.randn(1, 2, 6, 64, generator=g).bfloat16().cuda() for _ in range(3)]


@pytest.fixture
def cache():
    return salad.BlockCache.allocate(1, 2, 64, 2)


def test_the_check_itself():
    plain, asks = torch.zeros(2), torch.zeros(2, requires_grad=True)
    salad._no_grad("f", "records nothing", plain, None)
    with pytest.raises(ValueError, match="records nothing"):
        salad._no_grad("f", "records nothing", plain, None, asks)
    with torch.no_grad():
        salad._no_grad("f", "records nothing", asks)
        with forward_ad.dual_level():
            salad._no_grad("f", "records nothing", plain)
            dual = forward_ad.make_dual(plain, torch.ones(2))
            with pytest.raises(ValueError, match="forward-mode"):
                salad._no_grad("f", "records nothing", plain, dual)
            salad._no_grad("f", "records nothing", forward_ad.unpack_dual(dual).primal)
    at = plain._version
    salad._written(plain)
    assert plain._version > at


@needs_gpu
def test_tangents_are_refused(x, cache):
    q, k, v = x
    seq = salad.cache_append(cache, k, v, cache.new_seq())
    with torch.no_grad(), forward_ad.dual_level():
        dual = forward_ad.make_dual(q, torch.ones_like(q))
        for call in (lambda: salad.rope(dual, **GRID), lambda: salad.rope(q, dual, **GRID), lambda: salad.rope_backward(dual, **GRID),
                     lambda: salad.cache_append(cache, dual, v, seq), lambda: salad.cache_append(cache, k, dual, seq),
                     lambda: salad.cache_attn(cache, dual, seq), lambda: salad.cache_attn(cache, q, seq, o=dual)):
            with pytest.raises(ValueError, match="forward-mode"):
                call()
        assert torch.equal(salad.cache_attn(cache, forward_ad.unpack_dual(dual).primal, seq), salad.cache_attn(cache, q, seq))


@needs_gpu
def test_outputs_that_ask_for_a_gradient_are_refused(x, cache):
    q, k, v = x
    seq = salad.cache_append(cache, k, v, cache.new_seq())
    leaf = torch.zeros_like(q).requires_grad_()
    for call in (lambda: salad.rope(q, q_out=leaf, **GRID), lambda: salad.rope(q, k, k_out=leaf, **GRID),
                 lambda: salad.cache_attn(cache, q, seq, o=leaf),
                 lambda: salad.cache_attn(cache, q, seq, lse=torch.zeros(1, 2, 6, device="cuda", requires_grad=True))):
        with pytest.raises(ValueError):
            call()
        assert not leaf.any()


@needs_gpu
def test_what_is_written_counts_as_changed(x, cache):
    """A tensor that another operator saved for its backward pass."""
    q, k, v = x
    w = torch.ones(64, device="cuda", dtype=torch.bfloat16, requires_grad=True)

    def spoils(t, call):
        kept = (w * t).sum()             # saves t
        call()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            kept.backward()

    spoils(q, lambda: salad.rope(q, q_out=q, **GRID))
    o = torch.zeros_like(q)
    spoils(o, lambda: salad.rope(k, q, k_out=o, **GRID))
    spoils(cache.k_tail, lambda: salad.cache_append(cache, k, v, cache.new_seq()))
    seq = salad.cache_append(cache, k, v, cache.new_seq())
    spoils(o, lambda: salad.cache_attn(cache, q, seq, o=o))
    versions = [t._version for t in (q, k, v, cache.page_table)]
    salad.cache_attn(cache, q, seq)
    salad.cache_append(cache, k, v, seq)
    salad.rope(q, k, **GRID)
    assert versions == [t._version for t in (q, k, v, cache.page_table)]    # inputs are not
    lse, state = torch.zeros(1, 2, 6, device="cuda"), seq.clone()
    before = lse._version, state._version
    salad.cache_attn(cache, q, seq, lse=lse)
    salad.cache_append(cache, k, v, state, seq_out=state)
    assert lse._version > before[0] and state._version > before[1]
    salad.check_error()
