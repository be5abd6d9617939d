"""A BlockCache's attributes stay those whose addresses its calls use.  (On the
CPU the buffers are host tensors; nothing is launched on them.)"""
import copy
import io

import pytest
import torch

import sparse_linear_hybrid_top_b200 as salad

BUFFERS = ("k_pages", "v_pages", "k_scale", "v_scale", "k_tail", "v_tail", "page_table")


@pytest.fixture
def cache(monkeypatch):
    if not torch.cuda.is_available():
        monkeypatch.setattr(salad, "_dev_tensor", lambda t, dtype, name: None)
        return salad.BlockCache.allocate(2, 3, 64, 4, device="cpu")
    return salad.BlockCache.allocate(2, 3, 64, 4)


def _addresses(c):
    return c.args[:7] == tuple(getattr(c, n).data_ptr() for n in BUFFERS)


def test_attributes_cannot_be_assigned(cache):
    assert _addresses(cache)
    for name in BUFFERS + ("B", "H", "d", "pages", "blocks", "args", "index"):
        before = getattr(cache, name)
        with pytest.raises(AttributeError, match="another BlockCache"):
            setattr(cache, name, before)
        with pytest.raises(AttributeError):
            delattr(cache, name)
        assert getattr(cache, name) is before
    wider = torch.zeros(2, 9, dtype=torch.int32, device=cache.device)
    with pytest.raises(AttributeError):
        cache.page_table = wider
    grown = salad.BlockCache(*(getattr(cache, n) for n in BUFFERS[:-1]), wider)
    assert _addresses(grown) and grown.blocks == 9 and grown.args[:6] == cache.args[:6]


def _saved(cache):
    file = io.BytesIO()
    torch.save(cache, file)
    file.seek(0)
    return torch.load(file, weights_only=False)


@pytest.mark.parametrize("how", [copy.deepcopy, _saved])
def test_copies_use_their_own_buffers(cache, how):
    twin = how(cache)
    assert _addresses(twin) and _addresses(cache)
    assert not set(twin.args[:7]) & set(cache.args[:7]) and twin.args[7:] == cache.args[7:]


def test_a_shallow_copy_shares_them(cache):
    assert copy.copy(cache).args == cache.args


def test_other_attributes_are_the_programs(cache):
    """A default scale of the scores, and whatever a program notes on a cache."""
    cache.softmax_scale, cache.owner = 0.5, "layer 3"
    for twin in (copy.copy(cache), copy.deepcopy(cache), _saved(cache)):
        assert twin.softmax_scale == 0.5 and twin.owner == "layer 3" and _addresses(twin)
    del cache.owner
    assert not hasattr(cache, "owner")


@pytest.mark.gpu
def test_calls_on_a_copy_leave_the_cache_alone():
    g = torch.Generator().manual_seed(1)
    k, v, q = (torch.randn(1, 2, 100, 64, generator=g).bfloat16().cuda() for _ in range(3))
    cache = salad.BlockCache.allocate(1, 2, 64, 4)
    seq = salad.cache_append(cache, k, v, cache.new_seq())
    twin = copy.deepcopy(cache)
    want = salad.cache_attn(cache, q, seq)
    after = salad.cache_append(twin, v, k, seq)
    assert torch.equal(salad.cache_attn(cache, q, seq), want)
    assert not torch.equal(salad.cache_attn(twin, q, after), want)
    salad.check_error()
