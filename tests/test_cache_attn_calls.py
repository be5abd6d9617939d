"""Calls of the attention over the 8-bit block cache that a program makes beside
plain ones: pages given back behind a window."""
import pytest
import torch

import sparse_linear_hybrid_top_b200 as salad
from tests.test_cache_attn import _make, _q

needs_gpu = pytest.mark.gpu


@needs_gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,Hq", [(1, 2), (40, 2), (70, 2), (200, 4), (300, 2)])
@pytest.mark.parametrize("frame", [0, 1, 7])
def test_pages_before_the_window_may_be_given_back(d, N, Hq, frame):
    """Blocks that no row sees are not read: their table entries may be no page
    (no error is reported), or name memory that holds anything."""
    L = 1000
    for lo in (63, 64, 200, 256, 290):                     # the first key that is seen, nearly
        window = L - N - lo
        cache, seq = _make(1, 2, d, [L], seed=lo)
        q = _q(1, Hq, N, d, lo)
        want = salad.cache_attn(cache, q, seq, frame=frame, window=window)
        salad.check_error()
        first = (L - N) // frame * frame - window if frame else lo
        gone = cache.page_table[0, :max(0, first) // 64].long()
        cache.k_pages.view(torch.uint8)[gone] = 127        # NaN codes, scales as they were
        cache.v_pages.view(torch.uint8)[gone] = 127
        assert torch.equal(salad.cache_attn(cache, q, seq, frame=frame, window=window), want)
        cache.page_table[0, :len(gone)] = -1
        assert torch.equal(salad.cache_attn(cache, q, seq, frame=frame, window=window), want)
        salad.check_error()
