"""Settings of the draw given as numbers."""
import pytest
import torch


def test_top_k_as_a_number_is_an_integer_of_any_size():
    import numpy as np
    from ivf_quantizer_b200.sample import _count
    t = torch.zeros(3, dtype=torch.int32)
    assert _count(None, 50) is None and _count(t, 50) is t
    assert [_count(k, 50) for k in (0, 1, 50, 51, 1 << 40, -1, -(1 << 40), np.int64(7), 7.0, 1e30)] == \
        [0, 1, 50, 50, 50, 0, 0, 7, 7, 50]
    for bad in (2.5, "3", float("nan"), float("inf")):
        with pytest.raises(TypeError):
            _count(bad, 50)


@pytest.mark.gpu
@pytest.mark.parametrize("v", [500, 5000])
def test_large_and_fractional_top_k(v):
    import ivf_quantizer_b200 as q
    x = torch.randn(6, v, generator=torch.Generator().manual_seed(1)).cuda()
    u = torch.rand(6, dtype=torch.float64, generator=torch.Generator().manual_seed(2)).cuda()
    every = q.sample_logits(x, u)
    for k in (1 << 40, -(1 << 40), v, 0):
        got = q.sample_logits(x, u, top_k=k)
        assert torch.equal(got[0], every[0]) and torch.equal(got[1], every[1])
    with pytest.raises(TypeError):
        q.sample_logits(x, u, top_k=2.5)
