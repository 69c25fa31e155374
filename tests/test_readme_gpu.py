"""README's example of the codes and the draws, run as it stands."""
import os
import re

import pytest
import torch

pytestmark = pytest.mark.gpu

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_codes_and_draws(dtype):
    import ivf_quantizer_b200 as q
    code = [c for c in re.findall(r"```python\n(.*?)```", open(README).read(), re.S) if "q.MX4(X)" in c]
    assert len(code) == 1
    g = torch.Generator().manual_seed(1)
    X = (torch.randn(5000, 100, generator=g) * (1 + torch.rand(5000, 1, generator=g))).to(dtype).cuda()
    Q = torch.randn(20, 100, generator=g).to(dtype).cuda()
    ns = {"torch": torch, "q": q, "X": X, "Q": Q}
    exec(code[0], ns)
    s, ids, prob, X4 = (ns[k] for k in ("s", "ids", "prob", "X4"))
    assert s.shape == (20, 5000) and s.dtype == torch.float32 and X4.shape == X.shape
    # |q - x|^2 = |q|^2 - 2 s for what the codes stand for; 102 roundings of the sum of products and
    # the bias, 101 more of the bias's own squares
    xv, qv = X4.double(), q.MX4(Q).decode().double()
    want = qv @ xv.T - 0.5 * xv.square().sum(1)
    mag = qv.abs() @ xv.abs().T + 0.5 * xv.square().sum(1)
    assert bool(((s.double() - want).abs() <= 203 * 2.0 ** -24 * mag).all())
    least = s.topk(50, 1).values[:, -1]
    assert bool((s[torch.arange(20), ids.long()] >= least).all()) and bool((prob > 0).all())
