"""min-p where the least weight it keeps is a few units of 2^-40 of the largest: the rounded weights
decide, whichever kernel a row takes."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

UNIT = 2.0 ** -40


def _logit(units, t):
    return t * math.log(units * UNIT)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("t", [1.0, 0.25, 8.0])
@pytest.mark.parametrize("min_p", [2.0 ** -42, UNIT, 1.5 * UNIT, 1e-11, 1000.25 * UNIT, 1e-6])
@pytest.mark.parametrize("v,kw", [(300, {}), (300, {"top_k": 5}), (1024, {}), (1100, {}), (3000, {}), (3000, {"top_k": 5}),
                                  (3000, {"top_k": 2000}), (3000, {"top_p": 0.9999999}), (50000, {}),
                                  (50000, {"top_k": 5}), (50000, {"top_k": 30000})])
def test_the_least_weight_of_min_p(v, kw, min_p, t, dtype):
    """Logits of a tenth of a unit above and below what rounds to the least weight (in bf16, the next
    ones whose distance from it is at least that): the one above is kept, and drawn by the largest
    uniform, the one behind it is not."""
    import ivf_quantizer_b200 as q
    least = math.ceil(float(torch.tensor(min_p, dtype=torch.float32)) / UNIT)
    assert least >= 1

    def near(units, step):
        x = torch.tensor(_logit(units, t), dtype=torch.float32).to(dtype).item()
        eps = torch.finfo(dtype).eps * abs(x)
        while (math.exp(x / t) / UNIT - units) * step < 0:
            x += step * eps
            x = torch.tensor(x, dtype=torch.float32).to(dtype).item()
        return x

    above, below = near(least - 0.4, 1), near(least - 0.6, -1)
    if least > 10000:                  # fp32 logits do not resolve a tenth of a unit there
        above, below = near(least * (1 + 1e-4), 1), near(least * (1 - 1e-4), -1)
    assert round(math.exp(above / t) / UNIT) >= least > round(math.exp(below / t) / UNIT)
    x = torch.full((2, v), -float("inf"))
    x[:, 7] = 0.0
    x[0, v - 2], x[:, v - 1] = above, below
    x = x.to(dtype).cuda()
    u = torch.full((2,), 1 - 2.0 ** -53, dtype=torch.float64).cuda()
    if "top_p" in kw and least * UNIT < 1e-6:
        kw = {"top_p": 1.0}            # (a lower one would cut the token before min-p does)
    # alone, and beside more tokens of the largest weight than one CTA ends a row for (their whole
    # weight is below 2^53 units, so the uniform's target is the last unit)
    for ones in (1, min(v // 2, 4000)):
        if ones > 1 and (kw.get("top_k", v) < ones + 2 or kw.get("top_p", 1.0) < 1):
            continue
        x[:, 7:7 + ones] = 0.0
        ids, prob = q.sample_logits(x, u, temperature=t, min_p=min_p, **kw)
        assert ids.tolist() == [v - 2, ones + 6]
        total = ones + round(math.exp(above / t) / UNIT) * UNIT
        want = torch.tensor([math.exp(above / t) / total, 1 / ones])
        assert torch.allclose(prob.cpu(), want, rtol=2.0 ** -23, atol=0)
