"""Draws from truncated softmaxes on the GPU against the fp64 oracle: ids equal, probabilities
within one fp32 rounding plus the error of a sum of V weights rounded to 2^-41 of the largest.
The inputs' margins (how near a draw is to another decision) are checked to be far above it."""
import numpy as np
import pytest
import torch

from oracle import sample_oracle as S

pytestmark = pytest.mark.gpu


def _np(t):
    return None if t is None else t.detach().cpu().double().numpy()


def _run(x, u, **kw):
    import ivf_quantizer_b200 as q
    return q.sample_logits(x, u, **kw)


def _check(x, u, t=None, k=None, p=None, m=None, got=None):
    ids, prob = got or _run(x, u, temperature=t, top_k=k, top_p=p, min_p=m)
    num = lambda v: _np(v) if isinstance(v, torch.Tensor) else v
    want, wprob, margin = S.rows(_np(x.float()), _np(u), num(t), num(k), num(p), num(m))
    v = x.shape[1]
    assert margin.min() > v * 2.0 ** -40        # both sums of a comparison
    np.testing.assert_array_equal(ids.cpu().numpy(), want)
    np.testing.assert_allclose(prob.cpu().numpy(), wprob, rtol=2.0 ** -24 + v * 2.0 ** -40, atol=0)


def _params(rows, v, seed):
    g = torch.Generator().manual_seed(seed)
    t = torch.rand(rows, generator=g) * 1.5 + 0.2
    t[::7] = 0
    k = torch.randint(0, min(v, 100) + 1, (rows,), generator=g, dtype=torch.int32)
    p = 1 - torch.rand(rows, generator=g) * 0.7
    p[::5] = 1
    m = torch.rand(rows, generator=g) * 0.2
    u = torch.rand(rows, generator=g, dtype=torch.float64)
    return [a.cuda() for a in (t, k, p, m, u)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,v", [(1, 1), (3, 2), (5, 31), (40, 1000), (17, 1024), (9, 4099),
                                    (6, 16384), (4, 50021), (2, 131072), (3, 262147)])
@pytest.mark.parametrize("use", ["", "k", "p", "m", "kp", "pm", "kpm"])
def test_draws_match_the_oracle(rows, v, dtype, use):
    g = torch.Generator().manual_seed(rows * 31 + v)
    x = (torch.randn(rows, v, generator=g) * 3).to(dtype)
    x[torch.rand(rows, v, generator=g) < 0.1] = -float("inf")
    x[:, v // 2] = 1.0
    t, k, p, m, u = _params(rows, v, v + len(use))
    _check(x.cuda(), u, t, k if "k" in use else None, p if "p" in use else None,
           m if "m" in use else None)


@pytest.mark.parametrize("spread", [0.0, 1e-3, 0.1, 30.0, 1e4])
def test_flat_and_peaked_rows(spread):
    g = torch.Generator().manual_seed(5)
    x = torch.randn(12, 5000, generator=g) * spread
    t, k, p, m, u = _params(12, 5000, 6)
    u = (torch.floor(u * 4096) + 0.5) / 4096 + 1e-7      # off every multiple of 1 / 5000
    for kw in ({}, {"p": p}, {"k": k}, {"k": k, "p": p}, {"k": torch.full_like(k, 4000), "p": p, "m": m}):
        if spread == 0.0 and "p" in kw:
            kw["p"] = torch.round(p * 512) / 512 + 1e-3 * (p < 1)
            kw["p"] = kw["p"].clamp(max=1.0)
        _check(x.cuda(), u, t, **kw)


def test_ties_at_the_border_go_to_the_lower_indices():
    x = torch.zeros(1, 3000)
    x[0, 1000:1010] = 1.0
    x = x.cuda()
    u = torch.tensor([1 - 2.0 ** -53], dtype=torch.float64, device="cuda")
    for k, want in ((1, 1000), (5, 1004), (10, 1009), (11, 1009), (12, 1009)):
        assert _run(x, u, top_k=k)[0].item() == want
    y = torch.zeros(1, 3000, device="cuda")
    for k in (1, 2, 32, 33, 1023, 1024, 1025, 2999):
        assert _run(y, u, top_k=k)[0].item() == k - 1
    # equal weights: the prefix that reaches half of them is the lower half, exactly
    assert _run(y, u, top_p=0.5)[0].item() == 1499
    ids, prob = _run(y, u)
    assert ids.item() == 2999 and abs(prob.item() * 3000 - 1) < 1e-6
    z = torch.tensor([[0.0, -0.0, 0.0, -1.0]], device="cuda")
    assert _run(z, u, top_k=2)[0].item() == 1 and _run(z, u, temperature=0)[0].item() == 0


def test_masks_lowest_values_infinities_and_nans():
    inf, low = float("inf"), torch.finfo(torch.float32).min
    x = torch.full((9, 700), -inf)
    x[1, 699] = -5.0
    x[2, :] = low
    x[3, :] = low
    x[3, 300] = 0.0
    x[4, 5] = inf
    x[4, 600] = inf
    x[5] = 0.0
    x[5, 699] = float("nan")
    x[6, 100:110] = -1e30
    x[7, 0] = 3.4e38
    x[7, 1] = low
    x[8, 350] = low
    u = torch.full((9,), 0.70041, dtype=torch.float64)
    for kw in ({}, {"k": 3}, {"p": 0.9}, {"m": 0.5}, {"k": 600, "p": 0.99, "m": 0.01}, {"t": 1e-30},
               {"t": 1e30}, {"t": 0.0}):
        kw = {a: (torch.full((9,), b, dtype=torch.int32 if a == "k" else torch.float32).cuda())
              for a, b in kw.items()}
        _check(x.cuda(), u.cuda(), **kw)
    ids, prob = _run(x.cuda(), u.cuda())
    assert ids[0].item() == -1 and prob[0].item() == 0
    assert ids[5].item() == -1 and torch.isnan(prob[5])


def test_parameters_outside_their_range_refuse_their_row_alone():
    x = torch.randn(12, 200, generator=torch.Generator().manual_seed(1)).cuda()
    nan, inf = float("nan"), float("inf")
    t = torch.tensor([1, -1, nan, inf, 1, 1, 1, 1, 1, 1, 1, 1.0]).cuda()
    p = torch.tensor([1, 1, 1, 1, 0, -1, 1.5, nan, 1, 1, 1, .5]).cuda()
    m = torch.tensor([0, 0, 0, 0, 0, 0, 0, 0, -.1, 1.1, nan, 0]).cuda()
    u = torch.full((12,), 0.4, dtype=torch.float64).cuda()
    ids, prob = _run(x, u, temperature=t, top_p=p, min_p=m)
    ok = torch.tensor([True] + [False] * 10 + [True])
    assert ((ids.cpu() >= 0) == ok).all() and (torch.isnan(prob.cpu()) == ~ok).all()
    for bad in (1.0, -0.1, nan, 2.0):
        assert _run(x[:1], torch.tensor([bad], dtype=torch.float64).cuda())[0].item() == -1


def test_extreme_uniforms_and_counts():
    x = torch.randn(4, 3001, generator=torch.Generator().manual_seed(2)).cuda()
    x[1, -1] = -float("inf")
    for uv in (0.0, 1 - 2.0 ** -53):
        u = torch.full((4,), uv, dtype=torch.float64).cuda()
        for kw in ({}, {"top_k": 1}, {"top_k": 5000}, {"top_k": -3}, {"top_p": 1e-6}, {"min_p": 1.0}):
            ids, prob = _run(x, u, **kw)
            assert ((ids >= 0) & (ids < 3001)).all() and (prob > 0).all()
            if "top_k" not in kw or kw["top_k"] != 1:
                if not kw or kw.get("top_k", 0) in (5000, -3):
                    first = 0 if uv == 0 else 3000
                    assert ids[0].item() == first and ids[1].item() == (0 if uv == 0 else 2999)
                else:
                    assert torch.equal(ids.long(), x.argmax(1))


def test_strides_and_rows_beyond_32_bit_offsets():
    big = torch.randn(30, 900, generator=torch.Generator().manual_seed(3)).cuda()
    t, k, p, m, u = _params(30, 900, 4)
    for x in (big[:, 1:778], big[::2, 3:], big.to(torch.bfloat16)[:, 5:]):
        n = x.shape[0]
        _check(x, u[:n], t[:n], k[:n], p[:n], m[:n])
    flat = torch.zeros((1 << 31) + 4000, dtype=torch.bfloat16, device="cuda")
    far = flat.as_strided((2, 2000), ((1 << 31) + 1000, 1))
    far.copy_(big[:2].to(torch.bfloat16).repeat(1, 3)[:, :2000])
    _check(far, u[:2], t[:2] + 0.1, k[:2], p[:2], m[:2])


def test_numbers_in_place_of_tensors_and_refusals():
    x = torch.randn(6, 500, generator=torch.Generator().manual_seed(7)).cuda()
    u = torch.rand(6, dtype=torch.float64, generator=torch.Generator().manual_seed(8)).cuda()
    full = lambda v, d: torch.full((6,), v, dtype=d, device="cuda")
    a = _run(x, u, temperature=0.7, top_k=20, top_p=0.8, min_p=0.05)
    b = _run(x, u, temperature=full(0.7, torch.float32), top_k=full(20, torch.int32),
             top_p=full(0.8, torch.float32), min_p=full(0.05, torch.float32))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    for kw in ({"top_k": full(3, torch.int64)}, {"temperature": full(1, torch.float64)},
               {"top_p": torch.ones(5, device="cuda")}, {"min_p": torch.zeros(6)}):
        with pytest.raises(ValueError):
            _run(x, u, **kw)
    with pytest.raises(ValueError):
        _run(x, u.float())
    with pytest.raises(ValueError):
        _run(x, None)
    with pytest.raises(TypeError):
        _run(x.half(), u)
    assert _run(x[:0], u[:0])[0].shape == (0,)
    big = torch.empty(1, (1 << 22) + 1, device="cuda")
    from ivf_quantizer_b200 import FgmmError
    with pytest.raises(FgmmError):
        _run(big, u[:1])


def test_largest_row():
    v = 1 << 22
    g = torch.Generator().manual_seed(9)
    x = (torch.randn(2, v, generator=g) * 2).cuda()
    t, k, p, m, u = _params(2, v, 10)
    t = t.clamp(min=0.5)
    _check(x, u, t, None, p.clamp(max=0.9))
    _check(x, u, t, torch.full_like(k, 1 << 20), None)
    _check(x, u, t)


def test_repeatable_on_another_stream_and_captured():
    import ivf_quantizer_b200 as q
    x = torch.randn(50, 20000, generator=torch.Generator().manual_seed(11)).cuda() * 2
    t, k, p, m, u = _params(50, 20000, 12)
    kw = dict(temperature=t, top_k=k, top_p=p, min_p=m)
    want = _run(x, u, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [_run(x, u, **kw) for _ in range(5)]
    main = [_run(x, u, **kw) for _ in range(5)]
    torch.cuda.synchronize()
    for a in got + main:
        assert torch.equal(a[0], want[0]) and torch.equal(a[1], want[1])
    graph = torch.cuda.CUDAGraph()
    xs = x.clone()
    with torch.cuda.graph(graph):
        out = q.sample_logits(xs, u, **kw)
    xs.copy_(x.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    _check(xs, u, t, k, p, m, got=out)


def test_queries_scored_on_codes_and_drawn():
    """The run of all operators: vectors kept as codes, queries scored against them, one vector
    drawn per query; beside the soft assignment of the same points."""
    import synth
    import ivf_quantizer_b200 as q
    from oracle import mx4_oracle as M
    X = synth.generate("table1", 4000, seed=21)
    w, mu, var = synth.init_params(X, 64, seed=21)
    index = q.MX4(torch.as_tensor(mu, dtype=torch.float32).cuda())
    points = X[:500].cuda()
    sq = (index.decode() ** 2).sum(1) * -0.5
    logits = index.scores(points, bias=sq)                 # log responsibilities of unit variances
    u = torch.rand(500, dtype=torch.float64, generator=torch.Generator().manual_seed(1)).cuda()
    ids, prob = q.sample_logits(logits, u, temperature=2.0, top_k=8, top_p=0.95, min_p=0.01)
    torch.cuda.synchronize()
    qv = M.decode(*M.encode(points.cpu().numpy()), 128)
    xv = M.decode(*M.encode(np.asarray(mu, dtype=np.float32)), 128)
    want, mag = M.scores(qv, xv, 1.0, sq.cpu().double().numpy())
    assert (np.abs(logits.cpu().numpy() - want) <= 130 * 2.0 ** -24 * mag).all()
    _check(logits, u, torch.full((500,), 2.0).cuda(), torch.full((500,), 8, dtype=torch.int32).cuda(),
           torch.full((500,), 0.95).cuda(), torch.full((500,), 0.01).cuda(), got=(ids, prob))
    g = q.GMM(64, 128)
    wd, md, vd = g.new_params(w, index.decode().cpu(), np.ones((64, 128), dtype=np.float32))
    hard, _ = g.soft_assign(points, wd, md, vd, top_m=1, r_threshold=0.5)
    greedy, _ = q.sample_logits(logits, u, temperature=0)
    torch.cuda.synchronize()
    g.close()
    # the points' own rounding to 4 bits moves some of them to a neighbour, not most
    assert (hard[:, 0] == greedy).float().mean().item() > 0.5


def test_draws_at_random_shapes_and_settings():
    rng = np.random.default_rng(23)
    for i in range(60):
        rows, v = int(rng.integers(1, 6)), int(np.exp(rng.uniform(0, np.log(70000))))
        g = torch.Generator().manual_seed(1000 + i)
        x = torch.randn(rows, v, generator=g) * float(rng.choice([0.05, 1.0, 3.0, 20.0]))
        x[torch.rand(rows, v, generator=g) < float(rng.choice([0.0, 0.5]))] = -float("inf")
        if i % 4 == 0:
            x = torch.round(x * 2) / 2                   # many ties
        x[:, int(rng.integers(0, v))] = 2.0
        t, k, p, m, u = _params(rows, v, 2000 + i)
        if i % 3 == 0:
            k = torch.randint(0, v + 1, (rows,), generator=g, dtype=torch.int32).cuda()
        use = int(rng.integers(0, 8))
        dt = (torch.float32, torch.bfloat16)[i % 2]
        _check(x.to(dt).cuda(), u, t, k if use & 1 else None, p if use & 2 else None, m if use & 4 else None)
