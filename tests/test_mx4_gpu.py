"""4-bit codes on the GPU against the fp64 oracle: codes and scales bit-exact, decoded values
exact, scores within the summation bound D 2^-24 sum |q x| (any order of fp32 sums; products of
two codes are exact) plus one rounding of the output."""
import numpy as np
import pytest
import torch

from oracle import mx4_oracle as M

pytestmark = pytest.mark.gpu


def _x(n, d, seed, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, d, generator=g) * torch.exp(torch.rand(d, generator=g) * 6 - 3)
    return x.to(dtype)


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _same_codes(m, x):
    c, s = M.encode(_np(x))
    np.testing.assert_array_equal(m.codes.cpu().numpy(), M.pack(c))
    np.testing.assert_array_equal(m.scales.cpu().numpy(), M.tile_scales(s))
    return M.decode(c, s, x.shape[1])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,d", [(1, 1), (1, 128), (5, 31), (127, 32), (128, 33), (129, 100),
                                 (300, 128), (257, 129), (33, 960), (7, 4097)])
def test_encode_and_decode_match_the_oracle(n, d, dtype):
    import ivf_quantizer_b200 as q
    x = _x(n, d, n * 7 + d, dtype).cuda()
    x[n // 2] = 0
    m = q.MX4(x)
    want = _same_codes(m, x)
    for out in (torch.float32, torch.bfloat16):
        got = m.decode(out)
        assert got.shape == (n, d) and got.dtype == out
        np.testing.assert_array_equal(_np(got), want)


def test_every_rounding_case_at_many_scales():
    """All grid values, the points halfway between them and their fp32 neighbours, with the
    block's largest value fixed, at exponents from the smallest to the largest."""
    import ivf_quantizer_b200 as q
    mid = (M.GRID[1:] + M.GRID[:-1]) / 2
    base = np.concatenate([M.GRID, mid, [6.5, 7.0, 7.9]]).astype(np.float32)
    base = np.concatenate([base, np.nextafter(base, np.float32(9)), np.nextafter(base, np.float32(-9))])
    base = np.concatenate([base, -base])
    base = base[np.abs(base) < 8]
    rows = []
    for e in (-149, -140, -127, -126, -125, -124, -60, -3, 0, 1, 30, 100, 124, 125):
        for lead in (4.0, 6.0, 7.5):
            for i in range(0, len(base), 31):
                v = np.zeros(32)
                v[0] = lead
                part = base[i:i + 31]
                v[1:1 + len(part)] = np.where(np.abs(part) <= lead, part, 0)
                rows.append(np.ldexp(v, e))
    x = torch.from_numpy(np.array(rows).astype(np.float32)).cuda()
    x = torch.where(torch.isfinite(x), x, torch.zeros_like(x))
    m = q.MX4(x)
    want = _same_codes(m, x)
    np.testing.assert_array_equal(m.decode().cpu().numpy().astype(np.float64), want)


def test_non_finite_blocks_decode_to_nan_and_leave_the_others():
    import ivf_quantizer_b200 as q
    x = _x(6, 100, 3).cuda()
    x[0, 0], x[1, 99], x[2, 40], x[3, 40] = float("nan"), float("inf"), -float("inf"), 3.4e38
    m = q.MX4(x)
    want = _same_codes(m, x)
    got = m.decode().cpu().numpy()
    np.testing.assert_array_equal(got, want.astype(np.float32))
    assert np.isnan(got[0, :32]).all() and np.isnan(got[1, 96:]).all() and np.isnan(got[2, 32:64]).all()
    s = m.scores(_x(2, 100, 4).cuda()).cpu().numpy()
    # row 3 holds 6 * 2^125: its product with a query value of 2 or more is beyond fp32
    assert np.isnan(s[:, :3]).all() and not np.isnan(s[:, 3]).any() and np.isfinite(s[:, 4:]).all()


def test_strides_and_odd_alignment():
    import ivf_quantizer_b200 as q
    big = _x(200, 300, 5).cuda()
    for x in (big[:, 3:103], big[::2, 1:130], big[50:, :96], big.to(torch.bfloat16)[:, 1:98]):
        m = q.MX4(x)
        _same_codes(m, x)
    with pytest.raises(ValueError):
        q.MX4(big.T)
    with pytest.raises(TypeError):
        q.MX4(big.half())
    # decode into rows of a larger buffer leaves the columns beside them as they were
    from ivf_quantizer_b200 import _lib
    m = q.MX4(big[:, :100])
    out = torch.full((200, 131), 7.0, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    assert _lib.LIB.fgmm_mx4_decode(m.codes.data_ptr(), m.scales.data_ptr(), 200, 100,
                                    out.data_ptr(), _lib.F32, 131, stream) == _lib.OK
    assert (out[:, 100:] == 7).all() and torch.equal(out[:, :100], m.decode())


def _check_scores(got, q, x, alpha, bias, d):
    qv, xv = (M.decode(*M.encode(_np(t)), d) for t in (q, x))
    want, mag = M.scores(qv, xv, alpha, None if bias is None else _np(bias))
    # summation of d terms, then alpha, bias and the output's own rounding
    tol = (max(d, 32) + 2) * 2.0 ** -24 * mag
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    err = np.abs(_np(got) - want)
    assert (err <= tol).all(), (err - tol).max()


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m,n,d", [(1, 1, 1), (1, 1000, 128), (3, 129, 100), (8, 257, 96), (16, 64, 33),
                                   (17, 300, 960), (33, 128, 256), (64, 500, 160), (65, 129, 129),
                                   (128, 640, 128), (129, 1000, 64), (200, 1, 320), (300, 777, 513),
                                   (5, 20000, 40), (700, 1500, 1056), (260, 400, 4128), (100, 200, 600),
                                   (300, 100, 600), (2, 500, 128), (70, 300, 256), (64, 300, 256), (600, 300, 288)])
def test_scores_match_the_oracle(m, n, d, out):
    import ivf_quantizer_b200 as q
    qs, x = _x(m, d, m + d).cuda(), _x(n, d, n + 1).cuda()
    bias = torch.linspace(-3, 5, n, device="cuda") if (m + n) % 2 else None
    index = q.MX4(x)
    got = index.scores(qs, alpha=0.25, bias=bias, dtype=out)
    assert got.shape == (m, n) and got.dtype == out
    _check_scores(got, qs, x, 0.25, bias, d)
    # queries encoded by the caller, and a second call: the same bits
    assert torch.equal(index.scores(q.MX4(qs), alpha=0.25, bias=bias, dtype=out), got)


def test_scores_bf16_queries_and_strided_output():
    import ivf_quantizer_b200 as q
    from ivf_quantizer_b200 import _lib
    qs, x = _x(40, 200, 9, torch.bfloat16).cuda(), _x(333, 200, 10).cuda()
    index, enc = q.MX4(x), q.MX4(qs)
    _check_scores(index.scores(qs), qs, x, 1.0, None, 200)
    for dt, code in ((torch.float32, _lib.F32), (torch.bfloat16, _lib.BF16)):
        out = torch.full((42, 339), 7.0, device="cuda", dtype=dt)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        stream = torch.cuda.current_stream().cuda_stream
        view = out[1:41, 3:336]
        assert _lib.LIB.fgmm_mx4_scores(enc.codes.data_ptr(), enc.scales.data_ptr(), 40,
                                        index.codes.data_ptr(), index.scales.data_ptr(), 333, 200, 1.0,
                                        None, view.data_ptr(), code, 339, status.data_ptr(),
                                        stream) == _lib.OK
        assert torch.equal(view, index.scores(qs, dtype=dt)) and int(status) == 0
        mask = torch.ones_like(out, dtype=torch.bool)
        mask[1:41, 3:336] = False
        assert (out[mask] == 7).all()


def test_scores_with_wide_spread_of_scales():
    import ivf_quantizer_b200 as q
    qs, x = _x(50, 256, 11).cuda(), _x(260, 256, 12).cuda()
    qs[:, :64] *= 2.0 ** 40
    x[:, :64] *= 2.0 ** -45
    x[:, 128:] *= 2.0 ** 20
    x[7] = 0
    _check_scores(q.MX4(x).scores(qs), qs, x, 1.0, None, 256)


def test_empty_batches():
    import ivf_quantizer_b200 as q
    e, x = torch.empty(0, 64, device="cuda"), _x(10, 64, 13).cuda()
    assert q.MX4(e).decode().shape == (0, 64)
    assert q.MX4(x).scores(e).shape == (0, 10) and q.MX4(e).scores(x).shape == (10, 0)


def test_binding_refusals():
    import ivf_quantizer_b200 as q
    x = _x(10, 64, 14).cuda()
    m = q.MX4(x)
    with pytest.raises(ValueError):
        m.scores(_x(3, 65, 1).cuda())
    with pytest.raises(ValueError):
        m.scores(x, bias=torch.zeros(9, device="cuda"))
    with pytest.raises(ValueError):
        m.scores(x, bias=torch.zeros(10, device="cuda", dtype=torch.float64))
    with pytest.raises(TypeError):
        m.scores(x, dtype=torch.float16)
    with pytest.raises(TypeError):
        m.decode(torch.float16)
    with pytest.raises(ValueError):
        q.MX4.from_codes(m.codes, m.scales, 65)
    with pytest.raises(ValueError):
        q.MX4.from_codes(m.codes[:, :16], m.scales, 32)
    with pytest.raises(ValueError):
        q.MX4(torch.zeros(4, 0, device="cuda"))


def test_other_stream_and_captured_graph():
    import ivf_quantizer_b200 as q
    x, qs = _x(500, 128, 15).cuda(), _x(20, 128, 16).cuda()
    index = q.MX4(x)
    want = index.scores(qs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = q.MX4(x).scores(qs)
    side.synchronize()
    assert torch.equal(got, want)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    qa, qb = qs.clone(), qs.clone()
    with torch.cuda.graph(g1):
        a = index.scores(qa)
    with torch.cuda.graph(g2):
        b = index.scores(qb, alpha=2.0)
    qa.copy_(qs * 2)
    for _ in range(3):
        g1.replay()
        g2.replay()
    torch.cuda.synchronize()
    # a power of two moves the scales alone
    assert torch.equal(a, want * 2) and torch.equal(b, want * 2)


def test_offsets_beyond_32_bits():
    """Rows whose elements, codes and scores lie beyond 2^31 elements of their buffers."""
    import ivf_quantizer_b200 as q
    n, d = (1 << 20) + 77, 2080
    tail = _x(64, d, 17, torch.bfloat16).cuda()
    x = torch.zeros(n, d, dtype=torch.bfloat16, device="cuda")
    x[-64:] = tail
    m = q.MX4(x)
    assert torch.equal(m.decode(torch.bfloat16)[-64:], q.MX4(tail).decode(torch.bfloat16))
    del x
    qs = _x(2100, d, 18).cuda()
    s = m.scores(qs, dtype=torch.bfloat16)
    ref = q.MX4(tail).scores(qs, dtype=torch.bfloat16)
    assert torch.equal(s[:, -64:], ref) and (s[-1, :1000] == 0).all()


def test_scores_at_random_shapes():
    """Every kernel and its ragged edges: few and many queries, short and long rows, any N."""
    import ivf_quantizer_b200 as q
    rng = np.random.default_rng(19)
    for i in range(60):
        m = int(np.exp(rng.uniform(0, np.log(600))))
        n = int(np.exp(rng.uniform(0, np.log(4000))))
        d = int(np.exp(rng.uniform(0, np.log(1500))))
        dt = (torch.float32, torch.bfloat16)[i % 2]
        qs, x = _x(m, d, i, dt).cuda(), _x(n, d, i + 100).cuda()
        bias = torch.randn(n, device="cuda") if i % 3 == 0 else None
        got = q.MX4(x).scores(qs, alpha=-0.5, bias=bias, dtype=(torch.float32, torch.bfloat16)[i // 2 % 2])
        _check_scores(got, qs, x, -0.5, bias, d)


def test_scores_of_very_small_values_lose_at_most_the_smallest_normal():
    import ivf_quantizer_b200 as q
    qs, x = _x(20, 300, 20).cuda() * 2.0 ** -70, _x(200, 300, 21).cuda() * 2.0 ** -58
    got = _np(q.MX4(x).scores(qs))
    qv, xv = (M.decode(*M.encode(_np(t)), 300) for t in (qs, x))
    want, mag = M.scores(qv, xv)
    assert np.isfinite(got).all() and (np.abs(got - want) <= 302 * 2.0 ** -24 * mag + 300 * 2.0 ** -126).all()


def test_non_finite_queries_spoil_their_row_alone():
    import ivf_quantizer_b200 as q
    x, qs = _x(300, 200, 22).cuda(), _x(70, 200, 23).cuda()
    index = q.MX4(x)
    want = index.scores(qs)
    qs[5, 7], qs[69, 199] = float("nan"), float("inf")
    got = index.scores(qs)
    bad = torch.zeros(70, dtype=torch.bool)
    bad[[5, 69]] = True
    assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], want[~bad])


def test_two_streams_at_once():
    """Kernels of different tile sizes side by side: they share the SMs' tensor memory."""
    import ivf_quantizer_b200 as q
    x, y = q.MX4(_x(6000, 600, 24).cuda()), q.MX4(_x(9000, 96, 25).cuda())
    calls = [(x, _x(300, 600, 26).cuda()), (y, _x(3, 96, 27).cuda()), (x, _x(20, 600, 28).cuda()),
             (y, _x(200, 96, 29).cuda())]
    want = [a.scores(b) for a, b in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    got = [[] for _ in calls]
    for _ in range(10):
        for s, g, (a, b) in zip(streams, got, calls):
            with torch.cuda.stream(s):
                g.append(a.scores(b))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(o, w) for o in g)


def test_status_reports_and_clears_a_wait_that_gave_up():
    import ivf_quantizer_b200 as q
    from ivf_quantizer_b200 import _lib, mx4
    index = q.MX4(_x(300, 64, 50).cuda())
    index.scores(_x(3, 64, 51).cuda())
    assert index.status() == _lib.OK
    word = mx4._words[index.codes.device.index]     # the kernels' argument
    word.fill_(_lib.ERR_TIMEOUT)
    index.scores(_x(3, 64, 51).cuda())              # (a call that ends well leaves it)
    with pytest.raises(_lib.FgmmError):
        index.check_status()
    assert index.status() == _lib.OK


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [1, 130, 257])
@pytest.mark.parametrize("d", [97, 104, 112, 220, 224, 352, 448, 480, 512])
def test_encode_rows_that_fill_their_scale_tiles(d, n, dtype):
    """Rows whose blocks fill at least 7/8 of their scale tiles, and ones that just do not, at each
    alignment of the rows."""
    import ivf_quantizer_b200 as q
    wide = _x(n, 544, n + d, dtype).cuda()
    for x in (wide[:, :d].contiguous(), wide[:, :d], wide[:, 8:d + 8], wide[:, 4:d + 4], wide[:, 1:d + 1]):
        _same_codes(q.MX4(x), x)


@pytest.mark.parametrize("n,d,dtype", [(400001, 128, torch.float32), (120001, 960, torch.bfloat16),
                                       (700001, 96, torch.float32)])
def test_encode_many_rows(n, d, dtype):
    """More pieces than threads: rows encoded alone have the same codes and scales."""
    import ivf_quantizer_b200 as q
    x = _x(n, d, 60, dtype).cuda()
    m = q.MX4(x)
    nkc = -(-d // 128)
    for r in (0, 128 * 700, n // 128 * 128 - 12800, n // 128 * 128):
        part = x[r:r + 12800]
        p = q.MX4(part)
        assert torch.equal(m.codes[r:r + 12800], p.codes)
        t = r // 128 * nkc * 512
        assert torch.equal(m.scales[t:t + p.scales.numel()], p.scales)
    _same_codes(p, part)
    out = m.decode()
    s = torch.randint(0, n, (300,), generator=torch.Generator().manual_seed(61)).cuda()
    np.testing.assert_array_equal(_np(out[s]), M.decode(*M.encode(_np(x[s])), d))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,d", [(1, 3), (130, 97), (31, 100), (257, 128), (65, 530)])
def test_decode_into_rows_of_each_alignment(n, d, dtype):
    """Rows of a larger buffer at offsets and strides of 32, 16, 8 and 4 bytes and of one value; what
    lies beside them stays."""
    import ivf_quantizer_b200 as q
    from ivf_quantizer_b200 import _lib
    m = q.MX4(_x(n, d, 70 + d).cuda())
    want = m.decode(dtype)
    np.testing.assert_array_equal(_np(want), M.decode(*M.encode(_np(_x(n, d, 70 + d))), d))
    stream = torch.cuda.current_stream().cuda_stream
    code = _lib.F32 if dtype == torch.float32 else _lib.BF16
    for off, ld in ((0, 544), (16, 560), (8, 552), (4, 548), (2, 546), (1, 545), (0, 545), (1, 544)):
        out = torch.full((n + 1, ld), 7.0, device="cuda", dtype=dtype)
        assert _lib.LIB.fgmm_mx4_decode(m.codes.data_ptr(), m.scales.data_ptr(), n, d,
                                        out[:, off:].data_ptr(), code, ld, stream) == _lib.OK
        assert torch.equal(out[:n, off:off + d], want)
        out[:n, off:off + d] = 7.0
        assert (out == 7).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_encode_rows_of_each_alignment(dtype):
    import ivf_quantizer_b200 as q
    for off, ld in ((0, 544), (16, 560), (8, 552), (4, 548), (2, 546), (1, 545), (0, 545), (1, 544)):
        wide = _x(130, ld, 80 + off, dtype).cuda()
        for d in (97, 100, 160, 520):
            _same_codes(q.MX4(wide[:, off:off + d]), wide[:, off:off + d])
