"""Scores where every CTA takes several tiles: accumulators, swizzled tiles and query tiles used
again, the walk over tiles, the bias read ahead, ragged ends after whole tiles.  Against the fp64
product of the decoded rows (decoding is compared bit by bit in test_mx4_gpu.py), within the
summation bound (D + 2) 2^-24 sum |q x| of any order of fp32 sums plus the output's rounding."""
import pytest
import torch

pytestmark = pytest.mark.gpu

SMS = 148

# m, n, d, tiles a step, query tile, CTAs an SM (a pair counts half): what the dispatch gives each kernel
SHAPES = {
    # bulk copies, rows of up to 128 dimensions
    "copies64_q16": (1, 250003, 96, 2, 16, 2), "copies64_q32": (20, 250003, 96, 2, 32, 2),
    "copies64_q64": (50, 120001, 120, 1, 64, 2), "copies64_q128": (300, 60001, 96, 1, 128, 1),
    "copies64_query_tiles": (600, 20001, 33, 1, 128, 1), "copies64_one_tile_of_vectors": (60001, 100, 96, 1, 128, 1),
    # bulk copies, rows of up to 256
    "copies128_q16": (3, 150001, 200, 1, 16, 2), "copies128_q32": (20, 150001, 230, 1, 32, 2),
    "copies128_q64": (64, 60001, 200, 1, 64, 1), "copies128_q128": (1000, 30011, 200, 1, 128, 1),
    "copies128_whole_rows": (70, 60001, 256, 1, 128, 1),
    # boxes
    "boxes64_q16": (1, 250003, 128, 1, 16, 4), "boxes128_whole_rows": (40, 60001, 256, 1, 64, 1),
    "boxes128_q16": (5, 150001, 288, 1, 16, 2), "boxes128_q32": (20, 150001, 600, 1, 32, 2),
    "boxes128_q64": (50, 60001, 288, 1, 64, 1), "boxes128_q128": (100, 150001, 288, 1, 128, 1),
    "boxes128_one_tile_of_vectors": (60001, 100, 288, 1, 128, 1),
    # pairs of CTAs, tiles of 256 x 256
    "pairs": (700, 30011, 300, 2, 256, 0.5), "pairs_long_rows": (300, 30011, 1100, 2, 256, 0.5),
}


@pytest.mark.parametrize("name", SHAPES)
def test_scores_of_many_tiles_a_cta(name):
    import ivf_quantizer_b200 as q
    m, n, d, sub, nt, ctas = SHAPES[name]
    assert -(-n // (128 * sub)) * -(-m // nt) > 2 * SMS * ctas      # a third tile somewhere
    g = torch.Generator().manual_seed(m + n + d)
    spread = torch.exp(torch.rand(d, generator=g) * 6 - 3)
    x = q.MX4((torch.randn(n, d, generator=g) * spread).cuda())
    qs = q.MX4((torch.randn(m, d, generator=g) * spread).cuda())
    bias = torch.randn(n, generator=g).cuda() * 5
    xv, qv = x.decode().double(), qs.decode().double()
    plain = 0.25 * (qv @ xv.T)
    mag = 0.25 * (qv.abs() @ xv.abs().T)
    for out in (torch.float32, torch.bfloat16):
        for b in (None, bias):
            got = x.scores(qs, alpha=0.25, bias=b, dtype=out)
            assert got.shape == (m, n) and got.dtype == out
            want = plain if b is None else plain + b.double()
            tol = (max(d, 32) + 2) * 2.0 ** -24 * (mag if b is None else mag + b.double().abs())
            if out == torch.bfloat16:
                tol = tol + 2.0 ** -8 * (want.abs() + tol)
            over = (got.double() - want).abs() - tol
            assert bool((over <= 0).all()), over.max().item()
            for _ in range(2):                                       # and again: the same bits
                assert torch.equal(x.scores(qs, alpha=0.25, bias=b, dtype=out), got)
    assert x.status() == 0
