"""Pins of the 4-bit code oracle (no GPU) and refusals of the C-ABI and the binding, none of
which reaches a device."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import mx4_oracle as M
from oracle import sample_oracle as S


def test_grid_values_are_fixed_points():
    v = np.concatenate([M.GRID, -M.GRID])
    for e in (-20, 0, 5):
        x = np.zeros((1, 32))
        x[0, :16] = v * 2.0 ** e
        c, s = M.encode(x)
        assert s[0, 0] == e + 127
        np.testing.assert_array_equal(M.decode(c, s, 32), x)


def test_ties_go_to_even_codes_and_large_values_saturate():
    x = np.zeros((1, 32))
    x[0, :9] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.9, -0.75]
    x[0, 9] = 4.0
    c, s = M.encode(x)
    assert s[0, 0] == 127
    np.testing.assert_array_equal(M.decode(c, s, 32)[0, :9], [0, 1, 1, 2, 2, 4, 4, 6, -1])


def test_zero_subnormal_and_non_finite_blocks():
    x = np.zeros((4, 64))
    x[1, 40] = 2.0 ** -140
    x[2, 3] = np.nan
    x[3, 63] = -np.inf
    c, s = M.encode(x)
    np.testing.assert_array_equal(s, [[0, 0], [0, 0], [255, 0], [0, 255]])
    v = M.decode(c, s, 64)
    assert np.isnan(v[2, :32]).all() and (v[2, 32:] == 0).all() and np.isnan(v[3, 32:]).all()
    assert (v[1] == 0).all()


def test_error_of_a_value_is_at_most_half_a_step():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((50, 96)) * np.exp(rng.uniform(-5, 5, 96))
    c, s = M.encode(x)
    v = M.decode(c, s, 96)
    top = np.repeat(np.abs(x.reshape(50, 3, 32)).max(2), 32, 1)
    scale = 2.0 ** (np.floor(np.log2(top)) - 2)
    # half of the largest step is 1 below 6; above it the value is cut to 6 (at most 2 away)
    assert (np.abs(v - x) <= np.where(np.abs(x) <= 6 * scale, 1.0, 2.0) * scale).all()


def test_pack_and_tiles_are_inverse():
    rng = np.random.default_rng(1)
    c = rng.integers(0, 16, (5, 64)).astype(np.uint8)
    np.testing.assert_array_equal(M.unpack(M.pack(c)), c)
    idx = M.tile_index(300, 9)
    assert len(np.unique(idx)) == idx.size and idx.max() < 3 * 3 * 512
    assert idx[33, 5] == 512 + 16 + 4 + 1 and idx[128, 0] == 3 * 512


def test_sampler_by_hand():
    x = np.log([0.1, 0.4, 0.2, 0.3])
    for u, want in ((0.0, 0), (0.0999, 0), (0.1001, 1), (0.4999, 1), (0.5001, 2), (0.7001, 3)):
        assert S.row(x, u)[0] == want
    assert S.row(x, 0.5, k=1)[:2] == (1, 1.0)
    i, pr, _ = S.row(x, 0.99, k=2)
    assert i == 3 and abs(pr - 3 / 7) < 1e-12
    assert S.row(x, 0.0, p=0.65)[0] == 1 and S.row(x, 0.99, p=0.65)[0] == 3     # 0.4 < 0.65 <= 0.7
    assert S.row(x, 0.99, p=0.39)[0] == 1                                       # the first reaches it
    assert S.row(x, 0.0, m=0.45)[0] == 1                                        # 0.1 / 0.4 is out
    assert S.row(x, 0.5, t=0)[:2] == (1, 1.0)
    assert S.row(np.zeros(4), 0.49, p=0.5)[0] == 0 and S.row(np.zeros(4), 0.51, p=0.5)[0] == 1
    assert S.row(np.full(3, -np.inf), 0.5)[:2] == (-1, 0.0)
    assert S.row([np.inf, 0, np.inf], 0.6)[0] == 2
    assert S.row([0, np.nan], 0.5)[0] == -1 and S.row(x, 1.0)[0] == -1 and S.row(x, 0.5, p=0.0)[0] == -1


def test_abi_refusals():
    from ivf_quantizer_b200 import _lib
    L, p, z = _lib.LIB, ctypes.c_void_p(64), ctypes.c_void_p(0)
    odd = ctypes.c_void_p(72)
    bad, uns = _lib.ERR_INVALID_ARG, _lib.ERR_UNSUPPORTED
    assert L.fgmm_mx4_codes_bytes(3, 33) == 3 * 32 and L.fgmm_mx4_scales_bytes(129, 129) == 4 * 512
    assert L.fgmm_mx4_codes_bytes(0, 4) == 0 and L.fgmm_mx4_scales_bytes(4, 0) == 0
    enc, dec, sc = L.fgmm_mx4_encode, L.fgmm_mx4_decode, L.fgmm_mx4_scores
    assert enc(z, 0, 0, 4, 4, z, z, z) == _lib.OK                 # no rows: nothing to do
    assert enc(p, 0, 2, 0, 4, p, p, z) == bad and enc(p, 0, 2, 4, 3, p, p, z) == bad
    assert enc(p, 7, 2, 4, 4, p, p, z) == bad and enc(z, 0, 2, 4, 4, p, p, z) == bad
    assert enc(p, 0, 2, 4, 4, odd, p, z) == bad and enc(p, 0, 2, 4, 4, p, z, z) == bad
    assert enc(ctypes.c_void_p(66), 0, 2, 4, 4, p, p, z) == bad and enc(p, 0, -1, 4, 4, p, p, z) == bad
    assert enc(p, 0, 1 << 31, 4, 4, p, p, z) == uns
    assert enc(p, 0, 2, (1 << 20) + 1, 1 << 21, p, p, z) == uns
    assert dec(p, p, 2, 4, z, 0, 4, z) == bad and dec(p, p, 2, 4, p, 3, 4, z) == bad
    assert dec(p, odd, 2, 4, p, 0, 4, z) == bad and dec(p, p, 2, 4, p, 0, 3, z) == bad
    assert dec(z, z, 0, 4, z, 0, 4, z) == _lib.OK
    one = ctypes.c_float(1.0)
    assert sc(p, p, 0, p, p, 4, 4, one, z, z, 0, 4, z, z) == _lib.OK
    assert sc(p, p, 2, p, p, 4, 4, one, z, z, 0, 4, z, z) == bad          # no output
    assert sc(p, p, 2, p, p, 4, 4, one, z, p, 0, 3, z, z) == bad          # ldo < N
    assert sc(p, odd, 2, p, p, 4, 4, one, z, p, 0, 4, z, z) == bad
    assert sc(p, p, 2, p, p, 4, 4, one, ctypes.c_void_p(66), p, 0, 4, z, z) == bad
    assert sc(p, p, 2, p, p, 1 << 31, 4, one, z, p, 0, 1 << 31, z, z) == uns
    sa = L.fgmm_sample_logits
    assert sa(z, 0, 0, 4, 4, z, z, z, z, z, z, z, z) == _lib.OK
    assert sa(p, 0, 2, 0, 4, z, z, z, z, p, p, z, z) == bad
    assert sa(p, 0, 2, 4, 3, z, z, z, z, p, p, z, z) == bad
    assert sa(p, 9, 2, 4, 4, z, z, z, z, p, p, z, z) == bad
    assert sa(p, 0, 2, 4, 4, z, z, z, z, z, p, z, z) == bad               # no uniforms
    assert sa(p, 0, 2, 4, 4, z, z, z, z, p, z, z, z) == bad               # no ids
    two = ctypes.c_void_p(66)
    for i in range(5, 12):                                               # pointers off their elements
        args = [p, 0, 2, 4, 4, z, z, z, z, p, p, z, z]
        args[i] = two
        assert sa(*args) == bad, i
    assert sa(two, 0, 2, 4, 4, z, z, z, z, p, p, z, z) == bad
    assert sc(p, p, 2, p, p, 4, 4, one, z, p, 0, 4, two, z) == bad        # the status word
    assert sa(p, 0, 2, (1 << 22) + 1, 1 << 23, z, z, z, z, p, p, z, z) == uns


def test_binding_refuses_cpu_tensors_and_bad_shapes():
    import ivf_quantizer_b200 as q
    with pytest.raises(ValueError):
        q.MX4(torch.zeros(4, 8))
    with pytest.raises(ValueError):
        q.MX4.from_codes(torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8), 8)
    with pytest.raises(ValueError):
        q.sample_logits(torch.zeros(4, 8), torch.zeros(4, dtype=torch.float64))
