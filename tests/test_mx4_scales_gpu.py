"""Scale bytes that encoding does not make (253 and 254) in codes made elsewhere."""
import numpy as np
import pytest
import torch

from oracle import mx4_oracle as M

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_largest_scales_decode_to_what_the_type_holds(dtype):
    import ivf_quantizer_b200 as q
    s = np.array([[252, 253, 254, 255, 0, 1]] * 3, dtype=np.uint8)
    c = np.tile(np.arange(32, dtype=np.uint8) % 16, (3, 6))
    m = q.MX4.from_codes(torch.from_numpy(M.pack(c)).cuda(), torch.from_numpy(M.tile_scales(s)).cuda(), 192)
    want = torch.from_numpy(M.decode(c, s, 192)).float()       # beyond the largest finite value: infinity
    got = m.decode(dtype)
    assert torch.isinf(want).any() and got.dtype == dtype
    np.testing.assert_array_equal(got.float().cpu().numpy(), want.numpy())
