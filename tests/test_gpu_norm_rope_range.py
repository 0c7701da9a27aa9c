"""Norms with rotary positions of heads whose squares leave fp32, on the GPU."""
import numpy as np
import pytest

import kv4_ref as ref
from test_gpu_kv4 import cuda, dbs, empty, host  # noqa: F401  (dbs: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_heads_whose_squares_leave_fp32(dbs, kind):
    """Too large ones are 0, and in their own head alone; small ones are the formula's down to where their mean is no fp32 number, and too
    small ones infinite or NaN, as with any eps that does not hold them up."""
    rng = np.random.default_rng(1)
    dim = 64
    x = ref.typed(rng.choice([-1.0, 1.0], (2, 6, dim)) * rng.uniform(0.5, 1, (2, 6, dim)), kind)
    size = [2.0 ** 80, 2.0 ** 127, 2.0 ** 55, 2.0 ** -55, 2.0 ** -90, 0.0]
    x = x * np.array(size, np.float32)[None, :, None]
    pos, freq = np.array([3, 70000], np.int32), 10000.0 ** (-np.arange(dim // 2) / (dim // 2))
    for eps in (0.0, 1e-6):
        out = empty(x.shape, "f32")
        dbs.dbs_norm_rope(cuda(x, kind), None, None, None, cuda(pos), cuda(freq), out, None, eps=eps)
        got = host(out)
        held = [2, 3] if eps == 0 else [2, 3, 4, 5]
        want, large = ref.norm_rope(x[:, held], None, float(np.float32(eps)), pos, freq, False)
        # the sum's 64 roundings in half, the root, the product, the turn (2^-22 of its size twice) and the output's
        assert (np.abs(got[:, held] - want) <= (64 + 8) * 2.0 ** -24 * large).all()
        assert (got[:, :2] == 0).all()
        if eps == 0:
            assert not np.isfinite(got[:, 4]).any() and np.isnan(got[:, 5]).all()
