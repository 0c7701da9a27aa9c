"""The attention over the cache of 4-bit keys and values in tables with far more room than the sequences have, on the GPU: most splits see
nothing and leave their rows of the workspace as they were."""
import numpy as np
import pytest

from test_gpu_kv4 import dbs  # noqa: F401
from test_gpu_kv4_paths import BOTH, check

pytestmark = pytest.mark.gpu


# lengths, new tokens of each, key heads, rows of a key head and token: one split of many with tokens in it, or two, for rows that have a workgroup
# each to join them and for so many that none does
@pytest.mark.parametrize("lengths,new,heads,rep", [([1500], [1], 2, 4), ([3000, 40, 0], [1, 1, 1], 2, 4), ([3001, 900], [5, 5], 2, 7), ([300], [300], 1, 2),
                                                   ([1100], [1100], 1, 8), ([1400, 700], [1200, 70], 2, 8)])
@pytest.mark.parametrize("dim,group", [(64, 32), (128, 128), (256, 64)])
def test_rows_that_no_split_wrote_are_not_taken(dbs, lengths, new, heads, rep, dim, group):
    """A workspace full of NaN, and a bound of the lengths beside none."""
    import torch

    for max_len in (0, max(lengths)):
        rng = np.random.default_rng(dim + sum(new))
        scratch = torch.full((1 << 29,), 0xFF, dtype=torch.uint8, device="cuda")
        check(dbs, rng, lengths, new, heads, rep, dim, group, types=BOTH, extra=1 << 14, max_len=max_len, many=4, workspace=scratch)
        assert bool((scratch[:: 1 << 12] != 0xFF).any()) or max_len
