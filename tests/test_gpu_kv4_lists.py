"""Lists of new tokens that the attention and the store over the cache of 4-bit keys and values clamp, on the GPU."""
import numpy as np
import pytest

import kv4_ref as ref
from test_gpu_kv4 import cuda, dbs, empty, host, on_gpu  # noqa: F401  (dbs: the fixture)

pytestmark = pytest.mark.gpu

TOKENS = 9


def calls(dbs, ptr, rows_per_key):
    """Attention and store under a list: the outputs within larger buffers, the pool, and what all of them held before."""
    import torch

    rng = np.random.default_rng(18)
    page = 16
    c = ref.Cache(8, 1, 64, 64, page)  # two pages more than the table names
    ref.random_bytes(rng, c)
    cache = on_gpu(dbs, c)
    table, lens = cuda(np.array([[0, 1], [2, 3], [4, 5]], np.int32)), cuda(np.array([20, 20, 20], np.int32))
    ptr = cuda(np.array(ptr, np.int32))
    q = cuda(rng.normal(0, 1, (TOKENS, rows_per_key, 64)).astype(np.float32))
    kv = cuda(rng.normal(0, 1, (TOKENS, 2, 64)).astype(np.float32))
    guarded = empty((TOKENS + 4, rows_per_key, 64), "f32")
    dbs.dbs_kv4_attention(cache, table, lens, q, guarded[2:-2], new_ptr=ptr)
    stands = empty((TOKENS + 4, 2, 64), "f32")
    dbs.dbs_kv4_store(cache, table, lens, kv[:, :1], kv[:, 1:], new_ptr=ptr, k_out=stands[2:-2, :1], v_out=stands[2:-2, 1:])
    torch.cuda.synchronize()
    return host(guarded), host(stands), cache.pool.cpu().numpy(), c.bytes


@pytest.mark.parametrize("rows_per_key", [2, 40])
@pytest.mark.parametrize("ptr", [[-3, 3, 5, 1 << 30], [0, 0, 9, 9], [2, 4, 4, 7], [-(1 << 31), -1, 0, 4], [9, 9, 9, 12]])
def test_entries_out_of_range_are_clamped(dbs, ptr, rows_per_key):
    """A list that does not decrease gives what it gives with its entries clamped to the rows that there are; rows that it does not name
    and what lies around the outputs are left alone."""
    clamped = [min(max(p, 0), TOKENS) for p in ptr]
    got, want = calls(dbs, ptr, rows_per_key), calls(dbs, clamped, rows_per_key)
    for x, y in zip(got, want):
        np.testing.assert_array_equal(x, y)
    named = np.zeros(TOKENS + 4, bool)
    named[2 + clamped[0] : 2 + clamped[-1]] = True
    for x in got[:2]:
        assert (x[~named] == 7.0).all() and (x[named] != 7.0).any(axis=(1, 2)).all()
    assert (got[2][6:] == got[3][6:]).all()


@pytest.mark.parametrize("rows_per_key", [2, 40])
@pytest.mark.parametrize("ptr", [[0, 3, 6, 4], [5, 2, 9, 9], [-3, 100, 3, 1 << 30], [9, 6, 3, 0]])
def test_lists_that_decrease_write_no_row_that_they_do_not_name(dbs, ptr, rows_per_key):
    """They name no sequences, and nothing is said of the rows between their entries; nothing else is written."""
    clamped = [min(max(p, 0), TOKENS) for p in ptr]
    guarded, stands, pool, before = calls(dbs, ptr, rows_per_key)
    named = np.zeros(TOKENS + 4, bool)
    for a, b in zip(clamped[:-1], clamped[1:]):
        named[2 + a : 2 + max(a, b)] = True
    assert (guarded[~named] == 7.0).all() and (stands[~named] == 7.0).all()
    assert (pool[6:] == before[6:]).all()
