"""The attention over the cache of 4-bit keys and values where there is no memory for its workspace, on the GPU."""
import pytest

from test_gpu_kv4 import dbs  # noqa: F401

pytestmark = pytest.mark.gpu


def test_a_workspace_that_cannot_be_allocated(dbs):
    """torch's own exception; the same call with an empty workspace, and with the memory back, is answered."""
    import torch

    page, pages, room = 64, 8, 1 << 14
    cache = dbs.dbs_kv4_cache(pages, 1, 128, 128, page)
    table = torch.full((1, room), -1, dtype=torch.int32, device="cuda")
    table[0, :pages] = torch.arange(pages, dtype=torch.int32)
    lens = torch.full((1,), pages * page, dtype=torch.int32, device="cuda")
    kv = torch.randn(pages * page, 1, 128, device="cuda")
    dbs.dbs_kv4_store(cache, table, lens, kv, kv)
    q = torch.randn(pages * page, 32, 128, device="cuda")
    outs = [torch.empty_like(q) for _ in range(3)]
    size = dbs.dbs_kv4_attention_workspace(cache, table, lens, q, outs[0])
    assert size > 1 << 24
    dbs.dbs_kv4_attention(cache, table, lens, q, outs[0])
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    limit = torch.cuda.memory_reserved() + size // 2
    held = []
    try:
        torch.cuda.set_per_process_memory_fraction(limit / torch.cuda.get_device_properties(0).total_memory)
        with pytest.raises(torch.OutOfMemoryError):  # what is free in segments that cannot be returned
            while True:
                held.append(torch.empty(size, dtype=torch.uint8, device="cuda"))
        with pytest.raises(torch.OutOfMemoryError):
            dbs.dbs_kv4_attention(cache, table, lens, q, outs[1])
        dbs.dbs_kv4_attention(cache, table, lens, q, outs[1], workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    finally:
        del held
        torch.cuda.set_per_process_memory_fraction(1.0)
    dbs.dbs_kv4_attention(cache, table, lens, q, outs[2])
    assert torch.equal(outs[2], outs[0])
    # each is off by 2 (dim + 8) roundings of a score's size, some 7 here, and by less for all else: 1.2e-4 of the largest value at most
    assert float((outs[1] - outs[0]).abs().max()) <= 3e-4 * float(kv.abs().max())
