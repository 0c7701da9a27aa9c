"""The attention's workspace over the cache of 4-bit keys and values is bounded, whatever the table has room for (CPU only)."""
import pytest

import spmspv_graph_traversal_amd.binding as b
from test_kv4_args import OK, PTR, workspace


@pytest.mark.parametrize("heads,key_heads", [(32, 8), (64, 8), (8, 8), (128, 1), (14, 2)])
@pytest.mark.parametrize("dim,group", [(64, 32), (128, 64), (192, 64), (256, 64)])
def test_workspace_is_bounded(heads, key_heads, dim, group):
    """From one token to prompts, of one sequence to many, even and ragged, in tables from nothing to the largest."""
    cut = 0
    for pages in (1, 32, 256, 2048, 1 << 14, 1 << 18, 1 << 22):
        for sequences in (1, 2, 8, 64, 1000):
            for each in (1, 2, 5, 17, 64, 65, 130, 520, 1100, 4160, 8192, 8320, 32768):
                tokens = sequences * each
                if tokens * heads > b.DBS_KV4_MAX_ROWS:
                    continue
                for ragged in (None, PTR):
                    for types in (0, 1):
                        for window in (0, 5000):
                            st, size = workspace(tokens=tokens, heads=heads, key_heads=key_heads, head_dim=dim, group=group, sequences=sequences,
                                                 table_pages=pages, ldtable=pages, page_tokens=256, new_ptr=ragged, qd=types, od=types, window=window)
                            assert st == OK and 0 <= size <= b.DBS_KV4_MAX_WORKSPACE
                            cut += size > 0
    assert cut > 0


def test_bound_of_the_header():
    import os

    header = open(os.path.join(os.path.dirname(__file__), "..", "include", "dbs.h")).read()
    assert f"#define DBS_KV4_MAX_WORKSPACE {b.DBS_KV4_MAX_WORKSPACE}\n" in header
