"""Each kernel of the 4-bit products, chosen by sizes and types, on inputs whose results are exact."""
import pytest

from q4_forms import CALLS, SCALES

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dbs():
    import spmspv_graph_traversal_amd as d

    return d


# x, gated, m, n, tokens: waves that share x go the same number of rounds, of which here the last has no column block for some
EMPTY_ROUNDS = [("bf16", False, 8300, 1100, 16), ("bf16", False, 8300, 1100, 6), ("f32", False, 8300, 1100, 16),
                ("f32", False, 8300, 1100, 6), ("f32", False, 8300, 600, 40), ("f32", False, 16500, 600, 7),
                ("bf16", True, 4200, 2100, 16), ("bf16", True, 4200, 2100, 5), ("f32", True, 4200, 2100, 16),
                ("f32", True, 4200, 2100, 5), ("bf16", True, 8300, 1100, 16), ("f32", True, 8300, 1100, 16),
                ("f32", True, 8300, 1100, 6), ("bf16", False, 26003, 1590, 32), ("bf16", True, 10000, 3101, 32)]


@pytest.mark.parametrize("kind,gated,m,n,tokens", EMPTY_ROUNDS)
def test_rounds_without_a_column_block_add_nothing(dbs, kind, gated, m, n, tokens):
    """With records of eight words, which take two loads, neither of which may reach the first tile's."""
    from q4_device import check_products, small

    check_products(dbs, m + n + tokens, m, n, tokens, 32, True, "f32", gated, small(n, tokens, n, kind))


@pytest.mark.parametrize("scales,group", SCALES)
@pytest.mark.parametrize("kind,gated,m,tokens,columns", CALLS)
def test_every_kernel_is_exact_on_integers(dbs, kind, gated, m, tokens, columns, scales, group):
    from q4_device import check_products, small

    for n in columns:
        check_products(dbs, m + n + tokens, m, n, tokens, group, group != 64, scales, gated, small(n, tokens, n, kind))


@pytest.mark.parametrize("scales,group", SCALES)
@pytest.mark.parametrize("kind,gated,m,tokens,columns", [c for c in CALLS if c[0] == "f32"])
def test_every_fp32_kernel_keeps_the_low_parts_of_x(dbs, kind, gated, m, tokens, columns, scales, group):
    from q4_device import check_products, wide

    for n in columns:
        check_products(dbs, 1 + m + n + tokens, m, n, tokens, group, group != 64, scales, gated, wide(n, tokens, n), halvings=1)


def test_row_groups_of_more_than_one_grid_row(dbs):
    """More row groups than eight grid rows of 65535 hold: the grid folds them."""
    import torch

    from q4_device import Q4, small

    m, n = 16 * 8 * 65535 + 5000, 9
    w = Q4(5, m, n, 32, True, "bf16")
    A, w64 = w.build(dbs), w.w.t()
    for tokens, kind in ((1, "bf16"), (3, "f32"), (6, "bf16")):
        x = small(tokens, tokens, n, kind)
        y = torch.full((tokens, m), 7.0, device="cuda")
        words = torch.full((tokens, (m + 31) // 32), -1, device="cuda", dtype=torch.int32)
        words[:, 100:-200] = 0
        dbs.dbs_q4_product_masked(A, x, words, y)  # sixteen rows a workgroup, up to four tokens
        expect = x.double() @ w64
        inside = slice(3200, (words.shape[1] - 200) * 32)
        assert torch.equal(y[:, :3200].double(), expect[:, :3200]) and (y[:, inside] == -torch.inf).all()
        assert torch.equal(y[:, inside.stop:].double(), expect[:, inside.stop:])
        dbs.dbs_q4_product(A, x, y)
        assert torch.equal(y.double(), expect)
