"""Each kernel of the 4-bit products, chosen by sizes and types, on inputs whose results are exact."""
import pytest

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
