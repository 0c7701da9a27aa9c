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


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,group,zeros,scales", [(48, 1000, 64, True, "bf16"), (70, 333, 32, True, "f32"), (40, 4100, 128, False, "bf16"),
                                                    (33, 31, 32, True, "bf16"), (5000, 700, 64, True, "f32")])
def test_weights_of_zero_add_nothing(dbs, kind, m, n, group, zeros, scales):
    """Rows and groups whose codes all equal their zero point, next to others, under x of real values: those rows are 0, so are
    ReLU gates of them, and the others' error has no part of such groups."""
    import numpy as np
    import torch

    import decode_ref as ref

    rng = np.random.default_rng(m + n)
    w, u = ref.Q4(rng, m, n, group, zeros, scales, exact=False), ref.Q4(rng, m, n, group, zeros, scales, exact=False)
    none = rng.random((m, w.s.shape[1])) < 0.5  # groups of weights 0
    none[::3] = True                            # and whole rows
    none[1::3, 0] = False
    w.q = np.where(none[:, w.of], w.offset, w.q).astype(np.uint8)
    assert (w.w[::3] == 0).all()
    A, U = w.build(dbs), u.build(dbs)
    for t in (1, 3, 7, 16, 37):
        x = rng.standard_normal((t, n)).astype(np.float32)
        x = ref.bf16(x) if kind == "bf16" else x
        xs = torch.from_numpy(x).cuda()
        xs = xs.bfloat16() if kind == "bf16" else xs
        y = torch.full((t, m), 7.0, device="cuda")
        dbs.dbs_q4_gated(A, U, xs, dbs.DBS_ACT_RELU, y)
        assert (y[:, ::3] == 0).all()
        dbs.dbs_q4_product(A, xs, y)
        assert (y[:, ::3] == 0).all()
        held = w.s
        w.s = np.where(none, 0, held)  # the bound of the other groups alone
        assert (np.abs(y.cpu().numpy() - x.astype(np.float64) @ w.w.T) <= w.bound(x)).all()
        w.s = held


def test_infinities_times_weights_of_zero(dbs):
    """An infinite x or scale makes NaN of a weight 0, as in the formula; a scale of 0 otherwise changes nothing."""
    import torch

    m, n = 20, 200
    zeros = torch.arange(m * 4, device="cuda").view(m, 4).remainder(16).to(torch.uint8)
    codes = (zeros * 17).repeat_interleave(32, 1)[:, :100].contiguous()
    scales = torch.ones(m, 4, device="cuda")
    scales[3, 1], scales[4, 3] = float("inf"), float("nan")
    A = dbs.dbs_q4_build(m, n, 64, codes, scales, zeros)
    x = torch.ones(3, n, device="cuda")
    x[1, 7], x[2, 150] = float("inf"), 3e38
    y = torch.full((3, m), 7.0, device="cuda")
    dbs.dbs_q4_product(A, x, y)
    expect = torch.zeros(3, m, device="cuda")
    expect[:, 3], expect[:, 4], expect[1] = torch.nan, torch.nan, torch.nan
    assert torch.equal(y.nan_to_num(-5.0), expect.nan_to_num(-5.0))


@pytest.mark.parametrize("kind", [0, 1])
def test_activations_keep_their_precision_for_negative_gates(dbs, kind):
    """act(g) g for gates g = k / 64, exact in the products, against 64 bits, relative to the result itself."""
    import numpy as np
    import torch

    import decode_ref as ref

    g = np.arange(-20 * 64, 20 * 64 + 1) / 64
    one = torch.ones(1, 1, device="cuda")
    A = dbs.dbs_q4_build(1, 1, 32, torch.full((1, 1), 9, dtype=torch.uint8, device="cuda"), one)  # W = 9 - 8
    y = torch.full((len(g), 1), 7.0, device="cuda")
    dbs.dbs_q4_gated(A, A, torch.from_numpy(g).float().cuda()[:, None], kind, y)
    u2 = 2 * np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3) if kind == 1 else g
    with np.errstate(over="ignore"):
        expect = g / (1 + np.exp(-u2)) * g
    # in half steps: the argument of exp 8 of itself (five for the cube, one for the sum, two for the factor; SiLU's is exact), exp 4,
    # the sum 1, the quotient 5, the product 1.  Where exp overflows the result is below 20^2 / 2^128.
    tol = ((8 * np.abs(u2) if kind == 1 else 0) + 11) * ref.U24 * np.abs(expect) + 400 * 2.0 ** -128
    error = np.abs(y[:, 0].cpu().numpy().astype(np.float64) - expect)
    assert (error <= tol).all(), (g[error > tol][:5], (error / tol).max())


def test_builds_on_a_stream(dbs):
    """A stream of the current device is used, one of another device refused."""
    import torch

    from q4_device import Q4, small

    class Stream:
        cuda_stream = 0
        device_index = torch.cuda.current_device() + 1

    w = Q4(3, 40, 100, 32, True, "f32")
    with pytest.raises(ValueError, match="stream"):
        dbs.dbs_q4_build(40, 100, 32, w.codes, w.scales, w.zeros, stream=Stream())
    x, y = small(1, 3, 100, "f32"), torch.full((3, 40), 7.0, device="cuda")
    torch.cuda.synchronize()
    A = dbs.dbs_q4_build(40, 100, 32, w.codes, w.scales, w.zeros, stream=torch.cuda.Stream())
    dbs.dbs_q4_product(A, x, y)
    assert torch.equal(y.double(), x.double() @ w.w.t())


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
