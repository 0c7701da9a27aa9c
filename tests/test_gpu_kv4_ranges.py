"""The attention over the cache of 4-bit keys and values at the ends of what q and the scale can be, against 64-bit references, on
the GPU: in the kernel for few rows and in the one for many, with tokens that some rows do not see in the same block."""
import math

import numpy as np
import pytest

import kv4_ref as ref
from test_gpu_kv4 import cuda, dbs, empty, host, on_gpu, tables  # noqa: F401  (dbs: the fixture)

pytestmark = pytest.mark.gpu

# rows of a sequence: the kernel for few rows with one tile a wave and two, the one for many rows
ROWS = [5, 30, 130]


def run(dbs, c, table, n, q, kind, out_kind, scale, **more):
    out = empty(q.shape, out_kind)
    dbs.dbs_kv4_attention(on_gpu(dbs, c), cuda(table), cuda(np.array([n], np.int32)), cuda(q, kind), out, scale=scale, **more)
    return host(out).astype(np.float64)


def one_sequence(seed, n, dim, group, page=64):
    rng = np.random.default_rng(seed)
    table, pages = tables(rng, [n], page)
    c = ref.Cache(pages, 1, dim, group, page)
    ref.random_bytes(rng, c)
    return rng, table, c


# (largest |q|, scale, head_dim, types): products down to where fp32 ends and behind it
SMALL = [(2.0 ** -140, None, 128, ("f32", "f32")), (2.0 ** -140, None, 64, ("f32", "bf16")), (2.0 ** -149, None, 256, ("f32", "f32")),
         (2.0 ** -133, None, 256, ("bf16", "bf16")), (1e-5, 1e-38, 64, ("bf16", "bf16")), (1e-5, 1e-38, 128, ("f32", "f32")),
         (1.0, 2.0 ** -149, 128, ("bf16", "bf16")), (2.0 ** -126, 2.0 ** -126, 64, ("f32", "f32"))]


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("size,scale,dim,types", SMALL)
def test_scores_that_are_next_to_nothing(dbs, size, scale, dim, types, rows):
    """Each row is the mean of what it sees, to fp32: scale q k is below 2^-100 wherever it is."""
    n = 150
    rng, table, c = one_sequence(rows + dim, n, dim, 64)
    q = ref.typed(size * rng.choice([-1.0, -0.5, 0.0, 0.5, 1.0], (rows, 1, dim)), types[0])
    q[:, 0, 3] = size
    assert q.max() > 0
    scale = 1 / math.sqrt(dim) if scale is None else scale
    got = run(dbs, c, table, n, q, *types, scale)
    k, v = ref.sequence_values(c, table[0], n)
    assert scale * size * np.abs(k).sum(-1).max() < 2.0 ** -100
    for i in range(rows):
        want, mass, score = ref.attention(q[i, 0].astype(np.float64), k[0], v[0], n - rows + i, scale)
        tol = ref.attention_tolerance(want, mass, score, dim, n, types[1], "f32" in types)
        assert (np.abs(got[i, 0] - want) <= tol).all(), f"token {i}"


# scores (times log2 e) around 2^26 and above, where fp32 has steps of 8 and more, to where they leave its range
LARGE = [(2.0 ** p, 1.0) for p in (19, 20, 21, 22, 23, 24, 30, 60, 118)] + [(2.0 ** 12, 2.0 ** 100), (2.0 ** 124, 2.0 ** 124), (1.0, 3e37)]


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("types", [("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("size,scale", LARGE)
def test_scores_of_any_size_single_out_the_largest(dbs, size, scale, types, rows):
    """Scores that lie much further apart than they are off: each row is the value of the token with the largest one."""
    n, dim = 200, 128
    rng, table, c = one_sequence(rows, n, dim, 128)
    q = ref.typed(size * rng.normal(0, 1, (rows, 1, dim)), types[0])
    got = run(dbs, c, table, n, q, *types, scale)
    k, v = ref.sequence_values(c, table[0], n)
    sure = 0
    for i in range(rows):
        x = q[i, 0].astype(np.float64) * np.float64(np.float32(scale))
        see = n - rows + i + 1
        score, of = k[0, :see] @ x, np.abs(k[0, :see]) @ np.abs(x)
        order = np.argsort(score)
        # a score is off by dim + 8 roundings of its size, and the bf16 kinds hold q as halves of the row's scale (2^-25 of its largest
        # element for those that are not exact): far less than the distance asked for, beyond which a weight is below 2^-90
        apart = score[order[-1]] - score[order[-2]]
        if apart < 4 * (dim + 8) * 2.0 ** -22 * of.max() + 64:
            continue
        sure += 1
        want = v[0, order[-1]]
        # one weight, which divides out: three roundings in fp32, and the output's
        assert (np.abs(got[i, 0] - want) <= (ref.HALF_STEP[types[1]] + 2.0 ** -22) * np.abs(want)).all(), f"token {i}"
    assert sure >= 0.8 * rows  # of the inputs


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("types", [("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")])
def test_infinite_queries_make_their_rows_nan(dbs, types, rows):
    """The difference of two infinite scores is no number.  A row that sees nothing is 0 all the same."""
    n, dim, heads = 140, 64, 2
    rng, table, c = one_sequence(rows, n, dim, 32)
    q = rng.normal(0, 1, (rows, heads, dim)).astype(np.float32)
    fine = run(dbs, c, table, n, q, *types, 0.125)
    wrong = q.copy()
    wrong[1, 0, 9], wrong[2, 1, 40] = np.inf, -np.inf
    got = run(dbs, c, table, n, wrong, *types, 0.125)
    assert np.isnan(got[1, 0]).all() and np.isnan(got[2, 1]).all()
    got[1, 0], got[2, 1] = fine[1, 0], fine[2, 1]
    np.testing.assert_array_equal(got, fine)
    empty_table = np.full_like(table, -1)
    assert (run(dbs, c, empty_table, n, wrong, *types, 0.125) == 0).all()


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_rows_whose_scores_are_all_minus_infinity(dbs, rows, sign):
    """One infinite element of a bf16 query and keys of one sign in its channel, in one piece and in splits."""
    n, dim, page = 140, 64, 64
    rng = np.random.default_rng(rows)
    table, pages = tables(rng, [n], page, extra=200)
    c = ref.Cache(pages, 1, dim, 32, page)
    k = rng.normal(0, 1, (n, 1, dim)).astype(np.float32)
    k[..., 7] = sign * (1 + np.abs(k[..., 7]))
    v = rng.normal(0, 1, (n, 1, dim)).astype(np.float32)
    for t in range(n):
        stands, _ = c.store(table[0, t // page], t % page, 0, k[t, 0], v[t, 0])
        assert sign * stands[7] > 0
    q = ref.typed(rng.normal(0, 1, (rows, 1, dim)), "bf16")
    q[rows // 2, 0, 7] = -sign * np.inf
    for max_len in (0, n):
        got = run(dbs, c, table, n, q, "bf16", "bf16", 0.125, max_len=max_len)
        assert np.isnan(got[rows // 2, 0]).all()
        assert np.isfinite(np.delete(got, rows // 2, 0)).all()


def strong_and_tail(dbs, below, rows, dim, group):
    """Outputs in fp32 for sequences of one token whose weight is 2^`below` times that of each of some 16000 others, which carry all of the
    values, in one piece: the channel of those values, got and wanted for each row, and what relative error the exponentials and the sums leave."""
    import torch

    n, page = 16001, 256
    rng = np.random.default_rng(dim)
    table, pages = tables(rng, [n], page)
    cache = dbs.dbs_kv4_cache(pages, 1, dim, group, page)
    k = np.zeros((n, 1, dim), np.float32)
    k[..., 1::group] = 15.0  # every group holds 0 and 15: s = 1, b = 0, and all small integers are themselves
    v = k.copy()
    k[0, 0, 5] = 1.0
    v[1:, 0, 4] = 8.0
    lens = cuda(np.array([n], np.int32))
    vo = empty(v.shape, "f32")
    dbs.dbs_kv4_store(cache, cuda(table), lens, cuda(k), cuda(v), v_out=vo)
    assert torch.equal(vo, cuda(v))
    q = np.zeros((rows, 1, dim), np.float32)
    q[..., 5] = np.float32(below * math.log(2.0))  # the only product that is not 0
    out = empty(q.shape, "f32")
    dbs.dbs_kv4_attention(cache, cuda(table), lens, cuda(q), out, scale=1.0, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    got = host(out).astype(np.float64)[:, 0, 4]
    tail = (n - rows + np.arange(rows)) * math.exp(-float(q[0, 0, 5]))
    # the exponent: q in two halves, the scale, their product, the difference; the power's own error; sums of two numbers, whose partial
    # sums have tokens / 32 + 64 roundings on their way (of both signs: all of them one way is the bound)
    return got, 8 * tail / (1 + tail), below * 4 * 2.0 ** -22 + 2.0 ** -21 + 2 * (n / 32 + 80) * 2.0 ** -24


@pytest.mark.parametrize("dim,group", [(64, 32), (128, 128), (256, 64)])
@pytest.mark.parametrize("rows", [3, 100])
def test_sums_of_many_small_weights_beside_a_large_one(dbs, rows, dim, group):
    """Weights 1.5 2^-24 of the largest, which halves hold: a pair of them is one and a half steps of a sum that has the largest one in it,
    and would be rounded to two each time."""
    got, want, bound = strong_and_tail(dbs, 24 - math.log2(1.5), rows, dim, group)
    assert (np.abs(got - want) <= bound * want).all(), (np.abs(got - want) / want).max()


@pytest.mark.parametrize("dim,group", [(64, 32), (128, 128), (256, 64)])
@pytest.mark.parametrize("rows", [3, 100])
@pytest.mark.parametrize("below", [17.3, 19.3, 21.6])
def test_a_long_tail_beside_one_strong_token(dbs, below, rows, dim, group):
    """In fp32 calls a weight is off by 2^-35 of the row's largest at most (half a step of the smaller half's 2^-24, the largest being 2^10 or
    more), and all of these err alike: 2^(below - 35) of the output."""
    got, want, bound = strong_and_tail(dbs, below, rows, dim, group)
    assert (np.abs(got - want) <= (bound + 2.0 ** (below - 35)) * want).all(), (np.abs(got - want) / want).max()
