"""The operators of a decoded token around the sparse products (4-bit products, logits adjustments, rotary
positions) against 64-bit references, on the GPU."""
import numpy as np
import pytest

import decode_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dbs():
    import spmspv_graph_traversal_amd as d

    return d


def cuda(a, kind=None):
    import torch

    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t.bfloat16() if kind == "bf16" else t


def empty(shape, kind):
    import torch

    return torch.full(shape, 7.0, dtype=torch.bfloat16 if kind == "bf16" else torch.float32, device="cuda")


def host(t):
    return t.float().cpu().numpy()


def rounded(a, kind):
    """64-bit values that fp32 holds exactly, rounded to the output's type."""
    return ref.bf16(a) if kind == "bf16" else np.asarray(a, np.float32)


def integers(rng, t, n):
    return rng.integers(-4, 5, (t, n)).astype(np.float32)


# m, n, group, zeros, scales: one column and row, cut tiles, groups and bytes, several of each
SHAPES = [
    (1, 1, 32, True, "bf16"),
    (16, 128, 128, False, "bf16"),
    (5, 31, 32, False, "f32"),
    (17, 33, 32, True, "bf16"),
    (33, 129, 64, True, "f32"),
    (100, 255, 128, True, "bf16"),
    (64, 1000, 64, False, "bf16"),
    (271, 2047, 32, True, "bf16"),
    (48, 5000, 128, True, "f32"),
    (1040, 640, 64, True, "bf16"),
    (40, 11008, 128, True, "bf16"),
]


@pytest.mark.parametrize("x_kind", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,group,zeros,scales", SHAPES)
def test_product_is_exact_on_integers(dbs, m, n, group, zeros, scales, x_kind):
    """Small integers times codes with power-of-two scales: every sum fits fp32, so any order gives the exact
    result, and one wrong index shows."""
    rng = np.random.default_rng(m * 7919 + n)
    w = ref.Q4(rng, m, n, group, zeros, scales)
    A = w.build(dbs)
    for t in (1, 2, 4, 5, 16, 17, 33, 64, 67):
        x = integers(rng, t, n)
        expect = x.astype(np.float64) @ w.w.T
        for y_kind in ("f32", "bf16"):
            y = empty((t, m), y_kind)
            dbs.dbs_q4_product(A, cuda(x, x_kind), y)
            np.testing.assert_array_equal(host(y), rounded(expect, y_kind), err_msg=f"{t} tokens, {y_kind}")


@pytest.mark.parametrize("x_kind", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,group,zeros,scales", [(8300, 300, 32, True, "bf16"), (8207, 1408, 128, False, "bf16"),
                                                    (33000, 130, 64, True, "f32"), (600, 9000, 128, True, "bf16")])
def test_products_of_many_rows_are_exact_on_integers(dbs, m, n, group, zeros, scales, x_kind):
    """Sizes that take each way of cutting a call into workgroups, for one matrix and for two."""
    import torch

    rng = np.random.default_rng(m)
    w, u = ref.Q4(rng, m, n, group, zeros, scales), ref.Q4(rng, m, n, group, zeros, scales)
    A, U = w.build(dbs), u.build(dbs)
    w64, u64 = torch.from_numpy(w.w).cuda().t(), torch.from_numpy(u.w).cuda().t()
    for t in (1, 4, 7, 16, 40, 130):
        x = cuda(integers(rng, t, n))
        xx = x.bfloat16() if x_kind == "bf16" else x
        g, h = x.double() @ w64, x.double() @ u64
        y = empty((t, m), "f32")
        dbs.dbs_q4_product(A, xx, y)
        assert torch.equal(y.double(), g), f"{t} tokens"
        dbs.dbs_q4_gated(A, U, xx, dbs.DBS_ACT_RELU, y)
        assert torch.equal(y, (g.clamp_min(0) * h).float()), f"{t} tokens, gated"
        words = cuda(rng.integers(-2 ** 31, 2 ** 31, (t, (m + 31) // 32)).astype(np.int32))
        words[:, : m // 80] = 0
        row = torch.arange(m, device="cuda")
        wanted = (words[:, row // 32] >> (row % 32)) & 1 != 0
        dbs.dbs_q4_product_masked(A, xx, words, y)
        assert torch.equal(y.double(), torch.where(wanted, g, -np.inf)), f"{t} tokens, masked"


@pytest.mark.parametrize("x_kind", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,group,zeros,scales", [(4099, 4100, 128, True, "bf16"), (4097, 700, 32, False, "f32"),
                                                    (7003, 2111, 64, True, "bf16"), (14500, 520, 64, False, "bf16")])
def test_products_of_two_row_blocks_are_exact_on_integers(dbs, m, n, group, zeros, scales, x_kind):
    """Matrices whose row blocks, and pairs of row and token blocks, are shared out two to a workgroup (and the counts beside)."""
    import torch

    rng = np.random.default_rng(m * 3 + n)
    w, u = ref.Q4(rng, m, n, group, zeros, scales), ref.Q4(rng, m, n, group, zeros, scales)
    A, U = w.build(dbs), u.build(dbs)
    w64, u64 = torch.from_numpy(w.w).cuda().t(), torch.from_numpy(u.w).cuda().t()
    for t in (1, 2, 3, 4, 5, 15, 16, 20, 31, 33):
        x = cuda(integers(rng, t, n))
        xx = x.bfloat16() if x_kind == "bf16" else x
        g, h = x.double() @ w64, x.double() @ u64
        y = empty((t, m), "f32")
        dbs.dbs_q4_product(A, xx, y)
        assert torch.equal(y.double(), g), f"{t} tokens"
        dbs.dbs_q4_gated(A, U, xx, dbs.DBS_ACT_RELU, y)
        assert torch.equal(y, (g.clamp_min(0) * h).float()), f"{t} tokens, gated"
        words = cuda(rng.integers(-2 ** 31, 2 ** 31, (t, (m + 31) // 32)).astype(np.int32))
        words[:, : m // 80] = 0
        words[:, -1] = 2 - (1 << 31)
        row = torch.arange(m, device="cuda")
        wanted = (words[:, row // 32] >> (row % 32)) & 1 != 0
        dbs.dbs_q4_product_masked(A, xx, words, y)
        assert torch.equal(y.double(), torch.where(wanted, g, -np.inf)), f"{t} tokens, masked"


@pytest.mark.parametrize("m,n,group,zeros,scales", [(26003, 1590, 32, True, "bf16"), (26003, 1537, 64, False, "f32"),
                                                    (24100, 3101, 128, True, "bf16")])
def test_products_of_two_token_tiles_are_exact_on_integers(dbs, m, n, group, zeros, scales):
    """Matrices of so many rows and columns that workgroups take 32 tokens, with a last tile that is cut, an infinity and
    rows of x and y with strides."""
    import torch

    rng = np.random.default_rng(m + n)
    w, u = ref.Q4(rng, m, n, group, zeros, scales), ref.Q4(rng, m, n, group, zeros, scales)
    A, U = w.build(dbs), u.build(dbs)
    w64, u64 = torch.from_numpy(w.w).cuda().t(), torch.from_numpy(u.w).cuda().t()
    for t in (17, 32, 50, 64, 90):
        wide = torch.full((t, n + 3), float("nan"), device="cuda", dtype=torch.bfloat16)
        x = wide[:, 1:n + 1]
        x.copy_(cuda(integers(rng, t, n)))
        g, h = x.double() @ w64, x.double() @ u64
        out = torch.full((t, m + 5), 7.0, device="cuda")
        y = out[:, 2:m + 2]
        dbs.dbs_q4_product(A, x, y)
        assert torch.equal(y.double(), g), f"{t} tokens"
        dbs.dbs_q4_gated(A, U, x, dbs.DBS_ACT_RELU, y)
        assert torch.equal(y, (g.clamp_min(0) * h).float()), f"{t} tokens, gated"
        words = cuda(rng.integers(-2 ** 31, 2 ** 31, (t, (m + 31) // 32)).astype(np.int32))
        words[:, m // 80: m // 40] = 0
        row = torch.arange(m, device="cuda")
        wanted = (words[:, row // 32] >> (row % 32)) & 1 != 0
        dbs.dbs_q4_product_masked(A, x, words, y)
        assert torch.equal(y.double(), torch.where(wanted, g, -np.inf)), f"{t} tokens, masked"
        x[t // 2, 5] = float("inf")
        dbs.dbs_q4_product(A, x, y)
        few = [0, t // 2 - 1, t // 2 + 1, t - 1]
        assert torch.equal(y[few].double(), g[few])
        spread = torch.where(w64[5] == 0, torch.nan, w64[5] * np.inf)
        assert torch.equal(y[t // 2].nan_to_num(3.0, 1.0, -1.0).double(), spread.nan_to_num(3.0, 1.0, -1.0))
        assert (out[:, :2] == 7).all() and (out[:, m + 2:] == 7).all()


@pytest.mark.parametrize("x_kind", ["bf16", "f32"])
@pytest.mark.parametrize("tokens", [1, 3, 8, 30, 64])
def test_product_of_real_values(dbs, tokens, x_kind):
    rng = np.random.default_rng(tokens)
    for m, n, group, zeros, scales in SHAPES:
        w = ref.Q4(rng, m, n, group, zeros, scales, exact=False)
        x = (rng.standard_normal((tokens, n)) * np.where(rng.random(n) < 0.01, 30, 1)).astype(np.float32)
        x = ref.bf16(x) if x_kind == "bf16" else x
        y = empty((tokens, m), "f32")
        dbs.dbs_q4_product(w.build(dbs), cuda(x, x_kind), y)
        err = np.abs(host(y) - x.astype(np.float64) @ w.w.T)
        assert (err <= w.bound(x)).all(), f"{m}x{n}: {np.max(err / w.bound(x)):.3g} of the bound"


@pytest.mark.parametrize("tokens", [1, 4, 16, 40])
def test_product_keeps_all_24_bits_of_fp32_x(dbs, tokens):
    """One entry of x with a full mantissa: the result is a few half steps of (16 + q) |x| off at most, while
    the last eight bits left out would be 2^-17 |x| |q - z| off."""
    rng = np.random.default_rng(5)
    w = ref.Q4(rng, 70, 300, 64, True)
    A = w.build(dbs)
    x = np.zeros((tokens, 300), np.float32)
    at = rng.integers(0, 300, tokens)
    x[np.arange(tokens), at] = ((1 << 23) + rng.integers(0, 1 << 22, tokens) * 2 + 1).astype(np.float32)
    y = empty((tokens, 70), "f32")
    dbs.dbs_q4_product(A, cuda(x), y)
    expect = x.astype(np.float64) @ w.w.T
    scale = w.scale[:, at].T * np.abs(x[np.arange(tokens), at])[:, None]
    # three parts, each multiplied exactly, their sums and the offset's: 6 roundings of at most 31 s |x|
    assert (np.abs(host(y) - expect) <= 6 * 31 * ref.U24 * scale).all()


def test_strides_offsets_and_untouched_surroundings(dbs):
    import torch

    rng = np.random.default_rng(11)
    w = ref.Q4(rng, 45, 203, 32, True)
    A = w.build(dbs)
    for t in (1, 3, 21):
        for off, ld in ((0, 203), (1, 204), (3, 251), (8, 208)):
            for kind in ("bf16", "f32"):
                flat = torch.full((off + t * ld + 5,), float("nan"), device="cuda", dtype=torch.bfloat16 if kind == "bf16" else torch.float32)
                x = integers(rng, t, 203)
                view = flat[off:off + t * ld].view(t, ld)[:, :203]
                view.copy_(torch.from_numpy(x))
                out = torch.full((t, 60), -3.0, device="cuda")
                dbs.dbs_q4_product(A, view, out[:, 7:52])
                np.testing.assert_array_equal(host(out[:, 7:52]), (x.astype(np.float64) @ w.w.T).astype(np.float32))
                assert (out[:, :7] == -3).all() and (out[:, 52:] == -3).all()


def test_vectors_of_one_dimension_and_no_tokens(dbs):
    import torch

    rng = np.random.default_rng(12)
    w = ref.Q4(rng, 20, 77, 32, False)
    A = w.build(dbs)
    assert dbs.dbs_q4_bytes(A) >= 2 * 1024
    x = integers(rng, 1, 77)
    y = empty((20,), "f32")
    dbs.dbs_q4_product(A, cuda(x[0]), y)
    np.testing.assert_array_equal(host(y), (x[0].astype(np.float64) @ w.w.T).astype(np.float32))
    dbs.dbs_q4_product(A, torch.empty(0, 77, device="cuda"), torch.empty(0, 20, device="cuda"))
    dbs.dbs_q4_free(A)


def same_kind(got, expect):
    np.testing.assert_array_equal(np.isnan(got), np.isnan(expect))
    inf = np.isinf(expect)
    np.testing.assert_array_equal(np.isinf(got), inf)
    np.testing.assert_array_equal(got[inf], expect[inf])


@pytest.mark.parametrize("x_kind", ["bf16", "f32"])
@pytest.mark.parametrize("tokens", [1, 6, 35])
def test_infinities_and_nan_spread_as_in_the_formula(dbs, tokens, x_kind):
    rng = np.random.default_rng(13)
    w = ref.Q4(rng, 50, 300, 64, True)
    A = w.build(dbs)
    x = integers(rng, tokens, 300)
    x[0, 17] = np.inf            # NaN in rows whose weight there is 0, else an infinity of the weight's sign
    if tokens > 1:
        x[2, 299] = np.nan
        x[3, 5], x[3, 200] = np.inf, -np.inf
        x[4, 64] = 2.0 ** 124    # 15 times it fits fp32, 16 times does not
    y = empty((tokens, 50), "f32")
    dbs.dbs_q4_product(A, cuda(x, x_kind), y)
    with np.errstate(invalid="ignore"):
        expect = ref.dot(w.w, x)
    same_kind(host(y), expect)
    fine = np.isfinite(expect)
    err = np.abs(np.where(fine, host(y).astype(np.float64) - np.where(fine, expect, 0), 0))
    assert (err <= np.where(fine, np.nan_to_num(w.bound(np.nan_to_num(x, posinf=0, neginf=0))), 1)).all()


def test_infinite_and_nan_scales_stay_in_their_rows(dbs):
    rng = np.random.default_rng(14)
    w = ref.Q4(rng, 40, 256, 128, False, "f32")
    w.s[3, 1], w.s[20, 0] = np.inf, np.nan
    x = integers(rng, 2, 256)
    y = empty((2, 40), "f32")
    dbs.dbs_q4_product(w.build(dbs), cuda(x), y)
    with np.errstate(invalid="ignore"):
        expect = ref.dot(w.w, x)
    same_kind(host(y), expect)
    rows = [i for i in range(40) if i not in (3, 20)]
    np.testing.assert_array_equal(host(y)[:, rows], expect[:, rows].astype(np.float32))


# --------------------------------------------------------------------------- masked
@pytest.mark.parametrize("x_kind", ["bf16", "f32"])
@pytest.mark.parametrize("tokens", [1, 2, 5, 19, 64, 70])
def test_masked_product(dbs, tokens, x_kind):
    rng = np.random.default_rng(20 + tokens)
    for m, n, share in ((1, 40, 0.5), (45, 203, 0.5), (513, 130, 0.03), (96, 64, 1.0)):
        w = ref.Q4(rng, m, n, 32, True)
        A = w.build(dbs)
        x = integers(rng, tokens, n)
        allowed = rng.random((tokens, m)) < share
        allowed[-1] = False  # nothing left
        if tokens > 1:
            allowed[0] = True
        y = empty((tokens, m), "f32")
        dbs.dbs_q4_product_masked(A, cuda(x, x_kind), cuda(ref.mask_words(allowed)), y)
        np.testing.assert_array_equal(host(y), np.where(allowed, x.astype(np.float64) @ w.w.T, -np.inf).astype(np.float32))
        y = empty((tokens, m), "bf16")
        dbs.dbs_q4_product_masked(A, cuda(x, x_kind), cuda(ref.mask_words(allowed)), y, fill=0.5)
        np.testing.assert_array_equal(host(y), ref.bf16(np.where(allowed, x.astype(np.float64) @ w.w.T, 0.5)))


def test_masked_product_ignores_bits_past_the_end_and_x_of_closed_tokens(dbs):
    rng = np.random.default_rng(30)
    w = ref.Q4(rng, 40, 100, 64, False)
    A = w.build(dbs)
    x = integers(rng, 3, 100)
    x[1] = np.nan
    words = np.full((3, 2), -1, np.int32)
    words[1] = 0
    words[1, 1] = -256  # bits 40 and above only
    y = empty((3, 40), "f32")
    dbs.dbs_q4_product_masked(A, cuda(x), cuda(words), y)
    expect = x.astype(np.float64) @ w.w.T
    expect[1] = -np.inf
    np.testing.assert_array_equal(host(y), expect.astype(np.float32))


# --------------------------------------------------------------------------- gated
@pytest.mark.parametrize("x_kind,y_kind", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("kind", [0, 1, 2])
def test_gated(dbs, kind, x_kind, y_kind):
    rng = np.random.default_rng(40 + kind)
    for m, n, group, zeros, scales in ((1, 1, 32, True, "bf16"), (50, 300, 64, True, "f32"), (333, 130, 128, False, "bf16"), (33, 1100, 32, True, "bf16")):
        g, u = ref.Q4(rng, m, n, group, zeros, scales), ref.Q4(rng, m, n, group, zeros, scales)
        g.s /= 64  # gates around zero, where the activations differ
        G, U = g.build(dbs), u.build(dbs)
        for t in (1, 3, 16, 41):
            x = integers(rng, t, n)
            y = empty((t, m), y_kind)
            dbs.dbs_q4_gated(G, U, cuda(x, x_kind), kind, y)
            xg, xu = x.astype(np.float64) @ g.w.T, x.astype(np.float64) @ u.w.T
            expect = ref.act(kind, xg) * xu
            # both products are exact; exp and tanh are within 2 ulp, and 1 + tanh may cancel: 8 half steps of |g u|
            tol = 16 * ref.U24 * np.abs(xg * xu) + ref.HALF_STEP[y_kind] * np.abs(expect) + 1e-37
            assert (np.abs(host(y) - expect) <= tol).all()
    dbs.dbs_q4_gated(G, G, cuda(x, x_kind), kind, y)  # one matrix twice
    expect = ref.act(kind, xg) * xg
    assert (np.abs(host(y) - expect) <= 16 * ref.U24 * xg * xg + ref.HALF_STEP[y_kind] * np.abs(expect) + 1e-37).all()


# --------------------------------------------------------------------------- logits
def ragged(lists, dtype):
    ptr = np.zeros(len(lists) + 1, np.int32)
    ptr[1:] = np.cumsum([len(v) for v in lists])
    return ptr, np.array([v for l in lists for v in l], dtype)


@pytest.mark.parametrize("in_kind,out_kind", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("rows,vocab,length", [(1, 1, 3), (1, 5000, 700), (3, 4097, 50), (7, 33, 200), (2, 12289, 9000), (40, 1003, 20)])
def test_logits(dbs, rows, vocab, length, in_kind, out_kind):
    rng = np.random.default_rng(rows * 31 + vocab)
    l = rng.normal(0, 3, (rows, vocab)).astype(np.float32)
    l[0, 0] = 0.0
    if vocab > 8:
        l[0, 3], l[-1, 4], l[-1, 5] = -np.inf, np.inf, np.finfo(np.float32).min / 4
    l = ref.bf16(l) if in_kind == "bf16" else l
    hist = [rng.integers(-2, max(3, vocab // 3), rng.integers(0, length + 1)) for _ in range(rows)]
    hist[-1] = np.full(length, vocab - 1)  # one id many times
    if rows > 2:
        hist[1] = np.zeros(0, np.int64)
    new = rng.integers(-1, length + 2, rows).astype(np.int32)
    rep, freq, pres = (rng.uniform(a, b, rows).astype(np.float32) for a, b in ((0.7, 1.6), (-0.5, 0.5), (0.0, 1.0)))
    bias = [[(int(v), np.float32(rng.normal())) for v in rng.integers(-1, vocab + 2, rng.integers(0, 30))] for _ in range(rows)]
    bias[-1] += [(0, np.float32(1.5)), (0, np.float32(-2.5)), (0, np.float32(0.25))]  # the last counts
    allowed = rng.random((rows, vocab)) < 0.6
    allowed[-1] = rows == 1
    hp, h = ragged(hist, np.int32)
    bp, bi = ragged([[v for v, _ in b] for b in bias], np.int32)
    bv = np.array([x for b in bias for _, x in b], np.float32)
    full = dict(hist_ptr=cuda(hp), hist=cuda(h), hist_new=cuda(new), repetition=cuda(rep), frequency=cuda(freq),
                presence=cuda(pres), bias_ptr=cuda(bp), bias_idx=cuda(bi), bias_val=cuda(bv), mask=cuda(ref.mask_words(allowed)))
    plain = dict(hist=hist, new=new, rep=rep, freq=freq, pres=pres, bias=bias, allowed=allowed)
    uses = [(), ("hist_ptr", "hist", "repetition"), ("hist_ptr", "hist", "frequency"), ("hist_ptr", "hist", "hist_new", "presence"),
            ("bias_ptr", "bias_idx", "bias_val"), ("mask",), tuple(full)]
    names = {"hist": "hist", "hist_new": "new", "repetition": "rep", "frequency": "freq", "presence": "pres", "bias_ptr": "bias", "mask": "allowed"}
    for use in uses:
        out = empty((rows, vocab), out_kind)
        x = cuda(l, in_kind)
        dbs.dbs_logits_adjust(x, out, **{k: full[k] for k in use})
        expect = ref.logits(l, **{names[k]: plain[names[k]] for k in use if k in names})
        got = host(out).astype(np.float64)
        same_kind(got, expect)
        fine = np.isfinite(expect)
        # four steps in fp32 (division, product with the count, two sums) on magnitudes of at most
        # |l| rep + |freq| c + pres + |bias|, then the output's own rounding
        mag = 1.6 * np.abs(np.where(np.isfinite(l), l, 0)) + 0.5 * length + 1 + 6
        tol = 6 * ref.U24 * mag + ref.HALF_STEP[out_kind] * np.abs(np.where(fine, expect, 0))
        changed = np.abs(np.where(fine, got - np.where(fine, expect, 0), 0)) > tol
        assert not changed.any(), (use, np.argwhere(changed)[:4])
        if in_kind == out_kind:  # in place, and entries that nothing adjusts keep their bits
            dbs.dbs_logits_adjust(x, x, **{k: full[k] for k in use})
            np.testing.assert_array_equal(host(x), host(out))
            if not use:
                np.testing.assert_array_equal(host(out), l)


def test_logits_rows_with_strides_and_bad_lists_stay_in_bounds(dbs):
    import torch

    rng = np.random.default_rng(50)
    l = rng.normal(0, 3, (3, 70)).astype(np.float32)
    big = torch.full((3, 101), 5.0, device="cuda")
    big[:, 3:73] = cuda(l)
    out = torch.full((3, 90), 9.0, device="cuda")
    # pointers outside the list are clamped to it: row 0 takes all entries, row 1 none, row 2 none
    hp = np.array([-5, 1000, 1000, -7], np.int32)
    h = np.array([1, 2, 2], np.int32)
    dbs.dbs_logits_adjust(big[:, 3:73], out[:, 1:71], hist_ptr=cuda(hp), hist=cuda(h), frequency=cuda(np.ones(3, np.float32)))
    expect = ref.logits(l, hist=[h, [], []], freq=np.ones(3))
    np.testing.assert_allclose(host(out[:, 1:71]), expect, rtol=1e-6)
    assert (out[:, 0] == 9).all() and (out[:, 71:] == 9).all()


def test_logits_lists_of_extreme_pointers_are_empty(dbs):
    rng = np.random.default_rng(51)
    lo, hi = np.iinfo(np.int32).min, np.iinfo(np.int32).max
    ptr = np.array([hi, lo, lo + 2, hi, hi - 5, 0, lo, 0], np.int32)  # only row 2's part is not empty: all three entries
    l = rng.normal(0, 3, (7, 60)).astype(np.float32)
    ids, ones = np.array([7, 8, 7], np.int32), np.ones(7, np.float32)
    out = empty((7, 60), "f32")
    dbs.dbs_logits_adjust(cuda(l), out, hist_ptr=cuda(ptr), hist=cuda(ids), hist_new=cuda(np.zeros(7, np.int32)),
                          frequency=cuda(ones), bias_ptr=cuda(ptr), bias_idx=cuda(ids), bias_val=cuda(ones[:3]))
    rows = [ids if b == 2 else [] for b in range(7)]
    expect = ref.logits(l, hist=rows, freq=ones, bias=[[(v, 1.0) for v in r] for r in rows])
    # two sums, each rounded on a magnitude below 16
    np.testing.assert_allclose(host(out), expect, rtol=0, atol=2 * 16 * ref.U24)


# --------------------------------------------------------------------------- rope
@pytest.mark.parametrize("x_kind,y_kind", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,heads,dim,rot", [(1, 1, 2, 2), (1, 40, 128, 128), (5, 3, 80, 32), (7, 2, 66, 66), (33, 5, 96, 50), (2, 3, 7, 0), (3, 2, 1100, 1024), (130, 8, 64, 64)])
def test_rope(dbs, tokens, heads, dim, rot, interleaved, x_kind, y_kind):
    rng = np.random.default_rng(tokens * 100 + dim)
    x = rng.standard_normal((tokens, heads, dim)).astype(np.float32)
    x = ref.bf16(x) if x_kind == "bf16" else x
    pos = rng.integers(0, 2_000_000, tokens).astype(np.int32)
    pos[0] = 0
    pos[-1] = 2 ** 31 - 1 if tokens > 1 else 900_001
    freq = 10000.0 ** (-np.arange(rot // 2) / max(1, rot // 2))
    layout = dbs.DBS_ROPE_INTERLEAVED if interleaved else dbs.DBS_ROPE_HALF
    for scale, inverse in ((1.0, False), (1.25, True)):
        y = empty((tokens, heads, dim), y_kind)
        dbs.dbs_rope(cuda(x, x_kind), cuda(pos), cuda(freq), y, layout=layout, scale=scale, inverse=inverse)
        expect = ref.rope(x, pos, freq, interleaved, scale, inverse)
        # the turn's fraction is rounded to fp32 (pi half steps), sine and cosine are within 2 ulp, two products
        # and a sum: 12 half steps of scale (|a| + |b|) <= 2 scale max|x|; 2^31 positions in 64 bits leave 2^-20
        far = 2.0 ** -20 if tokens > 1 else 0.0
        tol = (12 * ref.U24 + far * (pos == 2 ** 31 - 1)[:, None, None]) * 2 * scale * np.abs(x).max() + ref.HALF_STEP[y_kind] * np.abs(expect)
        assert (np.abs(host(y) - expect) <= tol).all()
        np.testing.assert_array_equal(host(y)[..., rot:], rounded(x[..., rot:], y_kind))


@pytest.mark.parametrize("x_kind,y_kind", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,heads,dim,rot", [(9, 3, 96, 24), (4, 5, 20, 12), (600, 2, 12, 6), (3, 7, 64, 18), (5, 1, 36, 2), (2, 9, 24, 0), (520, 3, 40, 38)])
def test_rope_widths(dbs, tokens, heads, dim, rot, interleaved, x_kind, y_kind):
    """Sizes made of units of each width, and units that rot_dim ends in."""
    test_rope(dbs, tokens, heads, dim, rot, interleaved, x_kind, y_kind)


def test_rope_of_more_tokens_than_one_launch_takes(dbs):
    import torch

    tokens = (1 << 31) // 64 + 1000  # workgroups of one wave
    pos = torch.full((tokens,), -1, device="cuda", dtype=torch.int32)
    x = torch.full((tokens, 1, 2), 1.0, device="cuda", dtype=torch.bfloat16)
    out = torch.full_like(x, 7.0)
    live = torch.tensor([0, 1, (1 << 31) // 64 - 2, (1 << 31) // 64 - 1, (1 << 31) // 64, tokens - 1], device="cuda")
    pos[live] = 1
    freq = torch.tensor([np.pi / 2], device="cuda", dtype=torch.float64)  # (1, 1) becomes (-1, 1)
    dbs.dbs_rope(x, pos, freq, out)
    # the sine of half a turn's half in fp32 and two products: far below a step of bf16 at 1
    assert torch.equal(out[live, 0], torch.tensor([[-1.0, 1.0]], device="cuda", dtype=torch.bfloat16).expand(len(live), 2))
    assert int((out != 7).any(-1).sum()) == len(live)


def test_rope_copies_what_stands_beside_infinities(dbs):
    """The elements from rot_dim on are copied, whatever their neighbours hold."""
    import torch

    for kind in ("f32", "bf16"):
        x = torch.full((1, 2, 16), 3.0, device="cuda", dtype=torch.float32 if kind == "f32" else torch.bfloat16)
        x[0, 0, 7::2] = float("inf")
        x[0, 1, 6::2] = float("nan")
        out, want = torch.zeros_like(x), x[..., 6:].clone()
        freq, _ = dbs.dbs_rope_frequencies(6)
        dbs.dbs_rope(x, torch.tensor([5], dtype=torch.int32, device="cuda"), freq.cuda(), out, layout=dbs.DBS_ROPE_INTERLEAVED)
        assert torch.equal(out[..., 6:].nan_to_num(1.0, 2.0), want.nan_to_num(1.0, 2.0)) and torch.isfinite(out[..., :6]).all()


def test_rope_strides_in_place_and_padding(dbs):
    import torch

    rng = np.random.default_rng(60)
    tokens, hq, hk, dim = 6, 4, 2, 64
    qkv = rng.standard_normal((tokens, (hq + 2 * hk) * dim)).astype(np.float32)
    pos = np.array([3, 4, -1, 100000, 0, -7], np.int32)
    freq, scale = dbs.dbs_rope_frequencies(48, 10000.0, dbs.DBS_ROPE_BANDS, 8.0, 1.0, 4.0, 8192)
    t = cuda(qkv)
    heads = t[:, :(hq + hk) * dim].unflatten(1, (hq + hk, dim))
    dbs.dbs_rope(heads, cuda(pos), freq.cuda(), heads, scale=scale)  # queries and keys in place, values left alone
    expect = qkv.astype(np.float64).copy()
    turned = ref.rope(expect[:, :(hq + hk) * dim].reshape(tokens, hq + hk, dim), pos, freq.numpy(), False).reshape(tokens, -1)
    live = pos >= 0
    expect[live, :(hq + hk) * dim] = turned[live]
    assert (np.abs(host(t) - expect) <= 12 * ref.U24 * 2 * np.abs(qkv).max() + ref.U24 * np.abs(expect)).all()
    np.testing.assert_array_equal(host(t)[~live], qkv[~live])
    np.testing.assert_array_equal(host(t)[:, (hq + hk) * dim:], qkv[:, (hq + hk) * dim:])
    # into a cache kept [head][token][dim], keys only
    cache = torch.full((hk, 10, dim), 2.0, device="cuda", dtype=torch.bfloat16)
    keys = cuda(qkv)[:, hq * dim:(hq + hk) * dim].unflatten(1, (hk, dim))
    dbs.dbs_rope(keys, cuda(pos), freq.cuda(), cache.transpose(0, 1)[2:8])
    got = host(cache).transpose(1, 0, 2)
    exp = ref.rope(qkv[:, hq * dim:(hq + hk) * dim].reshape(tokens, hk, dim), pos, freq.numpy(), False)
    assert (np.abs(got[2:8][live] - exp[live]) <= 2.0 ** -8 * np.abs(exp[live]) + 1e-5).all()
    assert (got[2:8][~live] == 2).all() and (got[:2] == 2).all() and (got[8:] == 2).all()


def test_rope_inverse_is_its_gradient(dbs):
    """<dy, R(x + d) - R(x)> = <R^-1 dy, d> (R is linear), against the formula's transpose and differences."""
    rng = np.random.default_rng(61)
    x, d, dy = (rng.standard_normal((9, 2, 32)).astype(np.float32) for _ in range(3))
    pos, freq = rng.integers(0, 5000, 9).astype(np.int32), 10000.0 ** (-np.arange(16) / 16)
    for layout in (dbs.DBS_ROPE_HALF, dbs.DBS_ROPE_INTERLEAVED):
        y0, y1, dx = (empty((9, 2, 32), "f32") for _ in range(3))
        dbs.dbs_rope(cuda(x), cuda(pos), cuda(freq), y0, layout=layout)
        dbs.dbs_rope(cuda(x + d), cuda(pos), cuda(freq), y1, layout=layout)
        dbs.dbs_rope(cuda(dy), cuda(pos), cuda(freq), dx, layout=layout, inverse=True)
        left = np.sum(dy.astype(np.float64) * (host(y1).astype(np.float64) - host(y0)))
        right = np.sum(host(dx).astype(np.float64) * ((x + d).astype(np.float64) - x))
        size = np.sum(np.abs(dy)) * (np.abs(x).max() + np.abs(d).max()) * 2
        assert abs(left - right) <= 4 * 12 * ref.U24 * 2 * size


# --------------------------------------------------------------------------- streams, graphs, a step
def test_calls_on_two_streams_with_one_handle(dbs):
    import torch

    rng = np.random.default_rng(70)
    w = ref.Q4(rng, 700, 900, 64, True)
    A = w.build(dbs)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    xs = [integers(rng, t, 900) for t in (1, 20)]
    ins = [cuda(x) for x in xs]
    outs = [empty((len(x), 700), "f32") for x in xs]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, x, y in zip(streams, ins, outs):
            dbs.dbs_q4_product(A, x, y, stream=s)
    torch.cuda.synchronize()
    for x, y in zip(xs, outs):
        np.testing.assert_array_equal(host(y), (x.astype(np.float64) @ w.w.T).astype(np.float32))


def test_captured_step_replays(dbs):
    """Head product, its adjustment, gate/up and rotation in one graph, replayed on changed inputs between eager
    work, every replay against the eager calls."""
    import torch

    rng = np.random.default_rng(71)
    w, g, u = ref.Q4(rng, 300, 256, 64, True), ref.Q4(rng, 128, 256, 64, True), ref.Q4(rng, 128, 256, 64, True)
    W, G, U = w.build(dbs), g.build(dbs), u.build(dbs)
    x = torch.zeros(3, 256, device="cuda")
    hp, hist = cuda(np.array([0, 2, 4, 9], np.int32)), cuda(rng.integers(0, 300, 9).astype(np.int32))
    rep = cuda(np.array([1.2, 1.0, 1.5], np.float32))
    mask = cuda(ref.mask_words(rng.random((3, 300)) < 0.5))
    pos, freq = cuda(np.array([5, 6, 7], np.int32)), cuda(10000.0 ** (-np.arange(32) / 32))

    def step(out):
        dbs.dbs_q4_gated(G, U, x, dbs.DBS_ACT_SILU, out[0])
        dbs.dbs_rope(x.view(3, 4, 64), pos, freq, out[1])
        dbs.dbs_q4_product_masked(W, x, mask, out[2])
        dbs.dbs_logits_adjust(out[2], out[3], hist_ptr=hp, hist=hist, repetition=rep, mask=mask)

    def buffers():
        return [empty((3, 128), "bf16"), empty((3, 4, 64), "bf16"), empty((3, 300), "f32"), empty((3, 300), "f32")]

    graphed, eager = buffers(), buffers()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(graphed)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(graphed)
    for _ in range(4):
        x.copy_(cuda(integers(rng, 3, 256)))
        for t in graphed:
            t.fill_(4.0)
        graph.replay()
        step(eager)
        torch.cuda.synchronize()
        for a, b in zip(graphed, eager):
            np.testing.assert_array_equal(host(a), host(b))


def test_decode_step(dbs):
    """One token through a layer and the head as a program runs it: stacked 4-bit Q/K/V, rotation in place, gate
    and up in 4 bits, the sparse down layer on the thresholded activation, masked head, logits. Each stage
    against its 64-bit reference on the inputs it really got."""
    import torch

    from gpu_helpers import build, csr_of

    rng = np.random.default_rng(72)
    d, ff, vocab, hq, hk, dim = 256, 640, 1000, 4, 2, 64
    qkv, gate, up, head = (ref.Q4(rng, m, d, 64, True, exact=False) for m in ((hq + 2 * hk) * dim, ff, ff, vocab))
    QKV, G, U, H = (w.build(dbs) for w in (qkv, gate, up, head))
    down = np.where(rng.random((d, ff)) < 0.5, rng.normal(0, 0.05, (d, ff)), 0).astype(np.float32)
    D = build(dbs, d, ff, *csr_of(down), dbs.DBS_F32)
    x = cuda(rng.standard_normal((1, d)).astype(np.float32), "bf16")
    x64 = host(x).astype(np.float64)
    y = empty((1, (hq + 2 * hk) * dim), "f32")
    dbs.dbs_q4_product(QKV, x, y)
    before = host(y).astype(np.float64)
    assert (np.abs(before - x64 @ qkv.w.T) <= qkv.bound(x64)).all()
    freq, scale = dbs.dbs_rope_frequencies(dim)
    heads = y[:, :(hq + hk) * dim].unflatten(1, (hq + hk, dim))
    dbs.dbs_rope(heads, cuda(np.array([777], np.int32)), freq.cuda(), heads, scale=scale)
    expect = ref.rope(before[:, :(hq + hk) * dim].reshape(1, hq + hk, dim), [777], freq.numpy(), False)
    assert (np.abs(host(heads) - expect) <= 14 * ref.U24 * 2 * np.abs(before).max()).all()
    h = empty((1, ff), "f32")
    dbs.dbs_q4_gated(G, U, x, dbs.DBS_ACT_RELU, h)
    threshold = 0.05
    out = torch.empty(d, device="cuda")
    dbs.dbs_spmspv_dense_threshold(D, h[0], threshold, dbs.DBS_PLUS_TIMES, out)
    h64 = host(h)[0].astype(np.float64)
    kept = np.where(np.abs(h64) > np.float32(threshold), h64, 0)
    assert (np.abs(host(out) - down.astype(np.float64) @ kept) <= 1e-5 * (np.abs(down.astype(np.float64)) @ np.abs(kept)) + 1e-6).all()
    allowed = rng.random((1, vocab)) < 0.1
    logit = empty((1, vocab), "f32")
    dbs.dbs_q4_product_masked(H, out, cuda(ref.mask_words(allowed)), logit[0])
    o64 = host(out)[None].astype(np.float64)
    assert (np.abs(np.where(allowed, host(logit) - o64 @ head.w.T, 0)) <= head.bound(o64)).all()
    raw = host(logit).astype(np.float64)
    hist = [[int(v) for v in np.argwhere(allowed[0])[:5, 0]]]
    dbs.dbs_logits_adjust(logit, logit, hist_ptr=cuda(np.array([0, 5], np.int32)), hist=cuda(np.array(hist[0], np.int32)), repetition=cuda(np.array([1.3], np.float32)))
    want = ref.logits(raw, hist=hist, rep=[np.float32(1.3)])
    same_kind(host(logit), want)
    fine = np.isfinite(want)
    assert (np.abs(host(logit)[fine] - want[fine]) <= 4 * ref.U24 * np.abs(raw[fine]) * 1.3).all()


# --------------------------------------------------------------------------- refusals by the binding
def test_choices_past_32_bits_are_refused(dbs):
    import torch

    A = ref.Q4(np.random.default_rng(81), 20, 64, 32, False).build(dbs)
    x, y = torch.zeros(3, 64, device="cuda"), torch.full((3, 20), 5.0, device="cuda")
    pos, freq = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.float64, device="cuda")
    with pytest.raises(ValueError):
        dbs.dbs_q4_gated(A, A, x, 1 << 32, y)
    with pytest.raises(ValueError):
        dbs.dbs_rope(x[:, None], pos, freq, x[:, None], layout=1 << 32)
    torch.cuda.synchronize()
    assert (y == 5).all()


@pytest.mark.parametrize("x_kind", ["bf16", "f32"])
def test_largest_calls(dbs, x_kind):
    import torch

    rng = np.random.default_rng(83)
    w = ref.Q4(rng, 20, 130, 64, True)
    A, w64 = w.build(dbs), torch.from_numpy(w.w).cuda().t()
    tokens = dbs.DBS_Q4_MAX_TOKENS
    x = torch.randint(-4, 5, (tokens + 1, 130), device="cuda").to(torch.bfloat16 if x_kind == "bf16" else torch.float32)
    y = torch.zeros(tokens + 1, 20, device="cuda")
    dbs.dbs_q4_product(A, x[:tokens], y[:tokens])
    assert torch.equal(y[:tokens].double(), x[:tokens].double() @ w64) and (y[tokens] == 0).all()
    with pytest.raises(dbs.DBSError):
        dbs.dbs_q4_product(A, x, y)


@pytest.mark.parametrize("x_kind", ["bf16", "f32"])
def test_product_of_very_long_rows(dbs, x_kind):
    """A million columns and some, of which x has a few hundred: the sums stay exact."""
    import torch

    rng = np.random.default_rng(84)
    n = (1 << 20) + 77
    w = ref.Q4(rng, 35, n, 128, True)
    A, w64 = w.build(dbs), torch.from_numpy(w.w).cuda().t()
    for t in (1, 6, 20):
        x = np.zeros((t, n), np.float32)
        for row in x:
            row[rng.integers(0, n, 300)] = rng.integers(1, 5, 300)
            row[-3:] = 2
        x = cuda(x, x_kind)
        y = empty((t, 35), "f32")
        dbs.dbs_q4_product(A, x, y)
        assert torch.equal(y.double(), x.double() @ w64), f"{t} tokens"


def test_logits_of_the_most_rows(dbs):
    import torch

    rows = dbs.DBS_LOGITS_MAX_ROWS
    x = torch.zeros(rows + 1, 37, device="cuda")
    out = torch.full((rows + 1, 37), 5.0, device="cuda")
    ptr = torch.arange(rows + 1, dtype=torch.int32, device="cuda")
    ids = (torch.arange(rows, device="cuda") % 37).int()
    dbs.dbs_logits_adjust(x[:rows], out[:rows], hist_ptr=ptr, hist=ids, frequency=torch.ones(rows, device="cuda"))
    expect = torch.zeros(rows, 37, device="cuda")
    expect[torch.arange(rows, device="cuda"), ids.long()] = -1.0
    assert torch.equal(out[:rows], expect) and (out[rows] == 5).all()
    with pytest.raises(dbs.DBSError):
        dbs.dbs_logits_adjust(x, out)


def test_streams_of_another_device_are_refused(dbs):
    import torch

    class Stream:
        cuda_stream = 0

        def __init__(self, device_index):
            self.device_index = device_index

    x, y = torch.ones(2, 64, device="cuda"), torch.full((2, 64), 5.0, device="cuda")
    with pytest.raises(ValueError, match="stream"):
        dbs.dbs_logits_adjust(x, y, stream=Stream(torch.cuda.current_device() + 1))
    torch.cuda.synchronize()
    assert (y == 5).all()
    dbs.dbs_logits_adjust(x, y, stream=torch.cuda.default_stream())
    torch.cuda.synchronize()
    assert (y == 1).all()


def test_calls_of_two_threads_on_their_own_streams(dbs):
    import threading

    import torch

    rng = np.random.default_rng(82)
    w = ref.Q4(rng, 500, 700, 64, True)
    A = w.build(dbs)
    xs = [integers(rng, t, 700) for t in (1, 20)]
    ins, outs, errors = [cuda(x) for x in xs], [empty((len(x), 500), "f32") for x in xs], []
    torch.cuda.synchronize()

    def work(x, y):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(200):
                    dbs.dbs_q4_product(A, x, y)
                torch.cuda.current_stream().synchronize()
        except Exception as e:
            errors.append(e)

    threads = [threading.Thread(target=work, args=a) for a in zip(ins, outs)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not errors and not any(t.is_alive() for t in threads)
    for x, y in zip(xs, outs):
        np.testing.assert_array_equal(host(y), (x.astype(np.float64) @ w.w.T).astype(np.float32))


def test_refusals_of_tensors(dbs):
    import torch

    rng = np.random.default_rng(80)
    A, B = ref.Q4(rng, 20, 64, 32, False).build(dbs), ref.Q4(rng, 20, 64, 64, False).build(dbs)
    x, y = torch.zeros(3, 64, device="cuda"), torch.full((3, 20), 5.0, device="cuda")
    z = torch.zeros(3, 128, device="cuda")
    for error, call in (
            (ValueError, lambda: dbs.dbs_q4_product(A, x[:2], y)),
            (ValueError, lambda: dbs.dbs_q4_product(A, x[:, :63], y)),
            (ValueError, lambda: dbs.dbs_q4_product(A, z[:, ::2], y)),
            (ValueError, lambda: dbs.dbs_q4_product(A, x[:1].expand(3, 64), y)),
            (ValueError, lambda: dbs.dbs_q4_product(A, x[None], y)),
            (TypeError, lambda: dbs.dbs_q4_product(A, x.half(), y)),
            (TypeError, lambda: dbs.dbs_q4_product(A, x.cpu(), y)),
            (TypeError, lambda: dbs.dbs_q4_product(A, x, None)),
            (AttributeError, lambda: dbs.dbs_q4_product(A, x, y, stream=5)),
            (dbs.DBSError, lambda: dbs.dbs_q4_product(A, z.view(-1)[:64], z.view(-1)[60:80])),  # overlapping
            (dbs.DBSError, lambda: dbs.dbs_q4_gated(A, B, x, dbs.DBS_ACT_RELU, y)),  # two group sizes
            (dbs.DBSError, lambda: dbs.dbs_q4_gated(A, A, x, 3, y)),
            (ValueError, lambda: dbs.dbs_q4_product_masked(A, x, torch.zeros(3, 2, dtype=torch.int32, device="cuda"), y)),
            (TypeError, lambda: dbs.dbs_q4_product_masked(A, x, torch.zeros(3, 1, dtype=torch.int64, device="cuda"), y)),
            (ValueError, lambda: dbs.dbs_logits_adjust(y, y, hist=torch.zeros(2, dtype=torch.int32, device="cuda"))),
            (ValueError, lambda: dbs.dbs_logits_adjust(y, x[:, :20][:2])),
            (TypeError, lambda: dbs.dbs_logits_adjust(y, y, repetition=torch.zeros(3, dtype=torch.float64, device="cuda"))),
            (dbs.DBSError, lambda: dbs.dbs_logits_adjust(y, y, repetition=torch.ones(3, device="cuda"))),  # of no history
            (dbs.DBSError, lambda: dbs.dbs_q4_product(A, x, x[:, :20])),  # into x
            (ValueError, lambda: dbs.dbs_rope(x, x, x, x)),
            (TypeError, lambda: dbs.dbs_rope(x[:, None], torch.zeros(3, dtype=torch.int64, device="cuda"), torch.zeros(2, dtype=torch.float64, device="cuda"), x[:, None])),
            (dbs.DBSError, lambda: dbs.dbs_rope(x[:, None], torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(33, dtype=torch.float64, device="cuda"), x[:, None])),
            (ValueError, lambda: dbs.dbs_q4_build(20, 64, 48, torch.zeros(20, 32, dtype=torch.uint8, device="cuda"), x[:, :2])),
            (dbs.DBSError, lambda: dbs.dbs_q4_build(3, 64, 64, torch.zeros(3, 32, dtype=torch.uint8, device="cuda"), torch.ones(3, 1, device="cuda"), torch.full((3, 1), 16, dtype=torch.uint8, device="cuda")))):
        with pytest.raises(error):
            call()
    dbs.dbs_q4_free(A)
    with pytest.raises(dbs.DBSError):
        dbs.dbs_q4_product(A, x, y)  # a freed matrix
    torch.cuda.synchronize()
    assert (y == 5).all() and (x == 0).all()
