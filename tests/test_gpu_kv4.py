"""The cache of 4-bit keys and values and the attention over it against 64-bit references, on the GPU."""
import numpy as np
import pytest

import kv4_ref as ref

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


def on_gpu(dbs, c):
    return dbs.dbs_kv4_cache(c.pages, c.heads, c.dim, c.group, c.page, pool=cuda(c.bytes))


def tables(rng, lengths, page, extra=0, spare=2):
    """A table of distinct random pages for sequences of these lengths, -1 behind them, and how many pages there are."""
    need = [-(-n // page) for n in lengths]
    width = max(1, max(need) + extra)
    pages = sum(need) + spare
    ids = rng.permutation(pages)
    table, at = np.full((len(lengths), width), -1, np.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at : at + n]
        at += n
    return table, pages


# head_dim, group: every padded size and every number of groups of it, cut heads
SHAPES = [(64, 32), (64, 64), (96, 32), (128, 32), (128, 64), (128, 128), (192, 32), (192, 64), (256, 32), (256, 64), (256, 128),
          (8, 32), (40, 64), (80, 32), (72, 32), (104, 128), (136, 64), (160, 32), (200, 128)]


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("dim,group", SHAPES)
def test_store_writes_the_bytes_of_the_definition(dbs, dim, group, kind):
    """Every byte of the pool, those that no new token owns included, and what the cache stands for."""
    rng = np.random.default_rng(dim * 1000 + group)
    heads, page = 2, 16 if dim % 3 else 32
    lengths, new = [1, 23, 40, 0, 17], [1, 7, 40, 0, 9]
    table, pages = tables(rng, lengths, page, extra=1)
    c = ref.Cache(pages, heads, dim, group, page)
    c.bytes[:] = rng.integers(0, 256, c.bytes.shape)
    cache = on_gpu(dbs, c)
    total = sum(new)
    k, v = (ref.typed(rng.normal(0, 1 + rng.uniform(0, 30, (total, heads, 1)), (total, heads, dim)), kind) for _ in range(2))
    k[0] = 2.5  # one value throughout: a scale of 0
    v[3, 1] = ref.typed(v[3, 1] * 1e-7, kind)
    ptr = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
    want_k, want_v = np.zeros(k.shape), np.zeros(v.shape)
    for b, (n, m) in enumerate(zip(lengths, new)):
        for i in range(m):
            t = n - m + i
            for h in range(heads):
                want_k[ptr[b] + i, h], want_v[ptr[b] + i, h] = c.store(table[b, t // page], t % page, h, k[ptr[b] + i, h], v[ptr[b] + i, h])
    for out_kind in ("bf16", "f32"):
        ko, vo = empty(k.shape, out_kind), empty(v.shape, out_kind)
        dbs.dbs_kv4_store(cache, cuda(table), cuda(np.array(lengths, np.int32)), cuda(k, kind), cuda(v, kind), new_ptr=cuda(ptr), k_out=ko, v_out=vo)
        np.testing.assert_array_equal(cache.pool.cpu().numpy(), c.bytes)
        np.testing.assert_array_equal(host(ko), ref.typed(want_k, out_kind))
        np.testing.assert_array_equal(host(vo), ref.typed(want_v, out_kind))


def test_store_token_by_token_is_store_at_once(dbs):
    """A prompt in one call, in pieces and token by token leaves the same bytes; without outputs, and in place."""
    rng = np.random.default_rng(5)
    heads, dim, group, page, n = 3, 128, 64, 16, 75
    table, pages = tables(rng, [n, n], page)
    k, v = (ref.typed(rng.normal(0, 2, (2 * n, heads, dim)), "bf16") for _ in range(2))
    start = rng.integers(0, 256, (pages, ref.Cache(1, heads, dim, group, page).head_bytes * heads)).astype(np.uint8)

    def run(cuts, in_place):
        cache = dbs.dbs_kv4_cache(pages, heads, dim, group, page, pool=cuda(start))
        for a, b in zip(cuts[:-1], cuts[1:]):
            rows = np.concatenate((np.arange(a, b), n + np.arange(a, b)))
            kk, vv = cuda(k[rows], "bf16"), cuda(v[rows], "bf16")
            dbs.dbs_kv4_store(cache, cuda(table), cuda(np.full(2, b, np.int32)), kk, vv, **(dict(k_out=kk, v_out=vv) if in_place else {}))
        return cache.pool.cpu().numpy()

    once = run([0, n], False)
    np.testing.assert_array_equal(run([0, 3, 8, 24, 25, 64, n], True), once)
    np.testing.assert_array_equal(run(list(range(n + 1)), False), once)


def test_store_of_values_that_are_not_finite(dbs):
    """A group with one is NaN; its neighbours are not touched by that."""
    rng = np.random.default_rng(6)
    c = ref.Cache(1, 1, 128, 32, 16)
    k = rng.normal(0, 1, (5, 1, 128)).astype(np.float32)
    v = k.copy()
    k[0, 0, 3], k[1, 0, 40], k[2, 0, 127], k[3, 0, 64], k[4, 0, 0] = np.nan, np.inf, -np.inf, 65025, -65024
    v[0, 0, 100], v[2, 0, 32] = -np.nan, 1e30
    cache = on_gpu(dbs, c)
    ko, vo = empty(k.shape, "f32"), empty(k.shape, "f32")
    dbs.dbs_kv4_store(cache, cuda(np.zeros((1, 1), np.int32)), cuda(np.array([5], np.int32)), cuda(k), cuda(v), k_out=ko, v_out=vo)
    for x, got in ((k, host(ko)), (v, host(vo))):
        want = np.array([c.value(*c.quantize(x[i, 0])) for i in range(5)])
        assert np.isnan(want).any()
        np.testing.assert_array_equal(got[:, 0], want.astype(np.float32))


def test_store_drops_what_has_no_page(dbs):
    """Entries outside the pool, tokens before the first and behind the table are stored nowhere, and returned all the same."""
    rng = np.random.default_rng(7)
    heads, dim, page = 2, 64, 16
    c = ref.Cache(3, heads, dim, 32, page, fill=0xA5)
    table = np.array([[0, -1, 1], [7, 3, -(1 << 31)], [2, 2, 2]], np.int32)
    lengths, n = np.array([45, 40, 5], np.int32), 40
    k, v = (rng.normal(0, 1, (3 * n, heads, dim)).astype(np.float32) for _ in range(2))
    for b in range(3):
        for i in range(n):
            t = lengths[b] - n + i
            if t >= 0 and 0 <= table[b, t // page] < 3:
                for h in range(heads):
                    c.store(table[b, t // page], t % page, h, k[b * n + i, h], v[b * n + i, h])
    cache = dbs.dbs_kv4_cache(3, heads, dim, 32, page, pool=cuda(np.full(c.bytes.shape, 0xA5, np.uint8)))
    ko = empty(k.shape, "f32")
    dbs.dbs_kv4_store(cache, cuda(table), cuda(lengths), cuda(k), cuda(v), k_out=ko)
    np.testing.assert_array_equal(cache.pool.cpu().numpy(), c.bytes)
    np.testing.assert_array_equal(host(ko)[:, 0], np.array([c.value(*c.quantize(x)) for x in k[:, 0]]).astype(np.float32))


def check(dbs, c, table, lengths, new, q, kind, out_kind, window=0, sinks=0, ragged=None, max_len=0, **more):
    """The call against the reference; the rows behind the last sequence keep what they held."""
    heads = q.shape[1]
    rep = heads // c.heads
    ptr = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
    ragged = len(set(new)) > 1 if ragged is None else ragged
    cache = on_gpu(dbs, c)
    out = empty(q.shape, out_kind)
    dbs.dbs_kv4_attention(cache, cuda(table), cuda(np.array(lengths, np.int32)), cuda(q, kind), out,
                          new_ptr=cuda(ptr) if ragged else None, window=window, sinks=sinks, max_len=max_len, **more)
    got = host(out).astype(np.float64)
    scale = 1 / np.sqrt(c.dim)
    wide = "f32" in (kind, out_kind)
    for b, (n, m) in enumerate(zip(lengths, new)):
        k, v = ref.sequence_values(c, table[b], n)
        has = ~np.isnan(k[0, :, 0]) if n else None
        for i in range(m):
            for h in range(heads):
                want, mass, size = ref.attention(q[ptr[b] + i, h].astype(np.float64), k[h // rep], v[h // rep], n - m + i, scale, window, sinks, has)
                tol = ref.attention_tolerance(want, mass, size, c.dim, n, out_kind, wide)
                off = np.abs(got[ptr[b] + i, h] - want)
                assert (off <= tol).all(), f"sequence {b}, token {i}, head {h}: off {off.max():.3g}, {(off / tol).max():.3g} of the tolerance"
    assert (got[ptr[-1] :] == 7.0).all()
    return out


TYPES = [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")]


@pytest.mark.parametrize("kind,out_kind", TYPES)
@pytest.mark.parametrize("dim,group", SHAPES)
def test_attention_of_every_shape(dbs, dim, group, kind, out_kind):
    """One token, drafts and a short prompt of every head size; pages of each size in turn."""
    rng = np.random.default_rng(dim * 31 + group)
    page = (16, 32, 64, 128, 256)[(dim // 8 + group // 32) % 5]
    lengths = [1, 37, 130, 0]
    table, pages = tables(rng, lengths, page)
    for kv_heads, rep, new in ((1, 1, [1, 1, 1, 1]), (2, 3, [1, 5, 2, 0]), (1, 4, [1, 37, 40, 0])):
        c = ref.Cache(pages, kv_heads, dim, group, page)
        ref.random_bytes(rng, c)
        q = ref.typed(rng.normal(0, 1, (sum(new) + 2, kv_heads * rep, dim)), kind)
        if len(set(new)) == 1:
            q = q[: sum(new)]
        check(dbs, c, table, lengths, new, q, kind, out_kind)


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 1), (7, 4), (32, 33), (64, 16), (100, 3), (1000, 4), (5, 1000)])
@pytest.mark.parametrize("rep,new", [(4, [1, 1, 1]), (7, [3, 6, 1]), (1, [50, 150, 70]), (8, [30, 64, 33])])
def test_attention_windows(dbs, window, sinks, rep, new):
    rng = np.random.default_rng(window * 7 + sinks + rep)
    lengths = [50, 301, 133]
    table, pages = tables(rng, lengths, 16)
    c = ref.Cache(pages, 1, 64, 32, 16)
    ref.random_bytes(rng, c)
    q = ref.typed(rng.normal(0, 1, (sum(new), rep, 64)), "bf16")
    check(dbs, c, table, lengths, new, q, "bf16", "bf16", window, sinks)


@pytest.mark.parametrize("rep,each", [(1, 1), (16, 1), (17, 1), (3, 11), (5, 13), (1, 64), (4, 16), (9, 9), (1, 129), (2, 130), (8, 40)])
def test_attention_is_exact_on_means(dbs, rep, each):
    """Queries of zero: each row is the mean of the integers that it sees; a wrong token, row or channel shows."""
    import torch

    rng = np.random.default_rng(rep * 100 + each)
    heads, dim, page, lengths = 2, 96, 32, [each, 333, each + 70]
    table, pages = tables(rng, lengths, page)
    c = ref.Cache(pages, heads, dim, 32, page)
    k = rng.normal(0, 1, (sum(lengths), heads, dim)).astype(np.float32)
    v = rng.integers(0, 16, (sum(lengths), heads, dim)).astype(np.float32) - 8
    v[..., 0::32], v[..., 1::32] = -8, 7  # every group holds both ends: s = 1, b = -8
    ptr = np.concatenate(([0], np.cumsum(lengths))).astype(np.int32)
    cache = on_gpu(dbs, c)
    dbs.dbs_kv4_store(cache, cuda(table), cuda(np.array(lengths, np.int32)), cuda(k), cuda(v), new_ptr=cuda(ptr))
    for kind in ("bf16", "f32"):
        q = torch.zeros(3 * each, heads * rep, dim, device="cuda", dtype=torch.bfloat16 if kind == "bf16" else torch.float32)
        for window, sinks in ((0, 0), (40, 5)):
            out = empty(q.shape, "f32")
            dbs.dbs_kv4_attention(cache, cuda(table), cuda(np.array(lengths, np.int32)), q, out, window=window, sinks=sinks)
            got = host(out)
            for b, n in enumerate(lengths):
                for i in range(each):
                    see = ref.visible(n - each + i, n, window, sinks)
                    want = v[ptr[b] : ptr[b + 1]][see].astype(np.float64).mean(0)
                    # sums of integers times 2^6 are exact; the reciprocal and the product round once each
                    for h in range(heads * rep):
                        np.testing.assert_allclose(got[b * each + i, h], want[h // rep], rtol=2.0 ** -22, atol=0)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("dim,group", [(64, 32), (80, 32), (128, 128), (256, 64)])
def test_attention_finds_single_tokens(dbs, dim, group, kind):
    """A query along one key that is far above all others in its score returns that token's value exactly: every channel of every key
    takes its place in the products."""
    rng = np.random.default_rng(dim)
    n, page = 200, 64
    table, pages = tables(rng, [n], page)
    c = ref.Cache(pages, 1, dim, group, page)
    k = np.zeros((n, 1, dim), np.float32)
    # binary words that differ from each other in many places: +-1 in every group
    while True:
        k[:, 0] = rng.integers(0, 2, (n, dim)) * 2 - 1
        k[:, 0, 0::group], k[:, 0, 1::group] = -1, 1
        gram = k[:, 0] @ k[:, 0].T
        if np.sort(gram, 1)[:, -2].max() < dim - 8:
            break
    v = rng.normal(0, 1, (n, 1, dim)).astype(np.float32)
    cache = on_gpu(dbs, c)
    vo = empty(v.shape, "f32")
    lens = cuda(np.array([n], np.int32))
    dbs.dbs_kv4_store(cache, cuda(table), lens, cuda(k), cuda(v), v_out=vo)
    ids = rng.integers(0, n - 60, (60, 3))
    q = 64 * k[ids, 0]
    out = empty(q.shape, "f32")
    dbs.dbs_kv4_attention(cache, cuda(table), lens, cuda(q, kind), out, scale=1.0)  # the others are 8 * 64 and more below
    # +-1 are s q + b with s = half(2/15): off by 2^-11 of it, the same for all; the value passes as a half, whole
    np.testing.assert_array_equal(host(out), host(vo)[ids, 0])


def test_attention_over_many_splits(dbs):
    """A long sequence beside short ones: the work is cut along the tokens, with a workspace, with a smaller one, without, and with a
    bound of the lengths that is wrong."""
    import torch

    rng = np.random.default_rng(11)
    lengths, rep, page = [5000, 3, 700, 0], 4, 64
    table, pages = tables(rng, lengths, page, extra=3)
    c = ref.Cache(pages, 2, 128, 128, page)
    ref.random_bytes(rng, c)
    for new in ([1, 1, 1, 1], [3, 1, 2, 0]):
        q = ref.typed(rng.normal(0, 2, (sum(new), 2 * rep, 128)), "bf16")
        first = check(dbs, c, table, lengths, new, q, "bf16", "f32")
        assert torch.equal(check(dbs, c, table, lengths, new, q, "bf16", "f32"), first)
        check(dbs, c, table, lengths, new, q, "bf16", "f32", max_len=64)
        check(dbs, c, table, lengths, new, q, "bf16", "f32", max_len=700)
        check(dbs, c, table, lengths, new, q, "bf16", "f32", workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
        check(dbs, c, table, lengths, new, q, "bf16", "f32", window=2000, sinks=40)


def test_attention_never_looks_at_freed_pages(dbs):
    """Entries of pages that no new token sees may hold anything; a page that is seen and not there is seen by nobody."""
    rng = np.random.default_rng(12)
    lengths, page = [400, 400], 16
    table, pages = tables(rng, lengths, page)
    c = ref.Cache(pages, 2, 64, 64, page)
    ref.random_bytes(rng, c)
    q = ref.typed(rng.normal(0, 1, (2, 8, 64)), "bf16")
    window, sinks = 100, 3
    freed = table.copy()
    freed[:, 1 : (400 - 100) // 16] = [[1 << 30], [-5]]
    check(dbs, c, freed, lengths, [1, 1], q, "bf16", "bf16", window, sinks)
    freed[0, 22] = pages  # one page inside the window
    freed[1, 0] = -1      # the first tokens
    check(dbs, c, freed, lengths, [1, 1], q, "bf16", "bf16", window, sinks)
    check(dbs, c, np.full_like(table, -1), lengths, [1, 1], q, "bf16", "bf16")


@pytest.mark.parametrize("kind,out_kind", TYPES)
def test_what_is_not_seen_takes_no_part(dbs, kind, out_kind):
    """NaN and infinite records in tokens behind a row, before its window and behind the length; those that are seen make
    their group of channels NaN in the rows that see them, and no others."""
    rng = np.random.default_rng(13)
    dim, group, page, n, each = 128, 32, 32, 150, 40
    table, pages = tables(rng, [n], page)
    c = ref.Cache(pages, 1, dim, group, page)
    ref.random_bytes(rng, c)
    window, sinks = 30, 2
    bad = {20: 0x7C00, 60: 0x7E00, 95: 0xFE00, 119: 0x7E00, 130: 0xFC00, 149: 0x7E00}  # token: bits of its value records

    def spoil(t, bits, values):
        page_bytes = c.bytes[table[0, t // page]]
        at, step = c.value_record(t % page) if values else c.key_record(t % page)
        for o in (0, step):
            page_bytes[at[1] + o : at[1] + o + 2] = np.frombuffer(np.uint16(bits).tobytes(), np.uint8)

    for t, bits in bad.items():
        spoil(t, bits, True)
    for t in range(n, len(table[0]) * page):  # behind the length
        spoil(t, 0x7E00, True)
        spoil(t, 0x7E00, False)
    q = ref.typed(rng.normal(0, 1, (each, 2, dim)), kind)
    cache = on_gpu(dbs, c)
    out = empty(q.shape, out_kind)
    dbs.dbs_kv4_attention(cache, cuda(table), cuda(np.array([n], np.int32)), cuda(q, kind), out, window=window, sinks=sinks)
    got = host(out)
    k, v = ref.sequence_values(c, table[0], n)
    clean = np.where(np.isfinite(v), v, 0.0)
    for i in range(each):
        position = n - each + i
        see = ref.visible(position, n, window, sinks)
        nan = any(see[t] for t in bad)
        for h in range(2):
            want, mass, size = ref.attention(q[i, h].astype(np.float64), k[0], clean[0], position, 1 / np.sqrt(dim), window, sinks)
            tol = ref.attention_tolerance(want, mass, size, dim, n, out_kind, "f32" in (kind, out_kind))
            spoiled = np.zeros(dim, bool)
            spoiled[group : 2 * group] = nan
            np.testing.assert_array_equal(np.isnan(got[i, h]), spoiled, err_msg=f"token {i}")
            assert (np.abs(got[i, h] - want) <= tol)[~spoiled].all(), f"token {i}"
    # keys that are not seen
    for t in (0, 50, 110):
        spoil(t, 0x7E00, False)
    cache = on_gpu(dbs, c)
    again = empty(q.shape, out_kind)
    dbs.dbs_kv4_attention(cache, cuda(table), cuda(np.array([n], np.int32)), cuda(q, kind), again, window=window, sinks=0)
    got = host(again)
    for i in range(each):
        see = ref.visible(n - each + i, n, window, 0)
        assert np.isnan(got[i, :, :group]).all() == bool(see[50] or see[110]), f"token {i}"


def test_queries_that_are_not_finite_stay_in_their_rows(dbs):
    rng = np.random.default_rng(14)
    n, each, dim = 77, 30, 64
    table, pages = tables(rng, [n], 16)
    c = ref.Cache(pages, 1, dim, 32, 16)
    ref.random_bytes(rng, c)
    q = rng.normal(0, 1, (each, 3, dim)).astype(np.float32)
    wrong = q.copy()
    wrong[4, 1, 9], wrong[20, 0, 63], wrong[29, 2, 0] = np.nan, np.inf, -np.inf
    got, fine = empty(q.shape, "f32"), empty(q.shape, "f32")
    cache, args = on_gpu(dbs, c), (cuda(table), cuda(np.array([n], np.int32)))
    dbs.dbs_kv4_attention(cache, *args, cuda(q), fine)
    dbs.dbs_kv4_attention(cache, *args, cuda(wrong), got)
    got, fine = host(got), host(fine)
    for i, h in ((4, 1), (20, 0), (29, 2)):
        assert np.isnan(got[i, h]).all()
        got[i, h] = fine[i, h]
    np.testing.assert_array_equal(got, fine)


@pytest.mark.parametrize("size", [1e-30, 1e-3, 3e4, 1e30])
def test_queries_of_any_size(dbs, size):
    """q is scaled by a power of two on its way to a half, and the scores back."""
    rng = np.random.default_rng(15)
    n, dim = 70, 128
    table, pages = tables(rng, [n], 64)
    c = ref.Cache(pages, 1, dim, 128, 64)
    ref.random_bytes(rng, c)
    cache, args = on_gpu(dbs, c), (cuda(table), cuda(np.array([n], np.int32)))
    q = rng.normal(0, 1, (6, 2, dim)).astype(np.float32)
    big = (q.astype(np.float64) * size).astype(np.float32)
    out = empty(q.shape, "f32")
    dbs.dbs_kv4_attention(cache, *args, cuda(big), out, scale=float(np.float32(0.1 / size)))
    k, v = ref.sequence_values(c, table[0], n)
    for i in range(6):
        for h in range(2):
            want, mass, sz = ref.attention(big[i, h].astype(np.float64), k[0], v[0], n - 6 + i, float(np.float32(0.1 / size)))
            tol = ref.attention_tolerance(want, mass, sz, dim, n, "f32", True)
            assert (np.abs(host(out)[i, h] - want) <= tol).all()


def test_strides_offsets_and_a_larger_pool(dbs):
    """q as part of a fused projection's rows, heads before tokens, rows at odd elements, layers' pages side by side."""
    import torch

    rng = np.random.default_rng(16)
    lengths, new, heads, dim, page = [90, 33], [4, 9], 6, 128, 16
    table, pages = tables(rng, lengths, page)
    c = ref.Cache(pages, 3, dim, 64, page)
    ref.random_bytes(rng, c)
    lens, ptr = cuda(np.array(lengths, np.int32)), cuda(np.array([0, 4, 13], np.int32))
    q = ref.typed(rng.normal(0, 1, (13, heads, dim)), "bf16")
    plain = empty(q.shape, "bf16")
    dbs.dbs_kv4_attention(on_gpu(dbs, c), cuda(table), lens, cuda(q, "bf16"), plain, new_ptr=ptr)
    size = c.bytes.shape[1]
    layers = torch.full((pages, 3, size), 0xFF, dtype=torch.uint8, device="cuda")
    layers[:, 1] = cuda(c.bytes)
    cache = dbs.dbs_kv4_cache(pages, 3, dim, 64, page, pool=layers[:, 1])
    wide_table = torch.full((2, table.shape[1] + 5), -7, dtype=torch.int32, device="cuda")
    wide_table[:, 2 : 2 + table.shape[1]] = cuda(table)
    row = torch.zeros(13, 2 * heads + 3, dim, dtype=torch.bfloat16, device="cuda")
    row[:, 3 : 3 + heads] = cuda(q, "bf16")
    flat = torch.zeros(13 * heads * dim + 3, dtype=torch.bfloat16, device="cuda")
    odd = flat[3:].view(13, heads, dim)
    odd.copy_(cuda(q, "bf16"))
    turned = cuda(q, "bf16").transpose(0, 1).contiguous().transpose(0, 1)
    for x in (row[:, 3 : 3 + heads], odd, turned):
        for out in (empty(q.shape, "bf16"), torch.full((13, 20, dim), 7.0, dtype=torch.bfloat16, device="cuda")[:, 5 : 5 + heads],
                    torch.full((heads, 13, dim + 5), 7.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)[..., 5:]):
            dbs.dbs_kv4_attention(cache, wide_table[:, 2 : 2 + table.shape[1]], lens, x, out, new_ptr=ptr)
            assert torch.equal(out, plain)
    kv = ref.typed(rng.normal(0, 1, (13, 6, dim)), "bf16")
    whole, parts = dbs.dbs_kv4_cache(pages, 3, dim, 64, page, pool=cuda(c.bytes)), cache
    both = cuda(kv, "bf16")
    dbs.dbs_kv4_store(whole, cuda(table), lens, both[:, :3].contiguous(), both[:, 3:].contiguous(), new_ptr=ptr)
    dbs.dbs_kv4_store(parts, cuda(table), lens, both[:, :3], both[:, 3:], new_ptr=ptr)
    assert torch.equal(layers[:, 1], whole.pool) and bool((layers[:, ::2] == 0xFF).all())


@pytest.mark.parametrize("sequences", [1, 63, 64, 65, 200, 4200])
def test_many_sequences(dbs, sequences):
    """The sequence of a workgroup is found among any number of them, empty ones included."""
    rng = np.random.default_rng(sequences)
    page, dim = 16, 64
    new = rng.integers(0, 3, sequences).tolist()
    new[sequences // 2] = 70
    lengths = [m + int(rng.integers(0, 20)) if m else 0 for m in new]
    table, pages = tables(rng, lengths, page)
    c = ref.Cache(pages, 1, dim, 64, page)
    total = sum(new)
    ptr = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
    v = rng.integers(0, 16, (sum(lengths), 1, dim)).astype(np.float32)
    v[..., 0], v[..., 1] = 0, 15
    cache = on_gpu(dbs, c)
    everything = np.concatenate(([0], np.cumsum(lengths))).astype(np.int32)
    lens = cuda(np.array(lengths, np.int32))
    dbs.dbs_kv4_store(cache, cuda(table), lens, cuda(v), cuda(v), new_ptr=cuda(everything))
    out = empty((total, 2, dim), "f32")
    dbs.dbs_kv4_attention(cache, cuda(table), lens, cuda(np.zeros((total, 2, dim), np.float32)), out, new_ptr=cuda(ptr))
    got = host(out)
    for b in range(sequences):
        x = v[everything[b] : everything[b + 1], 0].astype(np.float64)
        for i in range(new[b]):
            want = x[: lengths[b] - new[b] + i + 1].mean(0)
            np.testing.assert_allclose(got[ptr[b] + i], np.stack((want, want)), rtol=2.0 ** -22, atol=0)


def test_lengths_out_of_range_and_bad_lists(dbs):
    """Negative lengths and lengths past the table are clamped; rows that no list names are left alone."""
    import torch

    rng = np.random.default_rng(18)
    page = 16
    c = ref.Cache(6, 1, 64, 64, page)
    ref.random_bytes(rng, c)
    cache = on_gpu(dbs, c)
    table = cuda(np.array([[0, 1], [2, 3], [4, 5]], np.int32))
    q = cuda(rng.normal(0, 1, (9, 2, 64)).astype(np.float32))
    a, b = empty((9, 2, 64), "f32"), empty((9, 2, 64), "f32")
    dbs.dbs_kv4_attention(cache, table, cuda(np.array([-5, 1 << 30, 2], np.int32)), q, a)
    dbs.dbs_kv4_attention(cache, table, cuda(np.array([0, 32, 2], np.int32)), q, b)
    assert torch.equal(a, b) and bool((a[:3] == 0).all()) and bool((a[6] == 0).all()) and bool((a[7] != 0).any())
    for ptr in ([0, 3, 6, 4], [5, 2, 9, 9], [-3, 100, 3, 1 << 30]):
        out = empty((9, 2, 64), "f32")
        dbs.dbs_kv4_attention(cache, table, cuda(np.array([20, 20, 20], np.int32)), q, out, new_ptr=cuda(np.array(ptr, np.int32)))
        dbs.dbs_kv4_store(cache, table, cuda(np.array([20, 20, 20], np.int32)), q[:, :1], q[:, 1:], new_ptr=cuda(np.array(ptr, np.int32)))
    torch.cuda.synchronize()


def test_graph_of_a_step_replayed(dbs):
    """Norm and rotation, store and attention in a captured graph, on new lengths and inputs at each replay; another graph shares the
    pool's memory."""
    import torch

    rng = np.random.default_rng(19)
    heads, kv, dim, page, b = 8, 2, 128, 64, 3
    lengths = np.array([1500, 70, 300], np.int32)
    table, pages = tables(rng, [1600, 200, 400], page)
    c = ref.Cache(pages, kv, dim, 64, page)
    ref.random_bytes(rng, c)
    start = cuda(c.bytes)
    table = cuda(table)
    freq, _ = dbs.dbs_rope_frequencies(dim)
    freq = freq.cuda()
    weight = torch.ones(dim, device="cuda")

    def make():
        s = {"cache": dbs.dbs_kv4_cache(pages, kv, dim, 64, page, pool=start.clone()), "lens": cuda(lengths),
             "row": torch.zeros(b, heads + 2 * kv, dim, dtype=torch.bfloat16, device="cuda"), "pos": cuda(lengths - 1),
             "out": torch.zeros(b, heads, dim, dtype=torch.bfloat16, device="cuda")}
        return s

    def step(s):
        q, k, v = s["row"].split([heads, kv, kv], 1)
        dbs.dbs_norm_rope(q, k, weight, weight, s["pos"], freq, q, k)
        dbs.dbs_kv4_store(s["cache"], table, s["lens"], k, v)
        dbs.dbs_kv4_attention(s["cache"], table, s["lens"], q, s["out"])

    eager, graphs = make(), []
    for _ in range(2):
        s = make()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(s)
        torch.cuda.current_stream().wait_stream(side)
        s["cache"].pool.copy_(start)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(s)
        graphs.append((g, s))
    for turn in range(4):
        row = torch.randn(b, heads + 2 * kv, dim, device="cuda").bfloat16()
        for s in [eager] + [s for _, s in graphs]:
            s["row"].copy_(row)
            s["lens"].copy_(cuda(lengths + turn))
            s["pos"].copy_(cuda(lengths + turn - 1))
        step(eager)
        for g, s in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, s in graphs:
            assert torch.equal(s["out"], eager["out"]) and torch.equal(s["cache"].pool, eager["cache"].pool), f"replay {turn}"
        assert bool(torch.isfinite(eager["out"].float()).all())


def test_streams(dbs):
    """A call on a stream of its own, and two at once, each with its own workspace."""
    import torch

    rng = np.random.default_rng(20)
    n, page = 4000, 64
    table, pages = tables(rng, [n], page)
    c = ref.Cache(pages, 2, 128, 128, page)
    ref.random_bytes(rng, c)
    cache, lens, tab = on_gpu(dbs, c), cuda(np.array([n], np.int32)), cuda(table)
    qs = [cuda(rng.normal(0, 1, (1, 8, 128)).astype(np.float32)) for _ in range(2)]
    want = []
    for q in qs:
        want.append(empty(q.shape, "f32"))
        dbs.dbs_kv4_attention(cache, tab, lens, q, want[-1])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    outs = [[empty(q.shape, "f32") for _ in range(20)] for q in qs]
    torch.cuda.synchronize()
    for i in range(20):
        dbs.dbs_kv4_attention(cache, tab, lens, qs[0], outs[0][i], stream=streams[0])
        with torch.cuda.stream(streams[1]):
            dbs.dbs_kv4_attention(cache, tab, lens, qs[1], outs[1][i])
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(x, w) for x in o)


def test_step_with_the_layers_around_it(dbs):
    """A decoded token through the operators as a step uses them: 4-bit projections, norms and rotation, the cache, its attention and
    the output projection, against the same in 64 bits from the rounded intermediate results."""
    import torch

    import decode_ref as dref

    rng = np.random.default_rng(21)
    heads, kv, dim, page, b, hidden = 4, 2, 64, 16, 3, 256
    width = (heads + 2 * kv) * dim
    W, O = dref.Q4(rng, width, hidden, 64, True, exact=False), dref.Q4(rng, hidden, heads * dim, 64, True, exact=False)
    A, B = W.build(dbs), O.build(dbs)
    lengths = [19, 1, 50]
    table, pages = tables(rng, [n + 3 for n in lengths], page)
    c = ref.Cache(pages, kv, dim, 32, page)
    ref.random_bytes(rng, c)
    cache = on_gpu(dbs, c)
    freq, _ = dbs.dbs_rope_frequencies(dim)
    weight = rng.uniform(0.5, 1.5, dim).astype(np.float32)
    for step in range(3):
        now = np.array([n + step for n in lengths], np.int32)
        x = ref.typed(rng.normal(0, 1, (b, hidden)), "bf16")
        row = torch.empty(b, width, dtype=torch.bfloat16, device="cuda")
        dbs.dbs_q4_product(A, cuda(x, "bf16"), row)
        q, k, v = row.view(b, -1, dim).split([heads, kv, kv], 1)
        before = host(row).reshape(b, -1, dim)
        dbs.dbs_norm_rope(q, k, cuda(weight), cuda(weight), cuda(now - 1), freq.cuda(), q, k)
        after = host(row).reshape(b, -1, dim)
        for part in (slice(0, heads), slice(heads, heads + kv)):
            want, size = ref.norm_rope(before[:, part], weight, 1e-6, now - 1, freq.numpy(), False)
            assert (np.abs(after[:, part] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -19 * size).all()
        dbs.dbs_kv4_store(cache, cuda(table), cuda(now), k, v)
        for s in range(b):
            t = now[s] - 1
            for h in range(kv):
                c.store(table[s, t // page], t % page, h, after[s, heads + h], after[s, heads + kv + h])
        np.testing.assert_array_equal(cache.pool.cpu().numpy(), c.bytes)
        out = check(dbs, c, table, list(now), [1] * b, after[:, :heads], "bf16", "bf16")
        y = empty((b, hidden), "f32")
        dbs.dbs_q4_product(B, out.view(b, -1), y)
        want = host(out).reshape(b, -1).astype(np.float64) @ O.w.T
        assert np.abs(host(y) - want).max() <= 1e-4 * np.abs(want).max()


def test_refusals_of_the_binding(dbs):
    import torch

    cache = dbs.dbs_kv4_cache(4, 2, 64, 32, 16)
    table, lens = torch.zeros(2, 3, dtype=torch.int32, device="cuda"), torch.full((2,), 20, dtype=torch.int32, device="cuda")
    ptr = torch.tensor([0, 1, 4], dtype=torch.int32, device="cuda")
    q, k = torch.zeros(4, 4, 64, device="cuda"), torch.zeros(4, 2, 64, device="cuda")
    out, v = torch.zeros_like(q), torch.zeros_like(k)
    table[1] = 1

    def attend(cache=cache, table=table, lens=lens, q=q, out=out, **more):
        dbs.dbs_kv4_attention(cache, table, lens, q, out, **more)

    def store(cache=cache, table=table, lens=lens, k=k, v=v, **more):
        dbs.dbs_kv4_store(cache, table, lens, k, v, **more)

    store()
    attend(new_ptr=ptr)
    small = dbs.KV4Cache(cache.pool[:, :100], 2, 64, 32, 16)
    for call in (attend, store):
        for bad in (dict(cache=small), dict(cache=dbs.KV4Cache(cache.pool, 2, 64, 48, 16)), dict(cache=dbs.KV4Cache(cache.pool.int(), 2, 64, 32, 16)),
                    dict(table=table.long()), dict(table=table[0]), dict(table=table.t()), dict(lens=lens[:1]), dict(lens=lens.long()), dict(lens=None),
                    dict(new_ptr=ptr[:2]), dict(new_ptr=ptr.long())):
            with pytest.raises((ValueError, TypeError)):
                call(**bad)
    for bad in (dict(q=q[:3], out=out[:3]), dict(q=q[..., :32], out=out[..., :32]), dict(out=out[:, :2]), dict(q=q.half()), dict(q=q.cpu()), dict(q=q[0]),
                dict(workspace=torch.zeros(16, device="cuda")), dict(window=1 << 40), dict(out=out.transpose(1, 2))):
        with pytest.raises((ValueError, TypeError)):
            attend(**bad)
    for bad in (dict(q=q[:, :3], out=out[:, :3]), dict(out=q), dict(scale=0.0), dict(window=-1), dict(sinks=-1), dict(max_len=-1)):
        with pytest.raises(dbs.DBSError):
            attend(**bad)
    for bad in (dict(k=k[:, :1], v=v[:, :1]), dict(v=v.bfloat16()), dict(k_out=k.bfloat16(), v_out=torch.zeros_like(v)), dict(k_out=out), dict(v=v[:3])):
        with pytest.raises((ValueError, TypeError)):
            store(**bad)
    for bad in (dict(k_out=v), dict(k_out=out[:, :2], v_out=out[:, 1:3])):
        with pytest.raises(dbs.DBSError):
            store(**bad)
    assert dbs.dbs_kv4_attention_workspace(cache, table, lens, q, out) == 0
