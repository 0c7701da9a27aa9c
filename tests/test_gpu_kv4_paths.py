"""The attention over the cache of 4-bit keys and values at the sizes that its ways of cutting the work begin and end at, far offsets,
lists with gaps, and calls at the same time, on the GPU, against 64-bit references."""
import numpy as np
import pytest

import kv4_ref as ref
from test_gpu_kv4 import cuda, dbs, empty, host, tables  # noqa: F401

pytestmark = pytest.mark.gpu


def filled(dbs, rng, lengths, heads, dim, group, page, extra=0, pool=None):
    """A cache of random keys and values of these sequences: (cache, table, lens, k, v), k and v what it stands for, in 64 bits."""
    import torch

    table, pages = tables(rng, lengths, page, extra)
    total = sum(lengths)
    x = torch.from_numpy(rng.normal(0, 1, (2, total, heads, dim)).astype(np.float32)).cuda()
    cache = dbs.dbs_kv4_cache(pages, heads, dim, group, page, **({"pool": pool(pages)} if pool else {}))
    table, lens = cuda(table), cuda(np.array(lengths, np.int32))
    ptr = cuda(np.concatenate(([0], np.cumsum(lengths))).astype(np.int32))
    out = torch.empty_like(x)
    dbs.dbs_kv4_store(cache, table, lens, x[0], x[1], new_ptr=ptr, k_out=out[0], v_out=out[1])
    k, v = out.cpu().numpy().astype(np.float64)
    return cache, table, lens, k, v


def rows_off(rng, got, q, k, v, lengths, new, first, window, sinks, kind, wide, many):
    """The largest error of up to `many` rows of each sequence and head (the first and the last among them), in tolerances."""
    worst, start = 0.0, np.concatenate(([0], np.cumsum(lengths)))
    heads, dim = q.shape[1:]
    rep, scale = heads // k.shape[1], 1 / np.sqrt(dim)
    row = first
    for b, (n, m) in enumerate(zip(lengths, new)):
        if n and m:
            pick = np.unique(np.concatenate(([0, m - 1], rng.integers(0, m, many))))
            position = n - m + pick
            j = np.arange(n)
            see = j[None] <= position[:, None]
            if window:
                see &= (j[None] > position[:, None] - window) | (j[None] < sinks)
            for h in range(heads):
                kk, vv = k[start[b] : start[b + 1], h // rep], v[start[b] : start[b + 1], h // rep]
                qq = q[row + pick, h].astype(np.float64)
                s = np.where(see, scale * qq @ kk.T, -np.inf)
                size = np.where(see, scale * np.abs(qq) @ np.abs(kk).T, 0).max(1)[:, None]
                any_ = see.any(1)
                w = np.exp(s - np.where(any_, s.max(1), 0)[:, None])
                w /= np.where(any_, w.sum(1), 1)[:, None]
                want, mass = w @ vv, w @ np.abs(vv)
                tol = ref.attention_tolerance(want, mass, size, dim, n, kind, wide)
                worst = max(worst, float((np.abs(got[row + pick, h] - want) / tol).max()))
        elif m:
            assert (got[row : row + m] == 0).all()
        row += m
    return worst


def check(dbs, rng, lengths, new, heads, rep, dim, group, page=64, types=(("bf16", "bf16"),), window=0, sinks=0, max_len=0, extra=0, many=12,
          ragged=None, before=0, behind=3, **more):
    cache, table, lens, k, v = filled(dbs, rng, lengths, heads, dim, group, page, extra)
    ragged = len(set(new)) > 1 if ragged is None else ragged
    if not ragged:
        before = behind = 0
    rows = before + sum(new)
    ptr = cuda((before + np.concatenate(([0], np.cumsum(new)))).astype(np.int32)) if ragged else None
    for kind, out_kind in types:
        q = ref.typed(rng.normal(0, 1, (rows + behind, heads * rep, dim)), kind)
        out = empty(q.shape, out_kind)
        dbs.dbs_kv4_attention(cache, table, lens, cuda(q, kind), out, new_ptr=ptr, window=window, sinks=sinks, max_len=max_len, **more)
        got = host(out).astype(np.float64)
        off = rows_off(rng, got, q, k, v, lengths, new, before, window, sinks, out_kind, "f32" in (kind, out_kind), many)
        assert off <= 1, f"{kind} to {out_kind}: {off:.3g} of the tolerance"
        assert (got[:before] == 7).all() and (got[rows:] == 7).all()


PADDED = [(64, 32), (64, 64), (96, 32), (128, 32), (128, 64), (128, 128), (192, 32), (192, 64), (256, 32), (256, 64), (256, 128)]
BOTH = (("bf16", "bf16"), ("f32", "bf16"))

# sequences' lengths, new tokens of each, key heads, rows of a key head and token
WAYS = {
    "short": ([300, 1, 33], [1, 1, 1], 2, 3),
    "short of many": ([40, 7, 64, 15] * 75, [1] * 300, 1, 2),
    "some": ([510, 20], [1, 1], 2, 3),
    "some of many": ([500, 3, 130, 450] * 10, [1] * 40, 4, 2),
    "long": ([9000, 70], [1, 1], 1, 4),
    "drafts of a long one": ([6000, 90], [3, 3], 1, 4),
    "two tiles": ([1500, 70], [8, 3], 1, 7),
    "two tiles of a short one": ([60], [33], 2, 1),
    "piece": ([500, 65], [70, 65], 1, 3),
    "piece of a long one": ([7000], [40], 1, 4),
    "prompt": ([300], [300], 1, 2),
}


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("dim,group", PADDED)
def test_ways_of_cutting_the_work(dbs, dim, group, way):
    lengths, new, heads, rep = WAYS[way]
    rng = np.random.default_rng(dim + group + len(way))
    check(dbs, rng, lengths, new, heads, rep, dim, group, types=BOTH, many=3 if len(new) > 4 else 12)


@pytest.mark.parametrize("dim,group", [(128, 32), (128, 64), (128, 128), (192, 32), (192, 64), (104, 64), (136, 64)])
def test_prompts_of_eight_waves(dbs, dim, group):
    """Rows enough for workgroups of 256 of them: beside a long context, cut along it or not, ragged, under a window, from the first token."""
    rng = np.random.default_rng(group)
    check(dbs, rng, [8200], [512], 2, 4, dim, group, many=40)
    check(dbs, rng, [3000, 1700, 2500], [1500, 1100, 1300], 2, 4, dim, group, many=20)
    check(dbs, rng, [6000, 1100, 5001], [1100, 1000, 1201], 2, 4, dim, group, window=2000, sinks=70, many=20)
    check(dbs, rng, [6000, 1100, 5001], [1100, 1000, 1201], 2, 4, dim, group, window=100, many=20)
    check(dbs, rng, [1601], [1601], 16, 8, dim, group, many=3)


@pytest.mark.parametrize("rep", [17, 33, 64, 65, 80, 129, 200])
@pytest.mark.parametrize("dim,group", [(128, 64), (192, 64)])
def test_many_heads_on_one_key_head(dbs, rep, dim, group):
    rng = np.random.default_rng(rep)
    check(dbs, rng, [400, 31], [1, 1], 1, rep, dim, group, types=BOTH)


@pytest.mark.parametrize("window", [(1 << 31) - 1, 1 << 30, (1 << 30) - 1])
@pytest.mark.parametrize("each", [3, 30, 150])
def test_windows_and_sinks_of_any_size(dbs, window, each):
    """Of a sequence shorter than its new tokens too, whose first rows see nothing."""
    rng = np.random.default_rng(each)
    for sinks in (0, (1 << 31) - 1):
        cache, table, lens, k, v = filled(dbs, rng, [200, 300], 1, 64, 32, 16)
        q = cuda(rng.normal(0, 1, (2 * each, 2, 64)).astype(np.float32))
        for n in (lens, cuda(np.array([each // 2, 1], np.int32))):
            plain, out = empty(q.shape, "f32"), empty(q.shape, "f32")
            dbs.dbs_kv4_attention(cache, table, n, q, plain)
            dbs.dbs_kv4_attention(cache, table, n, q, out, window=window, sinks=sinks)
            np.testing.assert_array_equal(host(out), host(plain))


@pytest.mark.parametrize("before", [1, 40, 1000])
@pytest.mark.parametrize("new", [[1, 1, 1], [5, 0, 9], [70, 33, 0]])
def test_rows_before_the_first_sequence_are_left(dbs, before, new):
    rng = np.random.default_rng(before)
    check(dbs, rng, [200, 90, 33], new, 2, 3, 64, 64, types=BOTH, ragged=True, before=before)
    cache, table, lens, k, v = filled(dbs, rng, [200, 90, 33], 2, 64, 64, 16)
    was = cache.pool.clone()
    ptr = cuda((before + np.concatenate(([0], np.cumsum(new)))).astype(np.int32))
    x = cuda(rng.normal(0, 1, (2, before + sum(new) + 2, 2, 64)).astype(np.float32))
    out = empty(x.shape, "f32")
    dbs.dbs_kv4_store(cache, table, lens, x[0], x[1], new_ptr=ptr, k_out=out[0], v_out=out[1])
    got = host(out)
    assert (got[:, :before] == 7).all() and (got[:, before + sum(new) :] == 7).all() and (got[:, before : before + sum(new)] != 7).all()
    # the same tokens without the rows before them
    again = dbs.dbs_kv4_cache(cache.pool.shape[0], 2, 64, 64, 16, pool=was)
    dbs.dbs_kv4_store(again, table, lens, x[0, before:], x[1, before:], new_ptr=ptr - before)
    np.testing.assert_array_equal(again.pool.cpu().numpy(), cache.pool.cpu().numpy())


def test_pages_beyond_four_gigabytes(dbs):
    """Pages a gigabyte apart, and a compact pool of the same."""
    import torch

    lengths, new = [100, 61], [40, 1]
    size = dbs.dbs_kv4_page_bytes(2, 128, 64, 16)
    step = (1 << 30) + 16
    got = []
    for far in (True, False):
        rng = np.random.default_rng(3)
        hold = []

        def pool(pages):
            hold.append(torch.zeros((pages - 1) * step + size, dtype=torch.uint8, device="cuda"))
            return hold[0].as_strided((pages, size), (step, 1))

        cache, table, lens, k, v = filled(dbs, rng, lengths, 2, 128, 64, 16, pool=pool if far else None)
        assert not far or (cache.pool.shape[0] - 1) * step > 1 << 32
        for m in (1, 20, 60):
            q = cuda(rng.normal(0, 1, (2 * m, 8, 128)).astype(np.float32), "bf16")
            out = empty(q.shape, "bf16")
            dbs.dbs_kv4_attention(cache, table, lens, q, out)
            got.append(host(out))
        del cache, hold
    for a, b in zip(got[:3], got[3:]):
        np.testing.assert_array_equal(a, b)
        assert np.isfinite(a).all() and (a != 0).any()


@pytest.mark.parametrize("each", [1, 9, 40, 100, 300])
@pytest.mark.parametrize("dim,group", [(64, 32), (96, 32), (128, 64), (128, 128), (192, 64), (256, 128)])
def test_unused_places_may_hold_anything(dbs, dim, group, each):
    """Random bytes behind the lengths, in pages of no sequence and before the window: among them records that are finite and make
    values that are not."""
    rng = np.random.default_rng(dim + each)
    lengths, page = [2000 + each, 330], 256
    out = []
    for fill in range(3):
        rng = np.random.default_rng(dim + each)

        def pool(pages):
            size = dbs.dbs_kv4_page_bytes(2, dim, group, page)
            a = np.random.default_rng(fill).integers(0, 256, (pages, size), dtype=np.uint8) if fill else np.zeros((pages, size), np.uint8)
            return cuda(a)

        cache, table, lens, k, v = filled(dbs, rng, lengths, 2, dim, group, page, pool=pool)
        q = rng.normal(0, 1, (2 * each, 6, dim)).astype(np.float32)
        for kind in ("bf16", "f32"):
            got = empty(q.shape, kind)
            dbs.dbs_kv4_attention(cache, table, lens, cuda(q, kind), got)
            out.append(host(got))
            assert np.isfinite(out[-1]).all()
    for i in (2, 3, 4, 5):
        np.testing.assert_array_equal(out[i], out[i % 2])


def test_sequences_that_share_pages(dbs):
    """Rows of the table that name the same pages, each for its own length: a common beginning is held once."""
    rng = np.random.default_rng(4)
    cache, table, lens, k, v = filled(dbs, rng, [200], 2, 128, 64, 16)
    shared = table.expand(3, -1).contiguous()
    lens = cuda(np.array([200, 64, 130], np.int32))
    q = cuda(rng.normal(0, 1, (3 * 5, 4, 128)).astype(np.float32), "bf16")
    out = empty(q.shape, "bf16")
    dbs.dbs_kv4_attention(cache, shared, lens, q, out)
    for b in range(3):
        alone = empty((5, 4, 128), "bf16")
        dbs.dbs_kv4_attention(cache, table, lens[b : b + 1], q[5 * b : 5 * b + 5], alone)
        # one sequence may be cut in other places than three: two roundings of the output and both calls' weights
        np.testing.assert_allclose(host(out)[5 * b : 5 * b + 5], host(alone), rtol=2.0 ** -7, atol=2.0 ** -8)


def test_graphs_replayed_at_the_same_time(dbs):
    """Two graphs of a long context's step, whose splits have workspaces, on two streams: allocated in capture, or the caller's."""
    import torch

    rng = np.random.default_rng(5)
    cache, table, lens, k, v = filled(dbs, rng, [20000, 300], 2, 128, 64, 64)
    q = empty((2, 8, 128), "bf16")
    size = dbs.dbs_kv4_attention_workspace(cache, table, lens, q, q)
    assert size > 0
    for own in (False, True):
        steps = []
        for i in range(2):
            q = cuda(rng.normal(0, 1, (2, 8, 128)).astype(np.float32), "bf16")
            out, want = empty(q.shape, "bf16"), empty(q.shape, "bf16")
            more = dict(workspace=torch.empty(size, dtype=torch.uint8, device="cuda")) if own else {}
            dbs.dbs_kv4_attention(cache, table, lens, q, want)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                dbs.dbs_kv4_attention(cache, table, lens, q, out, **more)
            steps.append((graph, q, out, want, torch.cuda.Stream()))
        for round_ in range(5):
            torch.cuda.synchronize()
            for graph, q, out, want, stream in steps:
                out.fill_(7)
            torch.cuda.synchronize()
            for _ in range(4):
                for graph, q, out, want, stream in steps:
                    with torch.cuda.stream(stream):
                        graph.replay()
            torch.cuda.synchronize()
            for graph, q, out, want, stream in steps:
                assert torch.equal(out, want)


def test_a_prompt_captured(dbs):
    """Kernels with more shared memory than a launch gets unasked, in a graph that sees new tokens and lengths at each replay."""
    import torch

    rng = np.random.default_rng(6)
    for dim, group in ((128, 64), (256, 128)):
        cache, table, lens, k, v = filled(dbs, rng, [3000, 2500], 1, dim, group, 64)
        q = cuda(rng.normal(0, 1, (2 * 300, 4, dim)).astype(np.float32), "bf16")
        out = empty(q.shape, "bf16")
        stream = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            dbs.dbs_kv4_attention(cache, table, lens, q, out)
        for n in ([3000, 2500], [400, 301], [300, 0], [3000, 2500]):
            lens.copy_(torch.tensor(n, dtype=torch.int32))
            q.copy_(torch.randn_like(q))
            graph.replay()
            want = empty(q.shape, "bf16")
            dbs.dbs_kv4_attention(cache, table, lens, q, want)
            assert torch.equal(out, want)


def test_a_long_way(dbs):
    """As many tokens of one sequence as a table row of 16384 pages has room for, more than 2^17 of them far behind a window."""
    rng = np.random.default_rng(7)
    n = 16384 * 16 - 5
    check(dbs, rng, [n], [1], 1, 4, 64, 64, page=16)
    check(dbs, rng, [n], [2], 1, 4, 64, 64, page=16, window=5000, sinks=9)
    check(dbs, rng, [n], [40], 1, 4, 64, 64, page=16, many=3)
