"""Norms of query and key heads with their rotary positions against a 64-bit reference, on the GPU."""
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


def within(got, want, size, dim, kind):
    """The sum of squares is off by dim + 2 roundings of fp32 at most, its root by half of that and two; the products by the root, the
    weight, the cosine (2^-23 absolutely, the turn's fraction having 24 bits: 2 pi 2^-25 of it) and the sum of two by eight."""
    tol = ref.HALF_STEP[kind] * np.abs(want) + ((dim + 2) / 2 + 2 + 8 + 8) * 2.0 ** -24 * size + 1e-37
    off = np.abs(got - want)
    assert (off <= tol).all(), f"off {off.max():.3g}, {(off / tol).max():.3g} of the tolerance"


SIZES = [(1, 0), (2, 2), (64, 64), (80, 40), (80, 38), (96, 96), (128, 128), (128, 64), (128, 0), (192, 128), (256, 256), (100, 36), (130, 130), (72, 8),
         (33, 6), (511, 510), (1023, 0), (1024, 1024), (1000, 12)]


@pytest.mark.parametrize("kind,out_kind", [("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot", SIZES)
def test_every_head_size(dbs, dim, rot, interleaved, kind, out_kind):
    rng = np.random.default_rng(dim * 3 + rot)
    for tokens, qh, kh in ((1, 5, 2), (3, 1, 0), (40, 9, 3)):
        q, k = (ref.typed(rng.normal(0, 3, (tokens, h, dim)), kind) for h in (qh, kh))
        qw, kw = (ref.typed(rng.uniform(0.5, 2, dim), "bf16") for _ in range(2))
        pos = rng.integers(0, 1 << 20, tokens).astype(np.int32)
        freq = 10000.0 ** (-np.arange(rot // 2) / max(1, rot // 2))
        qo, ko = empty(q.shape, out_kind), empty(k.shape, out_kind)
        layout = dbs.DBS_ROPE_INTERLEAVED if interleaved else dbs.DBS_ROPE_HALF
        dbs.dbs_norm_rope(cuda(q, kind), cuda(k, kind), cuda(qw, "bf16"), cuda(kw, "bf16"), cuda(pos), cuda(freq), qo, ko, eps=1e-5, layout=layout, scale=1.25)
        for x, w, o in ((q, qw, qo), (k, kw, ko)):
            if x.size:
                want, size = ref.norm_rope(x, w, float(np.float32(1e-5)), pos, freq, interleaved, 1.25)
                within(host(o), want, size, dim, out_kind)


def test_alone_without_weights_and_in_place(dbs):
    import torch

    rng = np.random.default_rng(2)
    dim, tokens = 128, 600
    freq = 10000.0 ** (-np.arange(64) / 64)
    pos = np.arange(tokens, dtype=np.int32)
    pos[5], pos[599] = -1, -7  # padding: left as it was
    row = ref.typed(rng.normal(0, 1, (tokens, 7, dim)), "bf16")
    w = rng.uniform(0.5, 2, dim).astype(np.float32)
    x = cuda(row, "bf16")
    dbs.dbs_norm_rope(x[:, 1:5], x[:, 5:6], cuda(w), None, cuda(pos), cuda(freq), x[:, 1:5], x[:, 5:6])
    got = host(x)
    for part, weight in ((slice(1, 5), w), (slice(5, 6), None)):
        want, size = ref.norm_rope(row[:, part], weight, float(np.float32(1e-6)), np.maximum(pos, 0), freq, False)
        want[pos < 0], size[pos < 0] = row[:, part][pos < 0], 0
        within(got[:, part], want, size, dim, "bf16")
    np.testing.assert_array_equal(got[:, [0, 6]], row[:, [0, 6]])
    alone = empty((tokens, 4, dim), "bf16")
    dbs.dbs_norm_rope(cuda(row, "bf16")[:, 1:5], None, cuda(w), None, cuda(np.abs(pos)), cuda(freq), alone, None)
    keep = pos >= 0
    assert torch.equal(alone[cuda(keep)], x[:, 1:5][cuda(keep)])
    heads_first = cuda(row[:, 1:5].transpose(1, 0, 2), "bf16").transpose(0, 1)
    turned = torch.full((4, tokens, dim + 3), 7.0, dtype=torch.bfloat16, device="cuda")
    dbs.dbs_norm_rope(heads_first, None, cuda(w), None, cuda(np.abs(pos)), cuda(freq), turned.transpose(0, 1)[..., :dim], None)
    assert torch.equal(turned.transpose(0, 1)[..., :dim], alone) and bool((turned[..., dim:] == 7).all())


def test_agrees_with_the_rotation_alone(dbs):
    """Of heads whose mean square is 1, without weights, the norm is no change: the rotation's own bits."""
    import torch

    rng = np.random.default_rng(3)
    x = cuda((rng.integers(0, 2, (50, 6, 128)) * 2 - 1).astype(np.float32))
    pos, freq = cuda(np.arange(900000, 900050, dtype=np.int32)), dbs.dbs_rope_frequencies(96, base=500000.0)[0].cuda()
    for layout in (dbs.DBS_ROPE_HALF, dbs.DBS_ROPE_INTERLEAVED):
        a, b = torch.empty_like(x), torch.empty_like(x)
        dbs.dbs_norm_rope(x, None, None, None, pos, freq, a, None, eps=0.0, layout=layout, scale=0.5)
        dbs.dbs_rope(x, pos, freq, b, layout=layout, scale=0.5)
        assert torch.equal(a, b)


@pytest.mark.parametrize("fill,want", [(0.0, 0.0), (np.nan, np.nan), (np.inf, np.nan)])
def test_heads_of_zeros_and_of_values_that_are_not_finite(dbs, fill, want):
    """A head of zeros stays one; a NaN or an infinity fills its own head's results and no other's."""
    rng = np.random.default_rng(4)
    x = rng.normal(0, 1, (3, 4, 64)).astype(np.float32)
    if fill == 0.0:
        x[1, 2] = 0.0
    else:
        x[1, 2, 17] = fill
    out = empty(x.shape, "f32")
    freq = 10000.0 ** (-np.arange(32) / 32)
    pos = np.arange(3, dtype=np.int32)
    dbs.dbs_norm_rope(cuda(x), None, None, None, cuda(pos), cuda(freq), out, None)
    got = host(out)
    if fill == 0.0:
        assert (got[1, 2] == 0).all()
    else:
        assert np.isnan(got[1, 2, [17, 49]]).all()
    ok = np.ones((3, 4), bool)
    ok[1, 2] = False
    w, size = ref.norm_rope(np.where(np.isfinite(x), x, 0), None, float(np.float32(1e-6)), pos, freq, False)
    within(got[ok], w[ok], size[ok], 64, "f32")


def test_refusals_of_the_binding(dbs):
    import torch

    q, k = torch.zeros(2, 4, 64, device="cuda"), torch.zeros(2, 2, 64, device="cuda")
    w, pos, freq = torch.ones(64, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda"), torch.ones(32, dtype=torch.float64, device="cuda")
    qo, ko = torch.zeros_like(q), torch.zeros_like(k)

    def call(q=q, k=k, qw=w, kw=w, pos=pos, freq=freq, qo=qo, ko=ko, **more):
        dbs.dbs_norm_rope(q, k, qw, kw, pos, freq, qo, ko, **more)

    call()
    for bad in (dict(k=None), dict(ko=None), dict(k=None, ko=None), dict(qo=qo[:1]), dict(q=q[0]), dict(k=k[:, :, :32]), dict(qw=w[:32]), dict(kw=w[::2]),
                dict(pos=pos[:1]), dict(qo=qo.transpose(1, 2)), dict(k=k[:1], ko=ko[:1])):
        with pytest.raises((ValueError, TypeError)):
            call(**bad)
    for bad in (dict(k=k.bfloat16()), dict(ko=ko.bfloat16()), dict(kw=w.bfloat16()), dict(pos=pos.long()), dict(freq=freq.float()), dict(q=q.half()), dict(pos=None),
                dict(q=q.cpu()), dict(qw=w.half())):
        with pytest.raises(TypeError):
            call(**bad)
    for bad in (dict(qo=q[:, :, :], ko=q[:, 1:3]), dict(freq=torch.ones(33, dtype=torch.float64, device="cuda")), dict(eps=-1.0)):
        with pytest.raises(dbs.DBSError):
            call(**bad)
