"""What the decode-step entry points refuse, checked on the host before anything touches a GPU, and the rotary
frequencies (CPU only)."""
import ctypes as C
import math

import numpy as np
import pytest

import spmspv_graph_traversal_amd.binding as b
from spmspv_graph_traversal_amd.binding import _lib

P = 1 << 20  # an address that is never read
OK, INVALID, UNSUPPORTED = b.DBS_OK, b.DBS_ERR_INVALID_ARG, b.DBS_ERR_UNSUPPORTED


def q4_build(m=4, n=4, group=32, codes=P, scales=P, sd=0, out=True):
    h = C.c_void_p()
    return _lib.dbs_q4_build(m, n, group, codes, scales, sd, None, None, C.byref(h) if out else None)


@pytest.mark.parametrize("bad", [dict(m=0), dict(n=0), dict(m=-1), dict(group=0), dict(group=16), dict(group=48),
                                 dict(group=256), dict(codes=None), dict(scales=None), dict(sd=2), dict(sd=-1), dict(out=False)])
def test_q4_build_refusals(bad):
    assert q4_build(**bad) == INVALID


def test_q4_build_limits():
    assert q4_build(m=b.DBS_Q4_MAX_ROWS + 1) == UNSUPPORTED
    assert q4_build(n=b.DBS_Q4_MAX_COLUMNS + 1) == UNSUPPORTED


@pytest.mark.parametrize("m,n", [((1 << 32) + 4, 8), (4, (1 << 32) + 8), (b.DBS_Q4_MAX_ROWS + 1, 8)])
def test_q4_sizes_past_32_bits_are_not_cut(m, n):
    import torch

    with pytest.raises(ValueError, match="too large"):
        b.dbs_q4_build(m, n, 32, torch.zeros(16, dtype=torch.uint8), torch.ones(4))


def test_q4_calls_without_a_handle():
    v = C.c_int64()
    assert _lib.dbs_q4_bytes(None, C.byref(v)) == INVALID
    assert _lib.dbs_q4_free(None) == OK
    assert _lib.dbs_q4_product(None, 1, P, 0, 4, P, 0, 4, None) == INVALID
    assert _lib.dbs_q4_product_masked(None, 1, P, 0, 4, P, 1, 0.0, P, 0, 4, None) == INVALID
    assert _lib.dbs_q4_gated(None, None, 0, 1, P, 0, 4, P, 0, 4, None) == INVALID


def logits(rows=2, vocab=40, x=P, xd=0, ldx=40, out=2 * P, od=0, ldo=40, params=True, **fields):
    p = b.dbs_logits_params(**fields)
    return _lib.dbs_logits_adjust(rows, vocab, x, xd, ldx, bytes(p) if params else None, out, od, ldo, None)


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(vocab=0), dict(params=False), dict(xd=2), dict(od=2), dict(x=None), dict(out=None),
    dict(ldx=39), dict(ldo=39), dict(mask=P, ldmask=1), dict(hist_ptr=P, hist_len=3), dict(hist=P),
    dict(repetition=P), dict(frequency=P), dict(presence=P), dict(hist_new=P), dict(bias_ptr=P, bias_len=2, bias_idx=P),
    dict(bias_ptr=P, bias_len=2, bias_val=P), dict(bias_idx=P), dict(bias_val=P), dict(hist_ptr=P, hist=P, hist_len=-1),
    dict(hist_ptr=P, hist=P, hist_len=1 << 31), dict(bias_ptr=P, bias_idx=P, bias_val=P, bias_len=-1),
    dict(out=P, od=1),            # in place with another type
    dict(out=P, ldo=41),          # in place with another stride
    dict(out=P + 4 * 79),         # overlapping the last row's end
])
def test_logits_refusals(bad):
    assert logits(**bad) == INVALID


def test_logits_limits_and_nothing_to_do():
    assert logits(rows=0, x=None, out=None) == OK
    assert logits(rows=b.DBS_LOGITS_MAX_ROWS + 1) == UNSUPPORTED


def rope(tokens=2, heads=3, dim=8, rot=8, layout=0, pos=P, freq=P, x=P, xd=0, xt=24, xh=8, out=2 * P, od=0, ot=24, oh=8):
    return _lib.dbs_rope(tokens, heads, dim, rot, layout, pos, freq, 1.0, 0, x, xd, xt, xh, out, od, ot, oh, None)


@pytest.mark.parametrize("bad", [
    dict(tokens=-1), dict(heads=-1), dict(dim=0), dict(rot=-2), dict(rot=7), dict(rot=10), dict(layout=2), dict(layout=-1),
    dict(xd=2), dict(od=3), dict(pos=None), dict(freq=None), dict(x=None), dict(out=None), dict(oh=7), dict(oh=0),
    dict(ot=0), dict(ot=-7), dict(out=P, od=1), dict(out=P, ot=32), dict(out=P, oh=16),
])
def test_rope_refusals(bad):
    assert rope(**bad) == INVALID


def test_rope_limits_and_nothing_to_do():
    assert rope(tokens=0, pos=None, freq=None, x=None, out=None) == OK
    assert rope(heads=0) == OK
    assert rope(dim=2048, rot=1026, oh=2048, ot=3 * 2048) == UNSUPPORTED
    assert rope(heads=1 << 20, dim=1 << 11, oh=1 << 11, ot=1 << 31) == UNSUPPORTED


@pytest.mark.parametrize("oh,ot", [(8, 8), (8, 16), (8, 23), (8, 31), (15, 8), (-8, 24), (8, -25), (16, 7), (9, 0)])
def test_rope_refuses_outputs_whose_rows_meet(oh, ot):
    rows = [{t * ot + h * oh + d for d in range(8)} for t in range(2) for h in range(4)]
    assert len(set.union(*rows)) < 8 * len(rows)
    assert rope(tokens=2, heads=4, oh=oh, ot=ot) == INVALID


def test_rope_largest_head_that_a_lane_can_count():
    last = b.DBS_ROPE_MAX_ELEMENTS
    assert rope(heads=1, dim=last + 8, oh=last + 8, ot=last + 8) == UNSUPPORTED
    assert rope(heads=1, dim=2**31 - 1, rot=0, oh=2**31 - 1, ot=2**31 - 1) == UNSUPPORTED
    assert rope(tokens=0, heads=1, dim=last, oh=last, ot=last) == OK


def frequencies(**kw):
    o = dict(rot_dim=8, scaling=0, base=10000.0, factor=2.0, low=1.0, high=4.0, context=4096.0)
    o.update(kw)
    opt = b.dbs_rope_options(**o)
    f = (C.c_double * 512)()
    return _lib.dbs_rope_frequencies(C.byref(opt), f, None)


@pytest.mark.parametrize("bad", [
    dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=1026), dict(scaling=5), dict(scaling=-1), dict(base=1.0), dict(base=math.nan),
    dict(base=math.inf), dict(scaling=1, factor=0.5), dict(scaling=1, factor=math.nan), dict(scaling=2, rot_dim=2),
    dict(scaling=3, low=0.0), dict(scaling=3, high=1.0), dict(scaling=4, context=0.0), dict(scaling=4, high=math.inf),
    dict(scaling=3, context=math.nan)])
def test_frequency_refusals(bad):
    assert frequencies(**bad) == INVALID
    assert _lib.dbs_rope_frequencies(None, (C.c_double * 4)(), None) == INVALID


def test_frequencies():
    half = 64
    plain = 10000.0 ** (-np.arange(half) / half)
    f, scale = b.dbs_rope_frequencies(128)
    np.testing.assert_allclose(f.numpy(), plain, rtol=1e-14)
    assert scale == 1.0 and f.dtype.itemsize == 8
    f, _ = b.dbs_rope_frequencies(128, scaling=b.DBS_ROPE_LINEAR, factor=4)
    np.testing.assert_allclose(f.numpy(), plain / 4, rtol=1e-14)
    f, _ = b.dbs_rope_frequencies(128, scaling=b.DBS_ROPE_BASE, factor=4)
    np.testing.assert_allclose(f.numpy(), (10000.0 * 4 ** (128 / 126)) ** (-np.arange(half) / half), rtol=1e-13)
    # a whole factor at the lowest frequency, none at the highest
    np.testing.assert_allclose([f[0].item(), f[-1].item()], [1.0, plain[-1] / 4], rtol=1e-12)
    context = 8192
    turns = context * plain / (2 * np.pi)
    f, scale = b.dbs_rope_frequencies(128, scaling=b.DBS_ROPE_BANDS, factor=8, low=1, high=4, context=context)
    w = np.clip((turns - 1) / 3, 0, 1)
    np.testing.assert_allclose(f.numpy(), plain * ((1 - w) / 8 + w), rtol=1e-13)
    assert scale == 1.0 and (w == 0).any() and (w == 1).any() and ((w > 0) & (w < 1)).any()
    f, scale = b.dbs_rope_frequencies(128, scaling=b.DBS_ROPE_RAMP, factor=8, low=1, high=32, context=context)
    per = 128 / (2 * math.log(10000.0))
    first, last = math.floor(per * math.log(context / (2 * math.pi * 32))), math.ceil(per * math.log(context / (2 * math.pi)))
    w = np.clip((np.arange(half) - first) / (last - first), 0, 1)
    np.testing.assert_allclose(f.numpy(), plain * (w / 8 + 1 - w), rtol=1e-13)
    assert scale == pytest.approx(0.1 * math.log(8) + 1, rel=1e-6)
    assert 0 < first < last < half


def test_cpu_tensors_are_refused():
    import torch

    x = torch.zeros(2, 3, 8)
    with pytest.raises(TypeError):
        b.dbs_rope(x, torch.zeros(2, dtype=torch.int32), torch.ones(4, dtype=torch.float64), x)
    with pytest.raises(TypeError):
        b.dbs_logits_adjust(torch.zeros(4), torch.zeros(4))
    with pytest.raises(TypeError):
        b.dbs_q4_build(2, 4, 32, torch.zeros(2, 2, dtype=torch.uint8), torch.ones(2, 1))
    with pytest.raises(ValueError):
        b.dbs_q4_build(2, 4, 48, torch.zeros(2, 2, dtype=torch.uint8), torch.ones(2, 1))


def test_matrices_of_the_other_kind_are_refused():
    """A sparse matrix's handle is never read as a 4-bit one's, nor freed as one, and the other way round."""
    q4, sparse = b.Q4Matrix(C.c_void_p(), 4, 4, 32), b.Matrix(C.c_void_p(), 4, 4, b.DBS_F32)
    for call in (lambda: b.dbs_free(q4), lambda: b.dbs_get_stats(q4), lambda: b.dbs_set_option(q4, b.DBS_OPT_PATH, 0),
                 lambda: b.dbs_copy_array(q4, b.DBS_ARR_RB_PTR), lambda: b.dbs_q4_free(sparse), lambda: b.dbs_q4_bytes(sparse),
                 lambda: b.dbs_q4_product(sparse, None, None), lambda: b.dbs_q4_product_masked(sparse, None, None, None),
                 lambda: b.dbs_q4_gated(q4, sparse, None, 0, None), lambda: b.dbs_q4_gated(sparse, q4, None, 0, None)):
        with pytest.raises(TypeError, match="matrix"):
            call()
    assert b.dbs_q4_free(q4) is None and b.dbs_free(sparse) is None


@pytest.mark.parametrize("context,low,high,first,last", [
    (100, 1.0, 32.0, 0, 20),       # pair 0 turns fewer than `high` times: the ramp starts there
    (4, 1.0, 32.0, 0, None),       # fewer than `low` times even: f / factor behind pair 0
    (10 ** 15, 1.0, 32.0, None, None),  # every pair turns more than `high` times: f
    (10 ** 9, 1.0, 10.0 ** 8, 3, 127),  # the ramp's end is kept at the last element
])
def test_ramp_at_the_ends(context, low, high, first, last):
    plain = 10000.0 ** (-np.arange(64) / 64)
    at = lambda t: 128 * math.log(context / (2 * math.pi * t)) / (2 * math.log(10000.0))
    f, _ = b.dbs_rope_frequencies(128, scaling=b.DBS_ROPE_RAMP, factor=8, low=low, high=high, context=context)
    i = np.arange(64)
    if first is None:
        assert math.floor(at(high)) > 127
        w = np.zeros(64)
    elif last is None:
        assert math.ceil(at(low)) <= first
        w = (i > first).astype(float)
    else:
        assert max(math.floor(at(high)), 0) == first and min(math.ceil(at(low)), 127) == last
        w = np.clip((i - first) / (last - first), 0, 1)
    np.testing.assert_allclose(f.numpy(), plain * (w / 8 + 1 - w), rtol=1e-13)
