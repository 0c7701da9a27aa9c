"""What the calls of the 4-bit cache and of the norm with rotary positions refuse, checked on the host before anything touches
a GPU (CPU only)."""
import ctypes as C
import math

import numpy as np
import pytest

import kv4_ref as ref
import spmspv_graph_traversal_amd.binding as b
from spmspv_graph_traversal_amd.binding import _lib

P = 1 << 20  # an address that is never read
POOL, TABLE, LENS, PTR, Q, OUT, SPACE = P, 1 << 30, 2 << 30, 3 << 30, 4 << 30, 5 << 30, 6 << 30
OK, INVALID, UNSUPPORTED = b.DBS_OK, b.DBS_ERR_INVALID_ARG, b.DBS_ERR_UNSUPPORTED


def page_bytes(heads=2, dim=64, group=32, page=16, out=True):
    v = C.c_int64(-1)
    return _lib.dbs_kv4_page_bytes(heads, dim, group, page, C.byref(v) if out else None), v.value


@pytest.mark.parametrize("dim,group", [(8, 32), (64, 64), (80, 32), (96, 32), (104, 128), (128, 64), (192, 64), (256, 128)])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_page_bytes(dim, group, page):
    assert page_bytes(3, dim, group, page) == (OK, 3 * ref.Cache(1, 1, dim, group, page).head_bytes)


@pytest.mark.parametrize("bad", [dict(heads=0), dict(heads=-1), dict(heads=65536), dict(dim=0), dict(dim=4), dict(dim=68), dict(dim=264),
                                 dict(dim=-8), dict(group=16), dict(group=0), dict(group=96), dict(group=256), dict(dim=64, group=128),
                                 dict(dim=96, group=64), dict(dim=80, group=64), dict(dim=192, group=128), dict(page=8), dict(page=48),
                                 dict(page=512), dict(page=0), dict(page=-16), dict(out=False)])
def test_page_refusals(bad):
    assert page_bytes(**bad)[0] == INVALID


def view(pool=POOL, page_stride=None, pages=4, page_tokens=16, key_heads=2, head_dim=64, group=32, sequences=3, table_pages=5, table=TABLE,
         ldtable=5, lens=LENS, new_ptr=None):
    if page_stride is None:
        page_stride = max(page_bytes(key_heads, head_dim, group, page_tokens)[1], 16)
    return b.dbs_kv4_view(pool, page_stride, pages, page_tokens, key_heads, head_dim, group, sequences, table_pages, table, ldtable, lens, new_ptr)


def attend(tokens=3, heads=4, q=Q, qd=0, qt=256, qh=64, out=OUT, od=0, ot=256, oh=64, scale=1.0, window=0, sinks=0, max_len=0, space=None,
           space_bytes=0, cache=True, **kw):
    v = view(**kw)
    return _lib.dbs_kv4_attention(C.byref(v) if cache else None, tokens, heads, q, qd, qt, qh, out, od, ot, oh, scale, window, sinks, max_len, space,
                                  space_bytes, None)


def store(tokens=3, k=Q, kt=128, kh=64, v=None, vt=128, vh=64, xd=0, ko=OUT, kot=128, koh=64, vo=None, vot=128, voh=64, od=0, cache=True, **kw):
    c = view(**kw)
    return _lib.dbs_kv4_store(C.byref(c) if cache else None, tokens, k, kt, kh, Q + (1 << 20) if v is None else v, vt, vh, xd, ko, kot, koh,
                              OUT + (1 << 20) if vo is None else vo, vot, voh, od, None)


BAD_CACHES = [
    dict(cache=False), dict(tokens=-1), dict(tokens=4), dict(pool=None), dict(pool=P + 8), dict(page_stride=16), dict(page_stride=-16),
    dict(page_stride=page_bytes()[1] + 8), dict(pages=0), dict(pages=-1), dict(page_tokens=24), dict(key_heads=0), dict(head_dim=72, group=64),
    dict(group=0), dict(sequences=-1), dict(sequences=0), dict(table_pages=-1), dict(table=None), dict(ldtable=4), dict(lens=None)]


@pytest.mark.parametrize("bad", BAD_CACHES + [
    dict(heads=3), dict(heads=-2), dict(qd=2), dict(od=-1), dict(q=None), dict(out=None), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.inf),
    dict(scale=math.nan), dict(scale=3e38), dict(window=-1), dict(sinks=-1), dict(max_len=-1), dict(space_bytes=-1), dict(space_bytes=64), dict(space=P + 4, space_bytes=64),
    dict(oh=63), dict(ot=255), dict(ot=0), dict(out=Q), dict(out=Q + 4 * 700), dict(out=POOL), dict(out=POOL + 4 * page_bytes()[1] - 16), dict(out=LENS),
    dict(out=TABLE + 48), dict(new_ptr=PTR, out=PTR - 4), dict(out=LENS - 4 * 767)])
def test_attention_refusals(bad):
    assert attend(**bad) == INVALID


@pytest.mark.parametrize("bad", BAD_CACHES + [
    dict(xd=2), dict(od=3), dict(k=None), dict(v=0), dict(k=POOL), dict(v=POOL + 64), dict(koh=63), dict(kot=64), dict(vot=-64), dict(ko=POOL), dict(vo=TABLE),
    dict(ko=LENS), dict(ko=Q, od=1), dict(ko=Q, kot=256), dict(ko=Q + (1 << 20)), dict(vo=OUT), dict(vo=OUT + 4 * 300), dict(lens=POOL + 16),
    dict(table=POOL), dict(new_ptr=POOL + 4), dict(lens=POOL + 4 * page_bytes()[1] - 8)])
def test_store_refusals(bad):
    if bad.get("v") == 0:
        v = view()
        assert _lib.dbs_kv4_store(C.byref(v), 3, Q, 128, 64, None, 128, 64, 0, None, 0, 0, None, 0, 0, 0, None) == INVALID
        return
    assert store(**bad) == INVALID


def test_limits_and_nothing_to_do():
    assert attend(table_pages=1 << 26, ldtable=1 << 26, page_tokens=32) == UNSUPPORTED
    assert attend(sequences=b.DBS_KV4_MAX_SEQUENCES + 1, new_ptr=PTR) == UNSUPPORTED
    assert attend(tokens=3 << 20, heads=8) == UNSUPPORTED
    assert store(tokens=3 << 22, key_heads=2) == UNSUPPORTED
    many = dict(sequences=1 << 20, tokens=1 << 20, key_heads=16, heads=16, qt=1024, ot=1024, out=16 << 30, table_pages=1, ldtable=1)
    assert attend(**many) == UNSUPPORTED  # a workgroup a sequence and key head
    for none in (dict(tokens=0), dict(sequences=0, new_ptr=PTR), dict(sequences=0, tokens=0)):
        assert attend(pool=None, table=None, lens=None, q=None, out=None, **none) == OK
        assert store(pool=None, table=None, lens=None, k=None, ko=None, **none) == OK
    assert attend(heads=0) == OK


def workspace(tokens=3, heads=4, qd=1, od=1, window=0, sinks=0, max_len=0, out=True, **kw):
    v, c = C.c_int64(-1), view(**kw)
    return _lib.dbs_kv4_attention_workspace(C.byref(c), tokens, heads, qd, od, window, sinks, max_len, C.byref(v) if out else None), v.value


def test_workspace_goes_by_the_room_that_is_seen():
    """None where the rows or short lengths leave nothing to cut; as much for a window as for lengths of its size; a bound of the lengths
    counts, and one past the room does not."""
    assert workspace(out=False)[0] == INVALID and workspace(heads=3)[0] == INVALID
    assert workspace() == (OK, 0) and workspace(tokens=0, table_pages=4096, ldtable=4096) == (OK, 0)
    long = dict(table_pages=4096, ldtable=4096)
    st, all_of_it = workspace(**long)
    assert st == OK and all_of_it > 0 and all_of_it % (3 * 4 * (64 + 2) * 4) == 0
    assert workspace(max_len=1 << 30, **long) == (OK, all_of_it)
    assert workspace(max_len=100, **long) == (OK, 0)
    assert 0 < workspace(max_len=8192, **long)[1] < all_of_it
    assert 0 < workspace(window=8192, sinks=4, **long)[1] < all_of_it
    assert workspace(window=100, sinks=4, **long) == (OK, 0)
    assert workspace(tokens=3 << 15, heads=32, **long) == (OK, 0)


def part(x=P, xt=64, xh=8, out=2 * P, ot=64, oh=8, heads=3, weight=None):
    return b.dbs_norm_part(x, xt, xh, out, ot, oh, heads, weight)


def norm(tokens=2, dim=8, rot=8, layout=0, pos=10 * P, freq=11 * P, scale=1.0, eps=1e-6, parts=None, count=None, xd=0, od=0, wd=0):
    parts = [part(), part(x=3 * P, out=4 * P)] if parts is None else parts
    a = (b.dbs_norm_part * max(1, len(parts)))(*parts)
    return _lib.dbs_norm_rope(tokens, dim, rot, layout, pos, freq, scale, eps, a if parts else None, len(parts) if count is None else count, xd, od, wd, None)


@pytest.mark.parametrize("bad", [
    dict(tokens=-1), dict(dim=0), dict(rot=-2), dict(rot=7), dict(rot=10), dict(layout=2), dict(layout=-1), dict(pos=None), dict(freq=None),
    dict(eps=-1e-6), dict(eps=math.nan), dict(eps=math.inf), dict(parts=[]), dict(count=0), dict(count=3), dict(xd=2), dict(od=2), dict(wd=2), dict(wd=-1),
    dict(parts=[part(x=None)]), dict(parts=[part(out=None)]), dict(parts=[part(heads=-1)]), dict(parts=[part(oh=7)]), dict(parts=[part(ot=16)]),
    dict(parts=[part(out=P, ot=32)]), dict(parts=[part(out=P)], od=1), dict(parts=[part(out=P + 32)]),
    dict(parts=[part(), part(x=3 * P)]),                      # both into one output
    dict(parts=[part(), part(x=2 * P, out=4 * P)]),           # one writes what the other reads
    dict(parts=[part(out=4 * P), part(x=3 * P, out=P)]),
    dict(parts=[part(weight=2 * P + 32)]), dict(parts=[part(), part(x=3 * P, out=4 * P, weight=2 * P)]), dict(pos=2 * P + 4), dict(freq=4 * P),
    dict(parts=[part(out=P, heads=4, xt=72, ot=72), part(x=P + 4 * 24, out=P + 4 * 24, xt=72, ot=72)]),  # heads of a row that meet
])
def test_norm_refusals(bad):
    assert norm(**bad) == INVALID


def test_norm_limits_and_nothing_to_do():
    assert norm(tokens=0, pos=None) == OK
    assert norm(parts=[part(heads=0, x=None, out=None)], pos=None) == OK
    assert norm(dim=1026, rot=0, parts=[part(xh=1026, oh=1026, xt=9999, ot=9999)]) == UNSUPPORTED
    assert norm(dim=1024, rot=0, parts=[part(heads=1 << 20, xh=1024, oh=1024, xt=1 << 31, ot=1 << 31), part(x=3 << 40, out=4 << 40)]) == UNSUPPORTED


def test_binding_refuses_what_the_tensors_do_not_fit():
    import torch

    with pytest.raises(ValueError):
        b.dbs_kv4_page_bytes(1 << 32, 64, 32, 16)
    with pytest.raises(b.DBSError):
        b.dbs_kv4_page_bytes(2, 64, 48, 16)
    with pytest.raises(TypeError):
        b.dbs_kv4_cache(4, 2, 64, 32, 16, pool=torch.zeros(4, 4096, dtype=torch.uint8))  # not on a GPU


def test_definition_against_differences():
    """The codes of the definition are the nearest: no other code of the group's sixteen values is nearer by more than the records'
    rounding."""
    rng = np.random.default_rng(1)
    c = ref.Cache(1, 1, 128, 32, 16)
    for size in (1e-3, 1.0, 500.0):
        x = (rng.normal(0, size, 128)).astype(np.float32)
        q, s, of = c.quantize(x)
        got = c.value(q, s, of)
        for g in range(4):
            levels = np.float64(s[g]) * np.arange(16) + np.float64(of[g])
            part, span = x[32 * g : 32 * g + 32].astype(np.float64), np.float64(s[g])
            best = np.abs(part[:, None] - levels).min(1)
            # what is returned is the level rounded to a half: off by half a step of the level, which is within `best` of the value
            assert (np.abs(got[32 * g : 32 * g + 32] - part) <= best + 2.0 ** -11 * (np.abs(part) + best) + 1e-6 * span).all()
            assert (best <= span * (0.5 + 15 * 2.0 ** -11) + 2.0 ** -11 * np.abs(levels).max()).all()
