"""Outputs that overlap an input are refused by the decode-step entry points, on the host before anything touches a GPU
(CPU only; the calls that are accepted run in test_gpu_decode_step_overlap.py)."""
import pytest

import spmspv_graph_traversal_amd.binding as b
from spmspv_graph_traversal_amd.binding import _lib

P = 1 << 20  # an address that is never read
INVALID = b.DBS_ERR_INVALID_ARG


def rope(tokens=4, heads=3, dim=8, rot=8, x=P, xd=0, xt=24, xh=8, out=P, od=0, ot=24, oh=8, pos=1 << 30, freq=1 << 31):
    return _lib.dbs_rope(tokens, heads, dim, rot, 0, pos, freq, 1.0, 0, x, xd, xt, xh, out, od, ot, oh, None)


@pytest.mark.parametrize("bad", [
    dict(out=P + 4),                                     # by one element
    dict(out=P + 4 * 8), dict(out=P - 4 * 8),            # by a head
    dict(out=P + 4 * 24), dict(out=P - 4 * 24 * 3),      # by a token
    dict(xt=64, ot=64, out=P + 4 * 23),                  # parts of one buffer: queries' last element
    dict(xt=64, ot=64, out=P + 4 * (64 - 23)),           # the next token's first
    dict(od=1, out=P + 2),                               # narrowed over itself
    dict(xt=0, out=P - 4 * 40),                          # one row for all tokens
    dict(xt=48, ot=24, out=P + 4 * 24),                  # other token strides, spans that meet
    dict(xt=48, ot=48, xh=8, oh=16, out=P + 4 * 24),     # alike token strides, rows of a token together
    dict(tokens=1, xt=0, ot=100, out=P + 4 * 16),
    dict(heads=1, xh=0, oh=100, out=P + 4 * 24),
])
def test_rope_refuses_overlapping_outputs(bad):
    assert rope(**bad) == INVALID


@pytest.mark.parametrize("bad", [
    dict(pos=P), dict(pos=P - 12), dict(pos=P + 4 * 95), dict(freq=P), dict(freq=P - 28), dict(freq=P + 4 * 94),
    dict(ot=-24, pos=P - 4 * 72), dict(oh=-8, freq=P - 4 * 16), dict(ot=40, pos=P + 4 * 30),  # between its rows too
])
def test_rope_refuses_outputs_over_positions_and_frequencies(bad):
    assert rope(**{"x": P + (1 << 20), **bad}) == INVALID


def logits(rows=2, vocab=40, x=P, ldx=40, out=4 * P, ldo=40, **fields):
    p = b.dbs_logits_params(**fields)
    return _lib.dbs_logits_adjust(rows, vocab, x, 0, ldx, bytes(p), out, 0, ldo, None)


HIST = dict(hist_ptr=P, hist=2 * P, hist_len=7)
BIAS = dict(bias_ptr=P, bias_idx=2 * P, bias_val=3 * P, bias_len=7)


@pytest.mark.parametrize("bad", [
    dict(HIST, hist_ptr=4 * P), dict(HIST, hist_ptr=4 * P - 8), dict(HIST, hist=4 * P + 316), dict(HIST, hist=4 * P - 24),
    dict(HIST, hist_new=4 * P - 4), dict(HIST, repetition=4 * P + 316), dict(HIST, frequency=4 * P - 4), dict(HIST, presence=4 * P),
    dict(BIAS, bias_ptr=4 * P + 316), dict(BIAS, bias_idx=4 * P - 24), dict(BIAS, bias_val=4 * P + 100),
    dict(mask=4 * P - 12, ldmask=2), dict(mask=4 * P + 316, ldmask=2), dict(mask=4 * P - 100, ldmask=30),
    dict(ldo=60, mask=4 * P + 200, ldmask=2),  # between the rows
    dict(HIST, out=P), dict(BIAS, out=P, ldo=40),  # in place, over the pointers
])
def test_logits_refuse_outputs_over_their_lists(bad):
    assert logits(**bad) == INVALID
