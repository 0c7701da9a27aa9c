"""Decode-step calls on parts of one buffer that share no element."""
import numpy as np
import pytest

import decode_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dbs():
    import spmspv_graph_traversal_amd as d

    return d


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("tokens", [1, 5, 600])
def test_rope_between_parts_of_one_buffer(dbs, kind, tokens):
    import torch

    rng = np.random.default_rng(tokens)
    pos, freq = rng.integers(0, 5000, tokens).astype(np.int32), 10000.0 ** (-np.arange(16) / 16)
    p, f = torch.from_numpy(pos).cuda(), torch.from_numpy(freq).cuda()

    def views(b):  # x and out in a buffer of [tokens, 8 * 32]
        heads = b.view(tokens, 8, 32)
        halves = b.view(tokens, 4, 2, 32)
        yield heads[:, :3], heads[:, 3:6]          # one part of a row into another
        yield heads[:, 5:], heads[:, 1:4]
        yield halves[:, :, 0], halves[:, :, 1]     # every other head
        yield heads[:, ::2], heads[:, 1::2]
        yield heads[:, :1].expand(tokens, 4, 32), heads[:, 4:]  # one head for several
        if tokens > 1:
            yield b[: tokens // 2].view(-1, 8, 32), b[tokens - tokens // 2:].view(-1, 8, 32)
            yield b[0:tokens - 1:2].view(-1, 8, 32), b[1::2].view(-1, 8, 32)  # every other token

    start = rng.standard_normal((tokens, 256)).astype(np.float32)
    buffer = torch.from_numpy(start).cuda()
    buffer = buffer.bfloat16() if kind == "bf16" else buffer
    for k, (x, out) in enumerate(views(buffer)):
        before, x64 = buffer.clone(), x.double().cpu().numpy()
        n = x.shape[0]
        dbs.dbs_rope(x, p[:n], f, out)
        expect = ref.rope(x64, pos[:n], freq, False)
        # as in test_rope: 12 half steps of fp32 on 2 max|x|, then the output's rounding
        tol = 12 * ref.U24 * 2 * np.abs(x64).max() + ref.HALF_STEP[kind] * np.abs(expect)
        assert (np.abs(out.double().cpu().numpy() - expect) <= tol).all(), k
        got = out.clone()
        out.copy_(torch.zeros_like(out))
        rest = buffer.clone()
        out.copy_(got)
        kept = before.clone()
        for (_, o), i in zip(views(kept), range(k + 1)):
            if i == k:
                o.zero_()
        assert torch.equal(rest, kept), k  # nothing but out has changed
