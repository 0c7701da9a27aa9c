"""Plain 64-bit references (numpy) of the decode-step operators, and inputs for them."""
import numpy as np

U24 = 2.0 ** -24  # half a step of fp32, relative
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def bf16_bits(a):
    """fp32/fp64 values rounded to nearest even bf16, as uint16 bits (finite values)."""
    u = np.asarray(a, np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def bf16(a):
    """Values rounded to bf16, as float32."""
    return (bf16_bits(a).astype(np.uint32) << 16).view(np.float32)


class Q4:
    """Random codes, scales and zero points of an m x n matrix; `w` is W in 64 bits.

    exact=True draws power-of-two scales, so that products with small integers are exact in fp32."""

    def __init__(self, rng, m, n, group, zeros, scales="bf16", exact=True):
        self.m, self.n, self.group, self.scale_type = m, n, group, scales
        groups = -(-n // group)
        self.q = rng.integers(0, 16, (m, n)).astype(np.uint8)
        self.s = (2.0 ** -rng.integers(0, 4, (m, groups)) if exact else rng.uniform(0.004, 0.012, (m, groups))).astype(np.float32)
        if scales == "bf16":
            self.s = bf16(self.s)
        self.z = rng.integers(0, 16, (m, groups)).astype(np.uint8) if zeros else None
        self.of = np.arange(n) // group

    @property
    def codes(self):
        q = self.q if self.n % 2 == 0 else np.concatenate([self.q, np.full((self.m, 1), 9, np.uint8)], 1)
        return q[:, 0::2] | (q[:, 1::2] << 4)  # the unused nibble of an odd n holds anything

    @property
    def offset(self):
        return np.full((self.m, len(self.of)), 8.0) if self.z is None else self.z.astype(np.float64)[:, self.of]

    @property
    def scale(self):
        return self.s.astype(np.float64)[:, self.of]

    @property
    def w(self):
        return (self.q.astype(np.float64) - self.offset) * self.scale

    def build(self, dbs):
        import torch

        s = torch.from_numpy(self.s)
        if self.scale_type == "bf16":
            s = s.bfloat16()
        z = None if self.z is None else torch.from_numpy(self.z).cuda()
        return dbs.dbs_q4_build(self.m, self.n, self.group, torch.from_numpy(np.ascontiguousarray(self.codes)).cuda(),
                                s.cuda(), z)

    def bound(self, x):
        """Bound on the error of fp32 sums of W x, x [T, n]: the codes may be read with an offset of 16 that is
        subtracted as a multiple of the sum of x, so the summed magnitudes are s (16 + q) |x| and s (16 + z) |x|;
        a sum of d terms in any order is off by at most d half steps of the summed magnitudes (x in three parts:
        3 d); d <= 128 within a group, 3 roundings for its scaling, then one per group of the row."""
        mag = (np.abs(16.0 + self.q) + 16.0 + self.offset) * np.abs(self.scale)
        d = 3 * 128 + 3 + self.s.shape[1]
        return d * U24 * (np.abs(x).astype(np.float64) @ mag.T)


def dot(w, x):
    """x [T, n] @ w.T with infinities and NaN spreading as in the sum (no BLAS shortcuts)."""
    with np.errstate(invalid="ignore", over="ignore"):
        return np.stack([np.array([(w * r).sum(1)]).reshape(-1) for r in np.asarray(x, np.float64)]) if len(x) else np.zeros((0, w.shape[0]))


def act(kind, g):
    with np.errstate(over="ignore", invalid="ignore"):
        if kind == 0:
            return g / (1 + np.exp(-g))
        if kind == 1:
            return 0.5 * g * (1 + np.tanh(np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)))
        return np.where(g > 0, g, np.where(np.isnan(g), g, 0.0))


def mask_words(allowed):
    """bool [rows, width] -> int32 words, bit v % 32 of word v // 32."""
    rows, width = allowed.shape
    words = (width + 31) // 32
    bits = np.zeros((rows, words * 32), np.uint64)
    bits[:, :width] = allowed
    w = (bits.reshape(rows, words, 32) << np.arange(32, dtype=np.uint64)).sum(-1)
    return w.astype(np.uint32).view(np.int32)


def logits(l, hist=None, new=None, rep=None, freq=None, pres=None, bias=None, allowed=None):
    """Row by row, entry by entry: l [B, V] float64; hist and bias are lists of per-row lists."""
    out = np.array(l, np.float64)
    vocab = out.shape[1]
    for b in range(out.shape[0]):
        if hist is not None:
            start = max(0, new[b]) if new is not None else 0
            ids = [int(v) for v in hist[b]]
            for v in sorted({v for v in ids if 0 <= v < vocab}):
                c = sum(1 for k, i in enumerate(ids) if i == v and k >= start)
                if rep is not None:
                    out[b, v] = out[b, v] / float(rep[b]) if out[b, v] > 0 else out[b, v] * float(rep[b])
                out[b, v] -= (float(freq[b]) if freq is not None else 0.0) * c
                if c and pres is not None:
                    out[b, v] -= float(pres[b])
        if bias is not None:
            for v, value in {int(v): float(x) for v, x in bias[b]}.items():
                if 0 <= v < vocab:
                    out[b, v] += value
        if allowed is not None:
            out[b, ~allowed[b]] = -np.inf
    return out


def rope(x, pos, freq, interleaved, scale=1.0, inverse=False):
    x = np.array(x, np.float64)
    half = len(freq)
    angle = np.asarray(pos, np.float64)[:, None] * np.asarray(freq, np.float64)
    c, s = scale * np.cos(angle)[:, None], scale * np.sin(angle)[:, None]
    if inverse:
        s = -s
    ia = np.arange(0, 2 * half, 2) if interleaved else np.arange(half)
    ib = ia + 1 if interleaved else ia + half
    out = x.copy()
    out[..., ia], out[..., ib] = x[..., ia] * c - x[..., ib] * s, x[..., ia] * s + x[..., ib] * c
    return out
