"""Plain 64-bit references (numpy) of the cache of 4-bit keys and values, of the attention over it and of the norm with
rotary positions.  The layout is read from its description in include/dbs.h."""
import numpy as np

from decode_ref import bf16

HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def padded(dim):
    return next(d for d in (64, 96, 128, 192, 256) if d >= dim)


class Cache:
    """Pages of one layer in numpy: `bytes` uint8 [pages, page bytes], written and read token by token."""

    def __init__(self, pages, heads, dim, group, page, fill=None):
        self.pages, self.heads, self.dim, self.group, self.page = pages, heads, dim, group, page
        self.d = padded(dim)
        self.groups = self.d // group
        codes, records = page * self.d // 2, page * self.groups * 4
        self.parts = (0, codes, codes + records, 2 * codes + records)
        self.head_bytes = 2 * (codes + records)
        self.bytes = np.full((pages, heads * self.head_bytes), 0 if fill is None else fill, np.uint8)
        c = np.arange(self.d)
        # nibble addresses of a token's channels, and bytes of its records, from the page's part of a head
        self.key_nibble = lambda t: 8 * (t * (self.d // 8) + c % 32 // 8 * (self.d // 32) + c // 32) + c % 8
        self.value_nibble = lambda t: 2 * self.parts[2] + 8 * (t // 8 * self.d + c % 16 * (self.d // 16) + c // 16) + t % 8
        g = np.arange(self.groups)
        place = {0: 0, 4: 1, 1: 2, 5: 3, 2: 4, 6: 5, 3: 6, 7: 7}
        self.key_record = lambda t: (self.parts[1] + (t * self.groups + g) * 4, 2)
        self.value_record = lambda t: (self.parts[3] + (t // 8 * self.groups + g) * 32 + 2 * place[t % 8], 16)

    def quantize(self, x):
        """Codes [d], s and b [groups] of one head's x [dim] (float32), as the header defines them."""
        q, s, b = np.zeros(self.d, np.uint8), np.zeros(self.groups, np.float16), np.zeros(self.groups, np.float16)
        for g in range(self.groups):
            v = np.asarray(x, np.float32)[g * self.group : (g + 1) * self.group]
            if not len(v):
                continue
            if not (np.abs(v) <= 65024).all():
                s[g] = b[g] = np.nan
                continue
            b[g] = v.min().astype(np.float16)
            s[g] = max((v.max() - np.float32(b[g])) * np.float32(1 / 15), np.float32(0)).astype(np.float16)
            if s[g] > 0:
                t = (v - np.float32(b[g])) * (np.float32(1) / np.float32(s[g]))
                q[g * self.group : g * self.group + len(v)] = np.clip(np.rint(t), 0, 15)
        return q, s, b

    def value(self, q, s, b):
        with np.errstate(invalid="ignore"):
            v = np.repeat(s.astype(np.float64), self.group) * q + np.repeat(b.astype(np.float64), self.group)
            return v.astype(np.float16).astype(np.float64)[: self.dim]

    def _put(self, page, head, nibbles, codes, record, s, b):
        part = self.bytes[page, head * self.head_bytes : (head + 1) * self.head_bytes]
        for n, q in zip(nibbles, codes):
            keep = part[n // 2] & (0x0F if n % 2 else 0xF0)
            part[n // 2] = keep | (q << 4 if n % 2 else q)
        for at, x, y in zip(record[0], s, b):
            part[at : at + 2] = np.frombuffer(x.tobytes(), np.uint8)
            part[at + record[1] : at + record[1] + 2] = np.frombuffer(y.tobytes(), np.uint8)

    def store(self, page, t, head, k, v):
        """Puts one token's key and value; what they now stand for."""
        kq, vq = self.quantize(k), self.quantize(v)
        self._put(page, head, self.key_nibble(t), kq[0], self.key_record(t), *kq[1:])
        self._put(page, head, self.value_nibble(t), vq[0], self.value_record(t), *vq[1:])
        return self.value(*kq), self.value(*vq)

    def _get(self, page, head, nibbles, record):
        part = self.bytes[page, head * self.head_bytes : (head + 1) * self.head_bytes]
        q = (part[nibbles // 2] >> (4 * (nibbles % 2))) & 15
        halves = [np.array([part[a + o : a + o + 2] for a in record[0]]).copy().view(np.float16)[:, 0] for o in (0, record[1])]
        return self.value(q, *halves)

    def read(self, page, t, head):
        return self._get(page, head, self.key_nibble(t), self.key_record(t)), self._get(page, head, self.value_nibble(t), self.value_record(t))


def random_bytes(rng, cache, spread=1.0):
    """Random codes with records of moderate values in every place: what a cache looks like to its readers."""
    cache.bytes[:] = rng.integers(0, 256, cache.bytes.shape)
    for p in range(cache.pages):
        for h in range(cache.heads):
            part = cache.bytes[p, h * cache.head_bytes : (h + 1) * cache.head_bytes]
            for key in (True, False):
                low, high = (cache.parts[1], cache.parts[2]) if key else (cache.parts[3], cache.head_bytes)
                n = (high - low) // 4
                s = (spread * rng.uniform(0.1, 0.3, n)).astype(np.float16)
                b = (spread * rng.uniform(-2.5, -0.5, n)).astype(np.float16)
                both = np.stack((s, b), 1) if key else np.concatenate((s.reshape(-1, 8), b.reshape(-1, 8)), 1)
                part[low:high] = np.frombuffer(both.tobytes(), np.uint8)


def sequence_values(cache, table_row, length):
    """k, v [heads, length, dim] in 64 bits; tokens without a page are NaN."""
    k = np.full((cache.heads, length, cache.dim), np.nan)
    v = k.copy()
    for t in range(length):
        page = table_row[t // cache.page]
        if 0 <= page < cache.pages:
            for h in range(cache.heads):
                k[h, t], v[h, t] = cache.read(page, t % cache.page, h)
    return k, v


def visible(position, length, window, sinks):
    j = np.arange(length)
    see = j <= position
    if window:
        see &= (j > position - window) | (j < sinks)
    return see


def attention(q, k, v, position, scale, window=0, sinks=0, has_page=None):
    """One row in 64 bits: (output, sum of weights times |v|, largest |score| sum) over the tokens that it sees."""
    see = visible(position, k.shape[0], window, sinks)
    if has_page is not None:
        see &= has_page
    if not see.any():
        return np.zeros(v.shape[1]), np.zeros(v.shape[1]), 0.0
    k, v = k[see], v[see]
    s = scale * (k @ q)
    w = np.exp(s - s.max())
    w /= w.sum()
    size = scale * (np.abs(k) @ np.abs(q)).max()
    return w @ v, w @ np.abs(v), size


def attention_tolerance(out, mass, size, dim, tokens, kind, wide):
    """Per element: exponentials as halves (half a step of 2^-10, or two of them: 2^-21, relative; what the half's subnormals lose,
    2^-25 of 2^12 down, is below that for the weights that count and at most 2^-31 of the largest for the others), each of them off
    by its score's rounding in fp32 (dim products, the power of two and the scale: dim + 8 roundings of the size of the sum, in the
    numerator and in the sum) and by the power's own error (2^-22), sums of `tokens` terms in fp32, and the output's rounding."""
    weight = 2.0 ** -21 if wide else 2.0 ** -11
    score = 2 * (dim + 8) * 2.0 ** -24 * size + (2.0 ** -20 * size if wide else 0.0)
    # a product's sum: a term is added to at most tokens / 32 + 64 partial sums on its way
    total = (tokens / 32 + 64 + 16) * 2.0 ** -24 + 2.0 ** -21 + tokens * 2.0 ** -31
    return HALF_STEP[kind] * np.abs(out) + (weight + score + total) * (mass + np.abs(out)) + 1e-30


def norm_rope(x, w, eps, pos, freq, interleaved, scale=1.0):
    """[tokens, heads, dim] in 64 bits, and the size that the error is relative to."""
    x = x.astype(np.float64)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    if w is not None:
        y = y * w.astype(np.float64)
    rot = 2 * len(freq)
    a = (pos.astype(np.float64)[:, None] * freq)[:, None]
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    out, size = y.copy(), np.abs(y)
    u, v = y[..., first], y[..., second]
    out[..., first], out[..., second] = scale * (u * np.cos(a) - v * np.sin(a)), scale * (u * np.sin(a) + v * np.cos(a))
    size[..., first] = size[..., second] = abs(scale) * (np.abs(u) + np.abs(v))
    return out, size


def typed(a, kind):
    """Values rounded to the type, in float32."""
    return bf16(a) if kind == "bf16" else np.asarray(a, np.float32)
