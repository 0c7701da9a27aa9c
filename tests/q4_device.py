"""Random 4-bit matrices and vectors made on the GPU, whose products are exact in fp32 in any order of summing."""
import torch


class Q4:
    """Random codes, power-of-two scales and zero points of an m x n matrix; `w` is W in 64 bits."""

    def __init__(self, seed, m, n, group, zeros, scales, halvings=3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.m, self.n, self.group = m, n, group
        groups = -(-n // group)
        self.codes = torch.randint(0, 256, (m, (n + 1) // 2), device="cuda", generator=g, dtype=torch.uint8)
        self.scales = 2.0 ** -torch.randint(0, halvings + 1, (m, groups), device="cuda", generator=g).float()
        self.scales = self.scales.to(torch.bfloat16 if scales == "bf16" else torch.float32)
        self.zeros = torch.randint(0, 16, (m, groups), device="cuda", generator=g, dtype=torch.uint8) if zeros else None

    @property
    def w(self):
        q = torch.stack((self.codes & 15, self.codes >> 4), -1).view(self.m, -1)[:, :self.n].double()
        of = torch.arange(self.n, device="cuda") // self.group
        return (q - (8.0 if self.zeros is None else self.zeros.double()[:, of])) * self.scales.double()[:, of]

    def build(self, dbs):
        return dbs.dbs_q4_build(self.m, self.n, self.group, self.codes, self.scales, self.zeros)


def small(seed, tokens, n, kind):
    """Integers from -4 to 4, the last columns not 0.  Up to 34000 products of them with |q - z| <= 15 and scales of
    1 to 1/8 have a sum of fewer than 24 bits (34000 * 15 * 4 * 8 < 2^24), as has each group's sum with 16 + q."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randint(-4, 5, (tokens, n), device="cuda", generator=g).float()
    x[:, -3:] = 3.0
    return x.to(torch.bfloat16 if kind == "bf16" else torch.float32)


def wide(seed, tokens, n):
    """fp32 vectors of four odd integers of 17 bits and zeros.  Bits 16, 8 and 0 are set, so that each of the three bf16 parts of
    eight bits that the kernels cut them into holds something.  Their products with |q - z| <= 15 and scales of 1 and 1/2 have a sum of at most 24 bits (4 * 15 * 2^17 * 2 < 2^24), as
    have the sums with 16 + q of the first parts (multiples of 2^9) and of the others (below 2^9)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    at = torch.rand(tokens, n, device="cuda", generator=g).topk(min(4, n)).indices
    at[:, 0] = torch.arange(tokens, device="cuda") * 37 % n  # tokens together all over the columns
    value = torch.randint(1 << 16, 1 << 17, at.shape, device="cuda", generator=g) | 257
    value *= 2 * torch.randint(0, 2, at.shape, device="cuda", generator=g) - 1
    return torch.zeros(tokens, n, device="cuda").scatter_(1, at, value.float())


def open_rows(words, m):
    row = torch.arange(m, device=words.device)
    return (words[:, row // 32] >> (row % 32)) & 1 != 0


def check_products(dbs, seed, m, n, tokens, group, zeros, scales, gated, x, halvings=3):
    """The plain and the masked product, or the gated one, of x against 64 bits: bit for bit."""
    w = Q4(seed, m, n, group, zeros, scales, halvings)
    A, g = w.build(dbs), x.double() @ w.w.t()
    y = torch.full((tokens, m), 7.0, device="cuda")
    if gated:
        u = Q4(seed + 1, m, n, group, zeros, scales, halvings)
        dbs.dbs_q4_gated(A, u.build(dbs), x, dbs.DBS_ACT_RELU, y)
        assert torch.equal(y, (g.clamp_min(0) * (x.double() @ u.w.t())).float())
        return
    dbs.dbs_q4_product(A, x, y)
    assert torch.equal(y.double(), g)
    words = torch.randint(-2 ** 31, 2 ** 31, (tokens, (m + 31) // 32), device="cuda", dtype=torch.int64,
                          generator=torch.Generator(device="cuda").manual_seed(seed)).int()
    words[:, : words.shape[1] // 3] = 0  # workgroups with nothing to do
    dbs.dbs_q4_product_masked(A, x, words, y)
    assert torch.equal(y.double(), torch.where(open_rows(words, m), g, -torch.inf))
