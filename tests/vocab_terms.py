"""Inputs on which every bf16 term of an fp32 operand counts, and the gradients as three-term products
give them with one of the terms or products left out.

An fp32 number is t0 + t1 + t2, each the bf16 nearest to what is left.  Here t1 is some 2^-8 and t2 some
2^-17 of t0, all of one sign, so that what is left out does not average over a sum: a lost t2 is 5e-6 of the
result, a lost product of two t1 1.2e-5."""

import math

import torch


def heavy(shape, g):
    """Positive fp32 numbers in [1, 1.26) with large second and third terms."""
    r = lambda lo, hi: torch.randint(lo, hi, shape, generator=g).double()
    t0, t1 = 1 + r(0, 33) / 128, 2.0 ** -9 * (1 + r(120, 128) / 128)
    return t0 + t1 + 26 / 32 * 2.0 ** -17          # (24 bits: exact in fp32)


def terms(x, n=3):
    x, out = x.float(), []
    for _ in range(n):
        t = x.bfloat16().float()
        out.append(t.double())
        x = x - t
    return out


# (weights of products that a three-term product has: 1, 2^-8, 2^-16)
PRODUCTS = [(0, 0), (0, 1), (1, 0), (0, 2), (2, 0), (1, 1)]


def product(a, b, without=()):
    """a b from the terms of both, without some of the products."""
    x, y = terms(a), terms(b)
    return sum(x[i] @ y[j] for i, j in PRODUCTS if (i, j) not in without)


class Uniform:
    """Logits that are all 0 (states and words in other columns), so G is -dlogp / V in every place, with its own
    second and third terms.  All targets are word 0, whose row is zero."""

    def __init__(self, N, V, d, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.h, self.w = torch.zeros(N, d, dtype=torch.float64), torch.zeros(V, d, dtype=torch.float64)
        self.h[:, :d // 2] = heavy((N, d // 2), g)
        self.w[1:, d // 2:] = heavy((V - 1, d // 2), g)
        self.t = torch.zeros(N, dtype=torch.int64)
        self.dlogp = heavy((N,), g)
        self.lse = torch.full((N,), math.log(V)).float()
        self.scale = 1.0
        p = torch.exp(-self.lse.double())
        self.G = -(self.dlogp * p)[:, None].expand(N, V).clone()
        self.G[:, 0] += self.dlogp

    def grads(self, without_h=(), without_w=(), G=None):
        """dh, and dw but for word 0's."""
        G = self.G if G is None else G
        dh = product(G, self.w, without_h) if without_h is not None else G @ self.w
        dw = product(G.t().contiguous(), self.h, without_w) if without_w is not None else G.t() @ self.h
        return dh, dw[1:]

    def exact(self):
        return self.grads(None, None)


class Steep:
    """Logits of 30 or so, of which what is left out is 1.6e-4: as much of every probability.  All targets are word
    0 again; the other words' rows of dw are sums of one sign."""

    def __init__(self, N, V, d, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.h, self.w = heavy((N, d), g), heavy((V, d), g)
        self.scale = 2.0 ** round(math.log2(24 / d))
        self.t = torch.zeros(N, dtype=torch.int64)
        self.dlogp = heavy((N,), g)
        self.z = self.scale * (self.h @ self.w.t())
        self.lse = torch.logsumexp(self.z, 1).float()

    def dw(self, z=None):
        """dw but for word 0's, from logits z."""
        z = self.z if z is None else z
        G = -self.dlogp[:, None] * torch.exp(z - self.lse.double()[:, None])
        return self.scale * (G.t() @ self.h)[1:]


# What of fp32 operands' results may be off, relative to the norm: see test_gpu_logprob_norms.
GRAD_LIMIT, STEEP_LIMIT, LSE_LIMIT = 3e-6, 4e-5, 1e-6

# (powers of two: 1 / V leaves dlogp its terms)
UNIFORM = [(300, 2048, 128), (5, 8192, 208), (700, 128, 264), (100, 4096, 520)]
STEEP = [(300, 2048, 128), (5, 9001, 208), (130, 333, 72), (100, 4096, 520)]


def rel(x, want):
    return float((x.double() - want).norm() / want.norm())
