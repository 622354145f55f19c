"""The token embedding, the log probabilities of tokens and their gradients in 64
bits, straight from the formulas, with bounds for what fp32 sums and bf16 roundings
may be off.

Bounds.  A sum of n products in fp32, in any order and with each addition cut
rather than rounded, is off by at most n 2^-23 sum|a b|.  A rounding to bf16 is off
by at most 2^-8 of the value, one to fp32 by 2^-24."""

import torch

BF16_HALF = 2.0 ** -8
F32_CUT = 2.0 ** -23


def tokens_with_padding(n, V, g, pad=0.2, dtype=torch.int64):
    ids = torch.randint(0, V, (n,), generator=g)
    ids[torch.rand(n, generator=g) < pad] = -1
    return ids.to(dtype)


def embed(tokens, emb, scale):
    t = tokens.long()
    out = torch.zeros(*t.shape, emb.shape[1], dtype=torch.float64)
    out[t >= 0] = emb.double()[t[t >= 0]] * scale
    return out


def embed_grad(dout, tokens, V, scale):
    """The gradient and the sum of its terms' sizes."""
    t = tokens.long().reshape(-1)
    g = dout.double().reshape(len(t), dout.shape[-1])
    out = torch.zeros(V, g.shape[1], dtype=torch.float64)
    size = torch.zeros_like(out)
    for i in range(len(t)):
        if t[i] >= 0:
            out[t[i]] += g[i] * scale
            size[t[i]] += (g[i] * scale).abs()
    return out, size


def f32(x):
    """The value a float argument of the C interface takes."""
    return float(torch.tensor(x, dtype=torch.float32).double())


class LogProb:
    """Statistics of softmax(scale h w^T) in 64 bits, and bounds of their errors in fp32."""

    def __init__(self, h, w, targets, scale, top, products=1):
        h, w = h.double().reshape(-1, h.shape[-1]), w.double()
        scale = f32(scale)
        self.h, self.w, self.scale = h, w, scale
        self.z = z = scale * (h @ w.t())
        self.t = None if targets is None else targets.long().reshape(-1)
        self.lse = torch.logsumexp(z, 1)
        self.lp = z - self.lse[:, None]
        self.p = torch.exp(self.lp)
        self.entropy = -torch.where(self.p > 0, self.p * self.lp, torch.zeros_like(z)).sum(1)
        n, V, d = z.shape[0], z.shape[1], h.shape[1]
        if self.t is not None:
            self.logp = torch.where(self.t >= 0, self.lp.gather(1, self.t.clamp(min=0)[:, None])[:, 0],
                                    torch.zeros(n, dtype=torch.float64))
        _, ids = torch.sort(z, dim=1, descending=True, stable=True)
        self.top_ids = ids[:, :top]
        self.top_logp = self.lp.gather(1, self.top_ids)
        # a logit: its products' sum (of `products` sums where operands are split into terms),
        # the conversion to log2 units and back (three roundings of the value)
        size = abs(scale) * (h.abs() @ w.abs().t()).amax(1)
        self.z_off = products * d * F32_CUT * size + 3 * F32_CUT * z.abs().amax(1)
        # the sums of exponentials: each of 2^-21 (the exponential, the difference it is taken
        # of), summed 32 at a time, then over at most V / 32 groups
        self.s_off = 2.0 ** -21 + (32 + V / 32) * F32_CUT + 2 * self.z_off
        self.lse_off = self.z_off + self.s_off + F32_CUT * self.lse.abs()
        self.logp_off = 2 * self.z_off + self.s_off + F32_CUT * self.lp.abs().amax(1)
        # sum p (z - mean): terms of at most the logits' range
        span = z.amax(1) - z.amin(1) + 1
        self.ent_off = 2 * self.s_off * span + 4 * F32_CUT * span

    def grads(self, dlogp, dentropy, entropy=None, lse=None):
        """dh, dw and the sizes of their terms' sums: sum |G| |w|, sum |G| |h|."""
        ent = self.entropy if entropy is None else entropy.double()
        lp = self.z - (self.lse if lse is None else lse.double())[:, None]
        p = torch.exp(lp)
        n, V = lp.shape
        G = torch.zeros(n, V, dtype=torch.float64)
        part = torch.zeros(n, dtype=torch.bool)
        if self.t is not None:
            on = self.t >= 0
            part |= on
            gl = torch.where(on, dlogp.double(), torch.zeros(n, dtype=torch.float64))
            G -= p * gl[:, None]
            rows = torch.arange(n)[on]
            G[rows, self.t[on]] += gl[on]
        if dentropy is not None:
            part |= dentropy != 0
            G -= dentropy.double()[:, None] * p * (lp + ent[:, None])
        G[~part] = 0
        h = torch.where(part[:, None], self.h, torch.zeros_like(self.h))
        s = self.scale
        self.G = G
        # sizes without the cancellation inside G: |g| (1[j = t] + p) + |e| p (|log p| + H)
        size = torch.zeros(n, V, dtype=torch.float64)
        if self.t is not None:
            size += p * gl.abs()[:, None]
            size[rows, self.t[on]] += gl.abs()[on]
        if dentropy is not None:
            size += dentropy.double().abs()[:, None] * p * (lp.abs() + ent.abs()[:, None])
        size[~part] = 0
        return (s * G @ self.w, s * G.t() @ h, abs(s) * G.abs() @ self.w.abs(),
                abs(s) * G.abs().t() @ h.abs(), abs(s) * size @ self.w.abs(), abs(s) * size.t() @ h.abs())
