"""A plain 64-bit model of attention for trees of drafted tokens over a paged
memory, with an error bound for each output ("Transformer-XL: Attentive Language
Models Beyond a Fixed-Length Context", §3.3 score; distances by depth).

The bound, for an implementation that sums in fp32 (u = 2^-24 the half step of
fp32; sums of the tensor cores may drop bits instead of rounding, hence 2 u):
  * a score is two sums of 64 products with q and two with the biases:
      E_ij <= 2 u * 132 * scale * (sum |q + u||k| + sum |q + v||r| + the biases' parts)
    and 4 u |A_ij| for the scalings to log2 units and back;
  * a probability then carries the factor exp(+-2 max_j E_ij), exp2's own error (2^-22)
    and, on the bf16 path, 2^-16 for being held as two bf16 values, or, in trees of more
    than 16 nodes, 2^-8 for being rounded to one (half a step of bf16, relative);
  * the sums over K keys, 16 at a time, add (K / 16 + 64) 2 u;
so |out - want| <= half a step of the output type + (those) * sum_j p_j |v_j|, and
|lse - want| <= max E + 2^-22 + (K / 16 + 64) 2 u + 4 u |lse|.
"""

import numpy as np
import torch

U = 2.0 ** -24
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def f64(t):
    return t.detach().cpu().double().numpy()


def memory_rows(mem, layer, b):
    """Keys and values [H, fill, 64] of sequence b, and which rows lie in known pages."""
    begin, fill = int(mem.begin[b]), int(mem.fill[b])
    x = (begin + torch.arange(fill)) % mem.rows
    page = mem.table[b].cpu()[x // mem.page_rows].long()
    known = (page >= 0) & (page < mem.n_pages)
    page = torch.where(known, page, torch.zeros_like(page))
    k, v = (mem.pool[2 * layer + i].cpu()[page, :, x % mem.page_rows] for i in range(2))
    return f64(k).transpose(1, 0, 2), f64(v).transpose(1, 0, 2), known.numpy()


def depths_and_ancestors(par):
    n = len(par)
    depth, anc = np.zeros(n, dtype=int), np.zeros((n, n), dtype=bool)
    for i in range(n):
        anc[i, i] = True
        if 0 <= par[i] < i:
            depth[i] = depth[par[i]] + 1
            anc[i] |= anc[par[i]]
    return depth, anc


def tree_attention(q, k_new, v_new, mem, layer, r, u, vb, parents, scale, counts):
    """(out, lse, out_bound, lse_bound), NaN in the rows that a call leaves alone."""
    B, H, N, dh = q.shape
    q, kn, vn, r, u, vb = map(f64, (q, k_new, v_new, r, u, vb))
    par = np.broadcast_to(parents.cpu().numpy(), (B, N))
    half = HALF_STEP[mem.pool.dtype]
    extra = 2.0 ** -22
    if mem.pool.dtype == torch.bfloat16:
        extra += 2.0 ** -16 if N <= 16 else 2.0 ** -8
    res = [np.full(s, np.nan) for s in ((B, H, N, dh), (B, H, N)) * 2]
    out, lse, out_b, lse_b = res
    R = r.shape[1]
    for b in range(B):
        n = min(max(int(counts[b]), 0), N)
        mk, mv, known = memory_rows(mem, layer, b)
        F = mk.shape[1]
        depth, anc = depths_and_ancestors(par[b, :n])
        dist = np.concatenate([F + depth[:, None] - np.arange(F), depth[:, None] - depth], 1)
        seen = np.concatenate([np.broadcast_to(known, (n, F)), anc], 1) & (dist < R)
        row = np.clip(R - 1 - dist, 0, R - 1)
        for h in range(H):
            k = np.concatenate([mk[h], kn[b, h, :n]])
            v = np.concatenate([mv[h], vn[b, h, :n]])
            for i in range(n):
                at = seen[i]
                if not at.any():
                    out[b, h, i], lse[b, h, i], out_b[b, h, i], lse_b[b, h, i] = 0, -np.inf, 0, 0
                    continue
                ki, vi, ri = k[at], v[at], r[h, row[i, at]]
                qi = q[b, h, i]
                a = scale * (ki @ (qi + u[h]) + ri @ (qi + vb[h]))
                size = abs(scale) * (np.abs(ki) @ (np.abs(qi) + np.abs(u[h])) +
                                     np.abs(ri) @ (np.abs(qi) + np.abs(vb[h])))
                E = np.max(2 * U * 132 * size + 4 * U * np.abs(a))
                m = a.max()
                p = np.exp(a - m)
                s = p.sum()
                p /= s
                sums = (len(a) / 16 + 64) * 2 * U
                out[b, h, i] = p @ vi
                lse[b, h, i] = m + np.log(s)
                out_b[b, h, i] = half * np.abs(out[b, h, i]) + (2 * E + extra + sums) * (p @ np.abs(vi))
                lse_b[b, h, i] = E + 2.0 ** -22 + sums + 4 * U * abs(lse[b, h, i])
    return out, lse, out_b, lse_b
