"""What is measured of the model's two ends: the token embedding and the log
probabilities of tokens, each with its gradient.

Four operators of the library, in calls as a streaming evaluation, a decoder and
a training step make them:

  embed         rows of the embedding table, scaled, for the tokens of a segment
  embed_grad    the table's gradient: for every token the sum of the gradients of
                its occurrences
  logprob       logits of states against the (tied) table, of which only the log
                probability of a given token, the log-sum-exp, the entropy and the
                largest few alternatives are wanted
  logprob_grad  gradients of the states and of the table for gradients of those log
                probabilities (and of the entropies)

``run`` computes each in elementary torch operations, or calls the library when
``own`` is set.  A token or target of -1 stands for none (padding).
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SPARE = 12   # candidates beyond the alternatives asked for, ordered again in 64 bits


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _case(name, op, n, V, d, dtype="bf16", ids="i64", scale=1.0, top=0, ent=False):
    return {"name": name, "op": op, "n": n, "V": V, "d": d, "dtype": dtype, "ids": ids,
            "scale": scale, "top": top, "ent": ent}


def listed():
    return [
        # the next token of eight decoded streams
        _case("embed_token_B8", "embed", 8, 32000, 1024, scale=32.0),
        # prompts of 1600 tokens for 16 streams
        _case("embed_prompt_16x1600", "embed", 25600, 50001, 1024, scale=32.0),
        # a training segment of the character-level stack: every token occurs often
        _case("embed_grad_chars_16x512", "embed_grad", 8192, 204, 512, scale=512 ** 0.5),
        # a word-level segment in single precision, most words absent
        _case("embed_grad_words_f32", "embed_grad", 2047, 10007, 520, dtype="f32", ids="i32"),
        # a large word-level batch
        _case("embed_grad_words_128x512", "embed_grad", 65536, 32000, 1024, scale=32.0),
        # one decoded token: the distribution's largest eight
        _case("logprob_token_B1", "logprob", 1, 32000, 1024, top=8),
        # the nodes of 19 drafted trees of eight, checked against their
        # distributions; an odd vocabulary
        _case("logprob_draft_19x8", "logprob", 152, 50001, 1024, ids="i32", top=4),
        # evaluation of a word-level segment (16 x 128) with a large vocabulary
        _case("logprob_eval_16x128", "logprob", 2048, 131072, 1024),
        # a small check in single precision
        _case("logprob_f32_77", "logprob", 77, 5003, 512, dtype="f32", scale=0.8, top=5),
        # a training segment of the character-level stack, with an entropy term
        _case("logprob_grad_chars_16x512", "logprob_grad", 8192, 204, 512, ent=True),
        # a word-level training segment (16 x 128)
        _case("logprob_grad_words_16x128", "logprob_grad", 2048, 32000, 1024),
        # odd sizes in single precision
        _case("logprob_grad_f32_333", "logprob_grad", 333, 5003, 520, dtype="f32", ids="i32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "logprob", "logprob", "logprob_grad", "logprob_grad"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    d = 8 * _log(rng, 8, 160)
    ids = rng.choice(["i32", "i64"])
    scale = rng.choice([1.0, 0.7, 1.3]) if "logprob" in op else rng.choice([1.0, d ** 0.5])
    if "logprob" not in op:
        n, V = _log(rng, 1, 30000), _log(rng, 2, 50000)
        return {"op": op, "n": n, "V": V, "d": d, "dtype": dtype, "ids": ids, "scale": scale,
                "top": 0, "ent": False}
    most = 4e10 if op == "logprob_grad" else 1e11   # multiply-adds
    if dtype == "f32":
        most = 5e9
    n, V = _log(rng, 1, 5000), _log(rng, 100, 60000)
    while n * V * d > most:
        n, V = max(1, n * 3 // 4), max(100, V * 7 // 8)
    top = rng.choice([0, 1, 3, 8, 16]) if op == "logprob" else 0
    return {"op": op, "n": n, "V": V, "d": d, "dtype": dtype, "ids": ids, "scale": scale,
            "top": top, "ent": op == "logprob_grad" and rng.random() < 0.5}


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    i = 8 if case["ids"] == "i64" else 4
    n, V, d = case["n"], case["V"], case["d"]
    rows, table = n * d * e, V * d * e
    if case["op"] == "embed":
        # each occurring row once: at most n of them, at most the table
        return {"bytes": min(rows, table) + rows + n * i, "flops": 0}
    if case["op"] == "embed_grad":
        return {"bytes": rows + n * i + V * d * 4, "flops": n * d}
    if case["op"] == "logprob":
        return {"bytes": rows + table + n * (i + 12 + 8 * case["top"]), "flops": 2 * n * V * d}
    return {"bytes": 2 * rows + 2 * table + n * (i + 8), "flops": 6 * n * V * d}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

class _State:
    pass


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    n, V, d = case["n"], case["V"], case["d"]
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    st = _State()
    st.case = case
    # tokens as text has them: the r-th most frequent about 1 / r as often as the
    # first; one in twenty is padding
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    rank = (torch.exp(u * math.log(V + 1)) - 1).long().clamp(0, V - 1)
    ids = torch.randperm(V, generator=g, device="cuda")[rank]
    pad = torch.rand(n, generator=g, device="cuda") < 0.05
    ids = torch.where(pad, torch.full_like(ids, -1), ids)
    st.ids = ids.to(torch.int32 if case["ids"] == "i32" else torch.int64)
    if case["op"] == "embed":
        st.emb = (randn(V, d) * 0.02).to(dt)
        st.out = torch.empty(n, d, dtype=dt, device="cuda")
    elif case["op"] == "embed_grad":
        st.dout = (randn(n, d) / n).to(dt)
        st.out = torch.empty(V, d, dtype=torch.float32, device="cuda")
    else:
        # a trained model's logits: of a few units' spread, the text's token raised
        w = randn(V, d) * (2.5 / d ** 0.5)
        lift = w[ids.clamp(min=0)] * (randn(n, 1).abs() * 1.5)
        st.w = w.to(dt)
        st.h = (randn(n, d) + lift).to(dt)
        f32 = dict(dtype=torch.float32, device="cuda")
        if case["op"] == "logprob":
            k = case["top"]
            st.out = {"logp": torch.empty(n, **f32), "lse": torch.empty(n, **f32),
                      "entropy": torch.empty(n, **f32)}
            if k:
                st.out["top_logp"] = torch.empty(n, k, **f32)
                st.out["top_ids"] = torch.empty(n, k, dtype=torch.int32, device="cuda")
        else:
            # the mean negative log probability, weighted; a small entropy term
            st.dlogp = -(0.5 + torch.rand(n, generator=g, device="cuda")) / n
            st.dent = randn(n) * (0.1 / n) if case["ent"] else None
            # what the forward call of the same step left behind
            st.lse, st.entropy = _statistics(case, st)
            st.grads = torch.empty_like(st.h), torch.empty_like(st.w)
    if own:
        import transformer_xl_relative_pos_gb300 as txl
        st.txl = txl
        size = {"embed": lambda: 0,
                "embed_grad": lambda: txl.embed_bwd_workspace_size(n, V, d),
                "logprob": lambda: txl.logprob_fwd_workspace_size(n, V, d, dt, top=case["top"]),
                "logprob_grad": lambda: txl.logprob_bwd_workspace_size(n, V, d, dt)}[case["op"]]()
        st.ws = torch.empty(max(size, 256), dtype=torch.uint8, device="cuda")
    return st


def _statistics(case, st):
    """lse and entropy of the rows in single precision, from sums in 64 bits."""
    z = (st.h.float() @ st.w.float().t()).mul_(case["scale"])
    m = z.amax(1, keepdim=True)
    z -= m
    e = torch.exp(z)
    s = e.sum(1, dtype=torch.float64)
    e *= z
    ent = torch.log(s) - e.sum(1, dtype=torch.float64) / s
    return (m[:, 0].double() + torch.log(s)).float(), ent.float()


# ---------------------------------------------------------------------------
# the operators
# ---------------------------------------------------------------------------

def run(st):
    case = st.case
    op, scale = case["op"], case["scale"]
    if own:
        if op == "embed":
            return st.txl.embed_fwd(st.ids, st.emb, scale=scale, out=st.out)
        if op == "embed_grad":
            return st.txl.embed_bwd(st.dout, st.ids, case["V"], scale=scale, out=st.out,
                                    workspace=st.ws)
        if op == "logprob":
            o = st.out
            st.txl.logprob_fwd(st.h, st.w, st.ids, scale=scale, top=case["top"], workspace=st.ws,
                               out=st.txl.LogProbs(o["logp"], o["lse"], o["entropy"],
                                                   o.get("top_logp"), o.get("top_ids")))
            return o
        dh, dw = st.txl.logprob_bwd(st.h, st.w, st.ids, st.lse, st.dlogp, entropy=st.entropy,
                                    dentropy=st.dent, scale=scale, grads=st.grads, workspace=st.ws)
        return {"dh": dh, "dw": dw}
    return {"embed": _embed, "embed_grad": _embed_grad, "logprob": _logprob,
            "logprob_grad": _logprob_grad}[op](st)


def _embed(st):
    rows = st.emb[st.ids.long().clamp(min=0)].float() * st.case["scale"]
    return torch.where((st.ids >= 0)[:, None], rows, torch.zeros_like(rows)).to(st.emb.dtype)


def _embed_grad(st):
    case = st.case
    sums = torch.zeros(case["V"] + 1, case["d"], dtype=torch.float32, device="cuda")
    ids = torch.where(st.ids >= 0, st.ids.long(), torch.full_like(st.ids, case["V"]).long())
    sums.index_add_(0, ids, st.dout.float())
    return sums[:-1] * case["scale"]


def _logprob(st):
    case = st.case
    k = case["top"]
    z = (st.h.float() @ st.w.float().t()) * case["scale"]
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    s = e.sum(1, keepdim=True)
    lse = (m + torch.log(s))[:, 0]
    ent = torch.log(s)[:, 0] - (e * (z - m)).sum(1) / s[:, 0]
    t = st.ids.long()
    logp = torch.gather(z, 1, t.clamp(min=0)[:, None])[:, 0] - lse
    out = {"logp": torch.where(t >= 0, logp, torch.zeros_like(logp)), "lse": lse, "entropy": ent}
    if k:
        # the order among the largest in 64 bits, equal ones by their index
        cand = torch.sort(torch.topk(z, min(case["V"], k + SPARE), 1)[1], 1)[0]
        best = (st.w.double()[cand] * st.h.double()[:, None]).sum(2) * case["scale"]
        best, order = torch.sort(best, dim=1, descending=True, stable=True)
        out["top_logp"] = (best[:, :k] - lse[:, None].double()).float()
        out["top_ids"] = torch.gather(cand, 1, order[:, :k]).int()
    return out


def _logprob_grad(st):
    case = st.case
    h, w = st.h.float(), st.w.float()
    logp = (h @ w.t()) * case["scale"] - st.lse[:, None]
    p = torch.exp(logp)
    t = st.ids.long()
    gl = torch.where(t >= 0, st.dlogp, torch.zeros_like(st.dlogp))
    G = p * -gl[:, None]
    if st.dent is not None:
        G = G - p * (logp + st.entropy[:, None]) * st.dent[:, None]
    G.scatter_add_(1, t.clamp(min=0)[:, None], gl[:, None])
    G = G * case["scale"]
    return {"dh": (G @ w).to(st.h.dtype), "dw": (G.t() @ h).to(st.w.dtype)}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    """What ``run`` returns, from the definitions in 64 bits: sums over sorted
    tokens, and softmax rows in blocks."""
    if work(case)["flops"] > 8e12:
        return None
    st = prepare(case, seed)
    n, V, scale, k = case["n"], case["V"], case["scale"], case["top"]
    t = st.ids.long()
    if case["op"] == "embed":
        out = torch.zeros(n, case["d"], dtype=torch.float64, device="cuda")
        out[t >= 0] = st.emb.double()[t[t >= 0]] * scale
        return out
    if case["op"] == "embed_grad":
        order = torch.argsort(t, stable=True)
        ends = torch.searchsorted(t[order], torch.arange(-1, V, device="cuda"), right=True)
        upto = torch.cat([torch.zeros(1, case["d"], dtype=torch.float64, device="cuda"),
                          st.dout.double()[order].cumsum(0)])[ends]
        return (upto[1:] - upto[:-1]) * scale
    w = st.w.double()
    block = max(1, min(n, int(1e9) // (8 * V)))
    parts, dw = [], torch.zeros_like(w) if case["op"] == "logprob_grad" else None
    for i in range(0, n, block):
        h, ti = st.h[i:i + block].double(), t[i:i + block]
        z = torch.mm(h, w.t()) * scale
        rows = torch.arange(z.shape[0], device="cuda")[ti >= 0]
        if case["op"] == "logprob":
            lse = torch.logsumexp(z, 1)
            lp = z - lse[:, None]
            logp = torch.zeros_like(lse)
            logp[rows] = lp[rows, ti[rows]]
            part = {"logp": logp, "lse": lse, "entropy": -(lp * torch.exp(lp)).sum(1)}
            if k:
                top, at = torch.sort(lp, dim=1, descending=True, stable=True)
                part["top_logp"], part["top_ids"] = top[:, :k], at[:, :k].int()
        else:
            lp = z - st.lse[i:i + block].double()[:, None]
            onehot = torch.zeros_like(lp)
            onehot[rows, ti[rows]] = 1.0
            gl = (st.dlogp[i:i + block].double() * (ti >= 0))[:, None]
            G = gl * (onehot - torch.exp(lp))
            if st.dent is not None:
                G -= (st.dent[i:i + block].double()[:, None] * torch.exp(lp) *
                      (lp + st.entropy[i:i + block].double()[:, None]))
            part = {"dh": torch.mm(G, w) * scale}
            dw += torch.mm(G.t(), h) * scale
        parts.append(part)
    out = {name: torch.cat([p[name] for p in parts]) for name in parts[0]}
    if dw is not None:
        out["dw"] = dw
    return out
