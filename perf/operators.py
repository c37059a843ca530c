"""The language-model operators at the two ends of the stack of linear layers: what is measured.

Token embedding and its per-sample gradient, softmax cross entropy of a vocabulary head
that keeps no logits, and distillation from a teacher's top logits.  ``run`` computes
each in its plain form (elementary torch operations in 32 bits), or, with ``own`` set,
through the library's entry points; ``exact`` is the definition in 64 bits.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases ---------------------------------------------------------------------------

def listed():
    return [
        # one short micro-batch through a small head: launch latency counts
        dict(name="head_small", op="head", N=64, d=256, V=1000, dtype="bf16", mask=0.0, dH=True, dW=False),
        # validation loss of a masked-language-model head (vocabulary not a multiple of 8), no gradient
        dict(name="head_eval", op="head", N=2048, d=1024, V=50265, dtype="bf16", mask=0.0, dH=False, dW=False),
        # the 7B slice's batch (16 x 512 tokens, width 4096) with a frozen head: Gout of the last block
        dict(name="head_frozen_7b", op="head", N=8192, d=4096, V=32000, dtype="bf16", mask=0.0, dH=True, dW=False),
        # a trained head with half the tokens masked out of the loss
        dict(name="head_train_masked", op="head", N=8192, d=1024, V=50265, dtype="bf16", mask=0.5, dH=True, dW=True),
        # fp32 training of a small model, sizes off every tile
        dict(name="head_f32", op="head", N=509, d=764, V=10007, dtype="f32", mask=0.1, dH=True, dW=True),
        # a few rows of a small classifier-sized vocabulary in fp32: latency
        dict(name="distill_small", op="distill", N=16, V=1000, K=8, dtype="f32", mask=0.0, tau=1.0),
        # fine-tuning batch, 32 teacher entries a token, odd vocabulary, some tokens masked
        dict(name="distill_odd", op="distill", N=4096, V=50265, K=32, dtype="bf16", mask=0.15, tau=2.0),
        # a large vocabulary at the 7B slice's token count
        dict(name="distill_large", op="distill", N=8192, V=128000, K=64, dtype="bf16", mask=0.0, tau=1.0),
        # a short prompt's lookup from a bf16 table: latency
        dict(name="embed_small", op="embed", N=64, d=256, V=1000, table="bf16", out="bf16", mask=0.0),
        # the 7B slice's first input from its fp32 master table
        dict(name="embed_7b", op="embed", N=8192, d=4096, V=32000, table="f32", out="bf16", mask=0.0),
        # embedding gradient of the 7B slice's batch, 16 samples of 512 tokens
        dict(name="embed_grad_7b", op="embed_grad", B=16, T=512, d=4096, V=32000, dtype="bf16", mask=0.0),
        # long context: 8 samples of 8192 tokens, a tenth of them padding
        dict(name="embed_grad_long", op="embed_grad", B=8, T=8192, d=1024, V=50265, dtype="bf16", mask=0.1),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("head", "head", "distill", "embed", "embed_grad"))
    mask = rng.choice((0.0, 0.0, 0.1, 0.5, 0.9))
    if op == "head":
        dtype = "f32" if rng.random() < 0.2 else "bf16"
        limit = 4e9 if dtype == "f32" else 8192 * 4096 * 32000 / 2
        while True:
            N, V = _log(rng, 1, 8192), _log(rng, 500, 64000)
            d = _log(rng, 48, 4096)
            if rng.random() < 0.7:
                d = max(64, d // 64 * 64)
            if N * d * V <= limit:
                break
        return dict(op=op, N=N, d=d, V=V, dtype=dtype, mask=mask, dH=rng.random() < 0.8, dW=rng.random() < 0.4)
    if op == "distill":
        dtype = rng.choice(("bf16", "bf16", "f32"))
        while True:
            N, V = _log(rng, 1, 8192), _log(rng, 200, 131072)
            if N * V * (4 if dtype == "f32" else 2) <= 8192 * 128000 * 2:
                break
        return dict(op=op, N=N, V=V, K=_log(rng, 1, 128), dtype=dtype, mask=mask, tau=rng.choice((1.0, 2.0, 0.7)))
    d = _log(rng, 24, 4096)
    if rng.random() < 0.7:
        d = max(32, d // 32 * 32)
    if op == "embed":
        return dict(op=op, N=_log(rng, 1, 8192), d=d, V=_log(rng, 100, 32000), mask=mask,
                    table=rng.choice(("f32", "bf16")), out=rng.choice(("f32", "bf16")))
    while True:
        B, T, V = _log(rng, 1, 64), _log(rng, 1, 8192), _log(rng, 100, 64000)
        if B * T <= 65536 and B * T * d * 2 + V * d * 4 <= 4.5e8:
            break
    return dict(op=op, B=B, T=T, d=d, V=V, dtype=rng.choice(("bf16", "bf16", "f32")), mask=mask)


# ---- inputs ---------------------------------------------------------------------------

def _tokens(g, n, V, mask):
    """Token numbers with the frequencies of text (the v-th commonest in proportion to 1/v), a
    `mask` share of them -1: padding, or tokens without a loss."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    t = (torch.exp(u * math.log(V + 1)).long() - 1).clamp_(0, V - 1)
    if mask:
        t[torch.rand(n, generator=g, device="cuda") < mask] = -1
    return t


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    op, s = case["op"], {"case": dict(case)}
    if op == "head":
        N, d, V, dt = case["N"], case["d"], case["V"], DT[case["dtype"]]
        W = normal(V, d) * (2.5 / math.sqrt(d))
        labels = _tokens(g, N, V, case["mask"])
        # hidden rows that lean towards their token's weights by a varying amount, as a trained model's do
        lean = 3.0 * torch.rand(N, 1, generator=g, device="cuda") / 2.5
        s["H"] = (normal(N, d) + lean * W[labels.clamp(min=0)]).to(dt)
        s["W"], s["labels"] = W.to(dt), labels
        s["weights"] = 0.1 + 0.9 * torch.rand(N, generator=g, device="cuda")   # a sample's factor per token
    elif op == "distill":
        N, V, K, dt = case["N"], case["V"], case["K"], DT[case["dtype"]]
        start = torch.randint(V, (N, 1), generator=g, device="cuda")
        K = min(K, V)
        idx = (start + torch.arange(K, device="cuda") * max(1, V // K)) % V
        val = normal(N, K) - 0.15 * torch.arange(K, device="cuda") + 9.0
        logits = torch.empty(N, V, dtype=dt, device="cuda").normal_(0.0, 2.0, generator=g)
        logits.scatter_(1, idx, (val + normal(N, K)).to(dt))   # the student is near its teacher
        kept = torch.randint(1, K + 1, (N, 1), generator=g, device="cuda")
        idx = torch.where(torch.arange(K, device="cuda") < kept, idx, torch.full_like(idx, -1))
        weights = 0.1 + 0.9 * torch.rand(N, generator=g, device="cuda")
        weights[torch.rand(N, generator=g, device="cuda") < case["mask"]] = 0.0
        s.update(logits=logits, idx=idx.int(), val=val, weights=weights)
    elif op == "embed":
        s["table"] = normal(case["V"], case["d"]).to(DT[case["table"]])
        s["ids"] = _tokens(g, case["N"], case["V"], case["mask"])
        s["scale"] = math.sqrt(case["d"])
    else:
        B, T, d = case["B"], case["T"], case["d"]
        s["ids"] = _tokens(g, B * T, case["V"], case["mask"]).view(B, T)
        s["G"] = normal(B, T, d).mul_(0.05).to(DT[case["dtype"]])
        s["weights"] = 0.1 + 0.9 * torch.rand(B, generator=g, device="cuda")   # clip factors
        s["scale"] = math.sqrt(d)
    return s


# ---- one pass ---------------------------------------------------------------------------

def _head_plain(s, case):
    H, W, labels = s["H"], s["W"], s["labels"]
    live = ((labels >= 0) & (labels < W.shape[0])).nonzero()[:, 0]
    h, w, t, f = H[live].float(), W.float(), labels[live], s["weights"][live]
    z = h @ w.T
    rows = torch.arange(t.numel(), device=t.device)
    m = z.amax(1, keepdim=True) if t.numel() else z[:, :1]
    e = torch.exp(z - m)
    tot = e.sum(1, keepdim=True)
    loss = torch.zeros(H.shape[0], device=H.device)
    loss[live] = f * (m[:, 0] + torch.log(tot[:, 0]) - z[rows, t])
    out = {"loss": loss}
    if case["dH"] or case["dW"]:
        dz = e / tot
        dz[rows, t] -= 1.0
        dz *= f[:, None]
        if case["dH"]:
            out["dH"] = torch.zeros_like(H)
            out["dH"][live] = (dz @ w).to(H.dtype)
        if case["dW"]:
            out["dW"] = (dz.T @ h).to(W.dtype)
    return out


def _distill_plain(s, case):
    z, idx, tau = s["logits"].float() / case["tau"], s["idx"].long(), case["tau"]
    there = idx >= 0
    q = torch.where(there, s["val"] / tau, torch.full_like(s["val"], -math.inf))
    q = torch.exp(q - q.amax(1, keepdim=True))
    q = q / q.sum(1, keepdim=True)
    m = z.amax(1, keepdim=True)
    lse = m + torch.log(torch.exp(z - m).sum(1, keepdim=True))
    at = idx.clamp(min=0)
    logp = torch.gather(z, 1, at) - lse
    f = s["weights"]
    kl = torch.where(q > 0, q * (torch.log(q) - logp), torch.zeros_like(q)).sum(1)
    dz = torch.exp(z - lse)
    dz.scatter_add_(1, at, -q)
    dz *= (tau * f)[:, None]
    return {"loss": tau * tau * f * kl, "Gout": dz.to(s["logits"].dtype)}


def _embed_plain(s, case):
    ids = s["ids"]
    there = (ids >= 0) & (ids < case["V"])
    rows = s["table"][torch.where(there, ids, torch.zeros_like(ids))].float() * s["scale"]
    return {"out": torch.where(there[:, None], rows, torch.zeros_like(rows)).to(DT[case["out"]])}


def _embed_grad_plain(s, case):
    B, T, d, V, ids = case["B"], case["T"], case["d"], case["V"], s["ids"].reshape(-1)
    at = ((ids >= 0) & (ids < V)).nonzero()[:, 0]
    G = s["G"].reshape(B * T, d)[at].float() * s["scale"]
    sample = at // T
    runs, run_of = torch.unique(sample * V + ids[at], return_inverse=True)
    sums = torch.zeros(runs.numel(), d, device=ids.device).index_add_(0, run_of, G)
    sq = torch.zeros(B, device=ids.device).index_add_(0, runs // V, (sums * sums).sum(1))
    grad = torch.zeros(V, d, device=ids.device)
    grad.index_add_(0, runs % V, sums * s["weights"][runs // V][:, None])
    order = torch.argsort(torch.where((ids >= 0) & (ids < V), ids, torch.full_like(ids, V)), stable=True)
    return {"order": order.int(), "sqnorms": sq, "grad": grad}


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        from random_gradient_projection_b200 import lm
        if op == "head":
            r = lm.head_loss(s["H"], s["W"], s["labels"], weights=s["weights"], grad=case["dH"],
                             weight_grad=case["dW"])
            out = {"loss": r.loss}
            if case["dH"]:
                out["dH"] = r.dH
            if case["dW"]:
                out["dW"] = r.dW
            return out
        if op == "distill":
            loss, Gout = lm.distill_loss(s["logits"], s["idx"], s["val"], weights=s["weights"],
                                         temperature=case["tau"])
            return {"loss": loss, "Gout": Gout}
        if op == "embed":
            return {"out": lm.embed(s["table"], s["ids"], scale=s["scale"], dtype=case["out"])}
        order = lm.embed_order(s["ids"], case["V"])
        sq = lm.embed_sqnorms(order, s["G"], scale=s["scale"])
        grad = lm.embed_grad(order, s["G"], weights=s["weights"], scale=s["scale"])
        return {"order": order.positions, "sqnorms": sq, "grad": grad}
    if op == "head":
        return _head_plain(s, case)
    if op == "distill":
        return _distill_plain(s, case)
    if op == "embed":
        return _embed_plain(s, case)
    return _embed_grad_plain(s, case)


# ---- the definition in 64 bits -----------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "head":
        labels, V = s["labels"], case["V"]
        keep = (labels >= 0) & (labels < V)
        H, W = s["H"].double(), s["W"].double()
        f = torch.where(keep, s["weights"].double(), torch.zeros((), dtype=torch.float64, device="cuda"))
        loss = torch.zeros(case["N"], dtype=torch.float64, device="cuda")
        dH, dW = torch.zeros_like(H), torch.zeros_like(W)
        for a in range(0, case["N"], 2048):   # rows in pieces: the 64-bit logits of all of them are large
            z = H[a:a + 2048] @ W.T
            t = labels[a:a + 2048].clamp(0, V - 1)[:, None]
            logp = torch.log_softmax(z, 1)
            loss[a:a + 2048] = -f[a:a + 2048] * logp.gather(1, t)[:, 0]
            dz = f[a:a + 2048, None] * (logp.exp() - torch.zeros_like(z).scatter_(1, t, 1.0))
            if case["dH"]:
                dH[a:a + 2048] = dz @ W
            if case["dW"]:
                dW += dz.T @ H[a:a + 2048]
        out = {"loss": loss}
        if case["dH"]:
            out["dH"] = dH
        if case["dW"]:
            out["dW"] = dW
        return out
    if op == "distill":
        tau, V = case["tau"], case["V"]
        losses, grads = [], []
        for a in range(0, case["N"], 1024):
            idx, val = s["idx"][a:a + 1024].long(), s["val"][a:a + 1024].double()
            f = s["weights"][a:a + 1024].double()
            q = torch.softmax((val / tau).masked_fill(idx < 0, -math.inf), 1)
            logp = torch.log_softmax(s["logits"][a:a + 1024].double() / tau, 1)
            at = idx.clamp(min=0)
            losses.append(tau ** 2 * f * (torch.special.xlogy(q, q) - q * logp.gather(1, at)).sum(1))
            grads.append((tau * f[:, None] * (logp.exp() - torch.zeros_like(logp).scatter_add_(1, at, q))).float())
        return {"loss": torch.cat(losses), "Gout": torch.cat(grads)}
    if op == "embed":
        ids = s["ids"]
        there = ((ids >= 0) & (ids < case["V"])).double()[:, None]
        return {"out": s["table"].double()[ids.clamp(0, case["V"] - 1)] * (s["scale"] * there)}
    B, V = case["B"], case["V"]
    grad = torch.zeros(V, case["d"], dtype=torch.float64, device="cuda")
    sq = torch.zeros(B, dtype=torch.float64, device="cuda")
    for b in range(B):   # sample by sample: its whole table gradient, then the norm
        ids = s["ids"][b]
        there = ((ids >= 0) & (ids < V)).double()[:, None]
        mine = torch.zeros_like(grad).index_add_(0, ids.clamp(0, V - 1), s["G"][b].double() * (s["scale"] * there))
        sq[b] = torch.linalg.vector_norm(mine) ** 2
        grad += s["weights"][b].double() * mine
    return {"order": None, "sqnorms": sq, "grad": grad}


# ---- what a pass cannot do without ---------------------------------------------------------

def _distinct(n, V):
    """How many different tokens n draws of `_tokens` hold, on average."""
    c = 1.0 / math.log(V + 1)
    return sum(1.0 - (1.0 - c * math.log((v + 2) / (v + 1))) ** n for v in range(V))


def work(case):
    op, live = case["op"], 1.0 - case["mask"]
    if op == "head":
        N, d, V, el = case["N"], case["d"], case["V"], 4 if case["dtype"] == "f32" else 2
        wide = live * N * d * el + V * d * el + N * 16
        if case["dH"]:
            wide += N * d * el
        if case["dW"]:
            wide += V * d * el
        return {"bytes": wide, "flops": 2.0 * live * N * d * V * (1 + case["dH"] + case["dW"])}
    if op == "distill":
        N, V, el = case["N"], case["V"], 4 if case["dtype"] == "f32" else 2
        return {"bytes": (1.0 + live) * N * V * el + N * (case["K"] * 8 + 8), "flops": 6.0 * live * N * V}
    el = {"f32": 4, "bf16": 2}
    if op == "embed":
        N, d = case["N"], case["d"]
        rows = _distinct(live * N, case["V"])
        return {"bytes": rows * d * el[case["table"]] + N * d * el[case["out"]] + 8 * N, "flops": live * N * d}
    n, d = case["B"] * case["T"], case["d"]
    return {"bytes": live * n * d * el[case["dtype"]] + case["V"] * d * 4 + n * 12, "flops": 4.0 * live * n * d}
