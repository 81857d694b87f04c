"""Cases for the scoring and distillation operators: the same work in plain torch operations and,
with ``own`` set, through the library's entry points.

* ``score``    log-probs of given tokens, the entropy and the K most probable tokens of each
               logits row (``grpo_token_topk_logprobs``)
* ``distill``  distillation from a teacher's K top tokens, loss and dlogits in one call
               (``grpo_distill_topk_fwd_bwd``)
* ``lmhead``   the same loss from hidden states and the output embedding, with d_h and dW and no
               stored logits (``grpo_lmhead_distill_topk_fwd_bwd``)
"""
import math

import torch

own = False

FORWARD_TOPK, FORWARD_TAIL, REVERSE_TAIL = 0, 1, 2  # the distillation objectives (_lib.DISTILL_*)
TAIL_MIN = 2.0 ** -24  # a teacher remainder below this cannot be told from zero
V_QWEN = 151936  # the vocabulary of this repository's workloads

_DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def _score(name, T, V, dtype, K, temperature=1.0, pad=0, masked_vocab=0.0, masked_rows=0.0):
    return dict(name=name, op="score", T=T, V=V, dtype=dtype, K=K, temperature=temperature, pad=pad,
                masked_vocab=masked_vocab, masked_rows=masked_rows)


def _distill(name, T, V, dtype, K, kind, temperature=1.0, pad=0, ragged=0.0, masked_rows=0.0, weights=False):
    return dict(name=name, op="distill", T=T, V=V, dtype=dtype, K=K, kind=kind, temperature=temperature, pad=pad,
                ragged=ragged, masked_rows=masked_rows, weights=weights)


def _lmhead(name, T, V, H, K, ragged=0.0, masked_rows=0.0, weights=False):
    return dict(name=name, op="lmhead", T=T, V=V, H=H, K=K, ragged=ragged, masked_rows=masked_rows,
                weights=weights)


def listed():
    return [
        # a server answering one token with its log-prob and alternatives: latency
        _score("score one token", 1, V_QWEN, "bf16", 20),
        # one decoding step of a batch, float32 logits, scored at the sampling temperature
        _score("score decode batch f32", 64, V_QWEN, "f32", 8, temperature=0.7),
        # a vocabulary that is no multiple of a vector (rows unaligned), a tenth of it banned,
        # some rows masked
        _score("score odd vocabulary", 999, 50257, "bf16", 37, masked_vocab=0.1, masked_rows=0.1),
        # a teacher scoring one micro-batch (8 rollouts x 1024 tokens) for a distillation run
        _score("score teacher chunk", 8192, V_QWEN, "bf16", 64),
        # a few tokens: latency of the loss call
        _distill("distill few tokens", 8, V_QWEN, "bf16", 20, FORWARD_TOPK),
        # one micro-batch of a distillation step
        _distill("distill chunk", 8192, V_QWEN, "bf16", 64, FORWARD_TOPK),
        # on-policy distillation: reverse KL, float32 logits
        _distill("distill reverse f32", 2048, V_QWEN, "f32", 128, REVERSE_TAIL),
        # unaligned rows, ragged teacher lists, per-token weights, a raised temperature
        _distill("distill odd vocabulary", 1111, 50257, "bf16", 37, FORWARD_TAIL, temperature=2.0, ragged=0.3,
                 masked_rows=0.1, weights=True),
        # a small step from hidden states, ragged in every extent
        _lmhead("lmhead small", 300, 50257, 1024, 32, ragged=0.3, masked_rows=0.1, weights=True),
        # one micro-batch (2 rollouts x 2048 tokens) from hidden states, the logits never stored
        _lmhead("lmhead chunk", 4096, V_QWEN, 2048, 64),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["score", "distill", "lmhead"])
    if op == "lmhead":
        V = _log_int(rng, 1000, V_QWEN)
        H = 64 * _log_int(rng, 1, 32)
        T = _log_int(rng, 16, 4096)
        c = _lmhead("", T, V, H, rng.randint(1, 128), ragged=rng.choice([0.0, 0.3]),
                    masked_rows=rng.choice([0.0, 0.2]), weights=rng.random() < 0.5)
    else:
        V = _log_int(rng, 200, 200000)
        if rng.random() < 0.5:
            V = max(200, V // 8 * 8)
        dtype = rng.choice(["bf16", "f32"])
        size = 2 if dtype == "bf16" else 4
        T = _log_int(rng, 1, max(1, min(8192, 8192 * V_QWEN * 2 // (V * size))))
        K = min(V, rng.randint(1, 128))
        temperature = rng.choice([1.0, 1.0, 0.6, 1.7])
        pad = rng.choice([0, 0, 1, 8])
        rows = rng.choice([0.0, 0.2])
        if op == "score":
            c = _score("", T, V, dtype, K, temperature, pad, rng.choice([0.0, 0.3]), rows)
        else:
            c = _distill("", T, V, dtype, K, rng.choice([FORWARD_TOPK, FORWARD_TAIL, REVERSE_TAIL]), temperature,
                         pad, rng.choice([0.0, 0.3]), rows, rng.random() < 0.5)
    del c["name"]
    return c


# ---- inputs ------------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rows_mask(T, frac, g):
    """1 for the rows that count; the first row always does."""
    m = (torch.rand(T, generator=g, device="cuda") >= frac).to(torch.uint8)
    m[0] = 1
    return m


def _normal_rows(T, V, pad, dtype, std, g):
    """[T, V] view of a [T, V + pad] buffer of N(0, std) logits."""
    buf = torch.empty((T, V + pad), dtype=dtype, device="cuda")
    for a in range(0, T, 1024):
        b = min(T, a + 1024)
        buf[a:b].copy_(torch.randn((b - a, V + pad), generator=g, device="cuda") * std)
    return buf[:, :V]


def _teacher(T, V, K, ragged, g):
    """A teacher's K top tokens per row (distinct, spread over the vocabulary) and their
    log-probs in descending order, most of the mass on the first few, some of it outside the list.
    Ragged: the tail of some lists is unused (index -1)."""
    width = V // K
    idx = torch.arange(K, device="cuda") * width + torch.randint(width, (T, K), generator=g, device="cuda")
    idx = idx.gather(1, torch.rand((T, K), generator=g, device="cuda").argsort(1))
    u = (2.0 * torch.randn((T, K), generator=g, device="cuda")).sort(1, descending=True).values
    rest = torch.logsumexp(u, 1, keepdim=True) - 2.0 + torch.rand((T, 1), generator=g, device="cuda")
    logp = torch.log_softmax(torch.cat([u, rest], 1), 1)[:, :K]
    if ragged:
        n = torch.randint(1, K + 1, (T, 1), generator=g, device="cuda")
        cut = (torch.rand((T, 1), generator=g, device="cuda") < ragged) & (torch.arange(K, device="cuda") >= n)
        idx, logp = idx.masked_fill(cut, -1), logp.masked_fill(cut, -math.inf)
    return idx.to(torch.int32).contiguous(), logp.contiguous()


def prepare(case, seed):
    g = _gen(seed)
    T, V, K = case["T"], case["V"], case["K"]
    s = dict(case)
    s["mask"] = _rows_mask(T, case["masked_rows"], g)
    if case["op"] == "score":
        z = _normal_rows(T, V, case["pad"], _DTYPE[case["dtype"]], 3.0, g)
        if case["masked_vocab"]:
            banned = torch.rand(V, generator=g, device="cuda") < case["masked_vocab"]
            banned[:K] = False
            z.masked_fill_(banned, -math.inf)
        s["logits"] = z
        s["target"] = torch.randint(K, (T,), generator=g, device="cuda").to(torch.int32)
        if not case["masked_vocab"]:
            s["target"] = torch.randint(V, (T,), generator=g, device="cuda").to(torch.int32)
        for k in ("logp", "entropy"):
            s[k] = torch.empty(T, device="cuda")
        s["top_idx"] = torch.empty((T, K), dtype=torch.int32, device="cuda")
        s["top_logp"] = torch.empty((T, K), device="cuda")
        return s
    s["idx"], s["tlogp"] = _teacher(T, V, K, case["ragged"], g)
    s["w"] = torch.rand(T, generator=g, device="cuda") + 0.5 if case["weights"] else None
    s["scale"] = 1.0 / max(int(s["mask"].sum()), 1)
    s["loss"] = torch.empty(T, device="cuda")
    s["acc"] = torch.zeros(128, dtype=torch.uint8, device="cuda")  # the step accumulator
    if case["op"] == "distill":
        z = _normal_rows(T, V, case["pad"], _DTYPE[case["dtype"]], 3.0, g)
        # the student gives the teacher's tokens most of its mass, in roughly the teacher's order
        base = math.log(V) + 4.5 + 1.5
        lift = (s["tlogp"] + base + 0.5 * torch.randn((T, K), generator=g, device="cuda")) * case["temperature"]
        rows = torch.arange(T, device="cuda")[:, None].expand(T, K)
        used = s["idx"] >= 0
        z[rows[used], s["idx"][used].long()] = lift[used].to(z.dtype)
        s["logits"] = z
        s["dlogits"] = torch.empty((T, V + case["pad"]), dtype=z.dtype, device="cuda")[:, :V]
        return s
    H = case["H"]
    s["h"] = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    s["W"] = (0.02 * torch.randn((V, H), generator=g, device="cuda")).to(torch.bfloat16)
    s["d_h"] = torch.empty((T, H), device="cuda")
    s["dW"] = torch.empty((V, H), device="cuda")
    return s


# ---- the plain forms ---------------------------------------------------------------------------

def _softmax_parts(x):
    """(x - max, exp of it, its row sums) in the type of x."""
    d = x - x.max(1, keepdim=True).values
    e = d.exp()
    return d, e, e.sum(1, keepdim=True)


def _plain_score(s):
    z, V = s["logits"].float(), s["V"]
    d, e, tot = _softmax_parts(z / s["temperature"])
    lp = d - tot.log()
    logp = lp.gather(1, s["target"].long()[:, None])[:, 0]
    entropy = (tot.log() - torch.where(e > 0, e * d, 0.0).sum(1, keepdim=True) / tot)[:, 0]
    # descending logits, ties to the lowest index: one integer key for both
    bits = (z + 0.0).contiguous().view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
    key = (order << 32) + (V - 1 - torch.arange(V, device=z.device))
    idx = V - 1 - (key.topk(s["K"], 1).values & 0xFFFFFFFF)
    live = s["mask"] != 0
    return [torch.where(live, logp, 0.0), torch.where(live, entropy, 0.0),
            torch.where(live[:, None], idx, -1).int(), torch.where(live[:, None], lp.gather(1, idx), -math.inf)]


def _plain_distill(z, s, kind, temperature):
    """(loss per token, dlogits in 32 bits) of float32 logits z."""
    T, V = z.shape
    d, e, tot = _softmax_parts(z / temperature)
    used = s["idx"] >= 0
    at = s["idx"].long()
    slot = torch.where(used, at, V)
    lp = d.gather(1, at.clamp(min=0)) - tot.log()
    p = torch.where(used, lp.exp(), 0.0)
    tlp = torch.where(used, s["tlogp"], -math.inf)
    if kind == FORWARD_TOPK:
        q = tlp.double().exp()
        Q = q.sum(1, keepdim=True)
        some = Q > 0
        lq = tlp.double() - Q.log()
        q = torch.where(some, q / Q, 0.0)
        loss = torch.where(q > 0, q * (lq - lp), 0.0).sum(1)
        alpha, corr = some.double(), torch.where(some, p - q, 0.0)
    else:
        q = tlp.double().exp()
        qr = 1.0 - q.sum(1, keepdim=True)
        outside = torch.ones((T, V + 1), device=z.device).scatter_(1, slot, 0.0)[:, :V]
        pr = ((e * outside).sum(1, keepdim=True) / tot).double()
        none = used.sum(1, keepdim=True) >= V  # nothing outside the list
        if kind == FORWARD_TAIL:
            qr = torch.where((qr < TAIL_MIN) | none, 0.0, qr)
            loss = torch.where(q > 0, q * (tlp - lp.double()), 0.0).sum(1) \
                + torch.where(qr > 0, qr * (qr / pr).log(), 0.0)[:, 0]
            alpha = q.sum(1, keepdim=True) + qr - torch.where(qr > 0, qr / pr, 0.0)
            corr = p * (q.sum(1, keepdim=True) + qr) - q
        else:
            qr = qr.clamp(min=TAIL_MIN)
            f = lp.double() - tlp
            fr = (pr / qr).log()
            tail = (pr > 0) & ~none
            loss = torch.where(p > 0, p * f, 0.0).sum(1) + torch.where(tail, pr * fr, 0.0)[:, 0]
            alpha = torch.where(tail, fr - loss[:, None], 0.0)
            corr = torch.where(p > 0, p * (f - loss[:, None]), 0.0)
    dz = torch.empty((T, V + 1), device=z.device)
    torch.mul(e / tot, alpha.float(), out=dz[:, :V])
    dz.scatter_(1, slot, corr.float())
    live = s["mask"] != 0
    g = torch.where(live, s["scale"] / temperature * (1.0 if s["w"] is None else s["w"]), 0.0)
    return torch.where(live, loss, 0.0).float(), torch.where(live[:, None], dz[:, :V], 0.0) * g[:, None]


def _plain(s):
    if s["op"] == "score":
        return _plain_score(s)
    if s["op"] == "distill":
        loss, dz = _plain_distill(s["logits"].float(), s, s["kind"], s["temperature"])
        return [loss, dz.to(s["logits"].dtype)]
    h, W = s["h"].float(), s["W"].float()
    loss, dz = _plain_distill(h @ W.T, s, FORWARD_TOPK, 1.0)
    return [loss, (dz @ W).to(torch.bfloat16), (dz.T @ h).to(torch.bfloat16)]


# ---- the library's calls -----------------------------------------------------------------------

def _own(s):
    from rl_post_token_gb300 import _lib
    if s["op"] == "score":
        _lib.grpo_token_topk_logprobs(s["logits"], s["K"], target=s["target"], logp_tok=s["logp"],
                                      entropy_tok=s["entropy"], top_idx=s["top_idx"], top_logp=s["top_logp"],
                                      temperature=s["temperature"], mask=s["mask"])
        return [s["logp"], s["entropy"], s["top_idx"], s["top_logp"]]
    if s["op"] == "distill":
        _lib.grpo_distill_topk_fwd_bwd(s["logits"], s["idx"], s["tlogp"], s["mask"], s["kind"], s["scale"],
                                       s["dlogits"], s["loss"], s["acc"], temperature=s["temperature"],
                                       w_tok=s["w"])
        return [s["loss"], s["dlogits"]]
    ws = torch.empty(_lib.grpo_lmhead_distill_workspace_size(s["T"], s["V"], s["H"], s["K"]), dtype=torch.uint8,
                     device="cuda")
    _lib.grpo_lmhead_distill_topk_fwd_bwd(s["h"], s["W"], s["idx"], s["tlogp"], s["mask"], s["scale"], s["d_h"],
                                          s["dW"], s["loss"], s["acc"], ws, w_tok=s["w"])
    # the gradients as a bf16 model keeps them
    return [s["loss"], s["d_h"].to(torch.bfloat16), s["dW"].to(torch.bfloat16)]


def run(state):
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without -------------------------------------------------------------

def work(case):
    T, V, K = case["T"], case["V"], case["K"]
    if case["op"] == "lmhead":
        H = case["H"]
        return {"bytes": 4.0 * (T + V) * H + 8.0 * T * K, "flops": 6.0 * T * V * H}
    es = 2 if case["dtype"] == "bf16" else 4
    rows = T * (1.0 - case["masked_rows"])
    if case["op"] == "score":
        return {"bytes": rows * V * es + T * (8.0 * K + 13), "flops": 4.0 * rows * V}
    return {"bytes": (rows + T) * V * es + T * (8.0 * K + 5), "flops": 6.0 * rows * V}


# ---- the definitions in 64 bits ----------------------------------------------------------------

def _exact_loss(x, idx, tlp, kind):
    """The objective of one block of rows: x float64 scaled logits with a gradient."""
    ls = torch.log_softmax(x, 1)
    n, V = x.shape
    used = idx >= 0
    lp = ls.gather(1, idx.long().clamp(min=0))
    t = tlp.double().masked_fill(~used, -math.inf)
    if kind == FORWARD_TOPK:
        lse = torch.logsumexp(t, 1, keepdim=True)
        lq = torch.where(used & (lse > -math.inf), t - lse, -math.inf)
        on = lq > -math.inf
        return torch.where(on, lq.exp() * (lq.masked_fill(~on, 0.0) - lp.masked_fill(~on, 0.0)), 0.0).sum(1)
    out = torch.ones((n, V + 1), dtype=torch.bool, device=x.device)
    out = out.scatter_(1, torch.where(used, idx.long(), V), False)[:, :V]
    lr = torch.logsumexp(ls.masked_fill(~out, -math.inf), 1)  # log of the student's mass outside
    has = out.any(1) & (lr > -math.inf)
    lr = lr.masked_fill(~has, 0.0)
    qr = 1.0 - torch.where(used, t.exp(), 0.0).sum(1)
    if kind == FORWARD_TAIL:
        on = used & (t > -math.inf)
        a = torch.where(on, t.exp() * (t.masked_fill(~on, 0.0) - lp), 0.0).sum(1)
        keep = (qr >= TAIL_MIN) & out.any(1)
        return a + torch.where(keep, qr * (qr.clamp(min=TAIL_MIN).log() - lr), 0.0)
    a = torch.where(used, lp.exp() * (lp - t.masked_fill(~used, 0.0)), 0.0).sum(1)
    return a + torch.where(has, lr.exp() * (lr - qr.clamp(min=TAIL_MIN).log()), 0.0)


def _exact_rows(z, s, a, b, kind, temperature):
    x = (z.double() / temperature).requires_grad_(True)
    loss = _exact_loss(x, s["idx"][a:b], s["tlogp"][a:b], kind)
    live = s["mask"][a:b] != 0
    weight = torch.where(live, s["scale"] * (1.0 if s["w"] is None else s["w"][a:b].double()), 0.0)
    # d(scale w loss)/dz: x = z / temperature
    (dx,) = torch.autograd.grad((loss * weight).sum(), x)
    return torch.where(live, loss.detach(), 0.0), dx / temperature


def exact(case, seed):
    s = prepare(case, seed)
    T, V = case["T"], case["V"]
    step = max(1, (1 << 27) // V)
    blocks = [(a, min(T, a + step)) for a in range(0, T, step)]
    if case["op"] == "score":
        outs = []
        for a, b in blocks:
            z = s["logits"][a:b].double()
            ls = torch.log_softmax(z / case["temperature"], 1)
            idx = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :case["K"]]
            live = s["mask"][a:b] != 0
            p = ls.exp()
            outs.append([torch.where(live, ls.gather(1, s["target"][a:b].long()[:, None])[:, 0], 0.0),
                         torch.where(live, -torch.where(p > 0, p * ls, 0.0).sum(1), 0.0),
                         torch.where(live[:, None], idx, -1).int(),
                         torch.where(live[:, None], ls.gather(1, idx), -math.inf)])
        return [torch.cat(c) for c in zip(*outs)]
    if case["op"] == "distill":
        dz = torch.empty((T, V), dtype=torch.float64, device="cuda")
        loss = torch.empty(T, dtype=torch.float64, device="cuda")
        for a, b in blocks:
            loss[a:b], dz[a:b] = _exact_rows(s["logits"][a:b], s, a, b, case["kind"], case["temperature"])
        return [loss, dz]
    h, W = s["h"].double(), s["W"].double()
    d_h, dW = torch.empty_like(h), torch.zeros_like(W)
    loss = torch.empty(T, dtype=torch.float64, device="cuda")
    for a, b in blocks:
        loss[a:b], dz = _exact_rows(h[a:b] @ W.T, s, a, b, FORWARD_TOPK, 1.0)
        d_h[a:b] = dz @ W
        dW += dz.T @ h[a:b]
    return [loss, d_h, dW]
