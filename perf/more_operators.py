"""Cases for the LM-head cross entropy and for gradient norm and clipping: the same work in plain torch
operations and, with ``own`` set, through the library's entry points.

* ``ce``    softmax cross entropy of hidden states against the output embedding, with label smoothing,
            z-loss and a soft cap of the logits, loss and both gradients in one call, no stored logits
            (``grpo_lmhead_ce_fwd_bwd``)
* ``norm``  the global norm of many gradient tensors, each tensor's own, and the clip's factor
            (``grpo_grad_norm``)
* ``clip``  the norm and the clipped gradients (``grpo_grad_norm``, ``grpo_grad_clip``)
"""
import math

import torch

own = False

V_QWEN = 151936  # the vocabulary of this repository's workloads

_DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def _ce(name, T, V, H, grad=True, smoothing=0.0, z_loss=0.0, cap=0.0, masked=0.0, weights=False):
    return dict(name=name, op="ce", T=T, V=V, H=H, grad=grad, smoothing=smoothing, z_loss=z_loss, cap=cap,
                masked=masked, weights=weights)


def _grads(name, op, layout, n, numel, dtype, out="", odd=False, divisor=0, max_norm=1.0):
    return dict(name=name, op=op, layout=layout, n=n, numel=numel, dtype=dtype, out=out, odd=odd, divisor=divisor,
                max_norm=max_norm)


def listed():
    return [
        # a short sequence on a small head: latency
        _ce("ce few tokens", 16, 32000, 768),
        # extents that are no multiple of a tile, label smoothing, weighted tokens, some padding
        _ce("ce odd sizes", 999, 50257, 1000, smoothing=0.1, masked=0.1, weights=True),
        # evaluation: per-token loss and log-prob of held-out text, no gradient
        _ce("ce evaluation", 2048, V_QWEN, 2048, grad=False),
        # a head with capped logits and a z-loss
        _ce("ce soft cap", 2048, 65536, 1536, cap=30.0, z_loss=1e-4),
        # one micro-batch of supervised fine-tuning, half of its tokens prompt (masked)
        _ce("ce fine-tuning chunk", 8192, V_QWEN, 2048, z_loss=1e-4, masked=0.5),
        # the gradients of a few adapter matrices: latency
        _grads("norm adapters", "norm", "random", 12, 200_000, "f32"),
        # every gradient of a model of 24 layers and its embeddings, bf16
        _grads("norm model bf16", "norm", "layers", 24, 2048, "bf16"),
        # one flat gradient of more than 2^31 elements
        _grads("norm flat past 2^31", "norm", "flat", 1, (1 << 31) + 4099, "bf16"),
        # many small tensors at odd places of their buffer, clipped from the sums of 4096 tokens
        _grads("clip small odd", "clip", "random", 61, 700_000, "f32", "f32", odd=True, divisor=4096),
        # the output embedding's float32 sums clipped into the bf16 gradient that the optimizer takes
        _grads("clip embedding to bf16", "clip", "flat", 1, V_QWEN * 2048, "f32", "bf16", max_norm=0.5),
        # the gradients of 12 layers of 1024 and its embeddings, bf16
        _grads("clip model bf16", "clip", "layers", 12, 1024, "bf16", "bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ce", "norm", "clip"])
    if op == "ce":
        V = _log_int(rng, 500, V_QWEN)
        H = 8 * _log_int(rng, 1, 256)
        c = _ce("", _log_int(rng, 1, 4096), V, H, grad=rng.random() < 0.8, smoothing=rng.choice([0.0, 0.0, 0.1]),
                z_loss=rng.choice([0.0, 1e-4]), cap=rng.choice([0.0, 0.0, 30.0]), masked=rng.choice([0.0, 0.3]),
                weights=rng.random() < 0.4)
    else:
        layout = rng.choice(["random", "flat", "layers"])
        dtype = rng.choice(["bf16", "f32"])
        n, numel = 1, _log_int(rng, 1000, 600_000_000)
        if layout == "random":
            n, numel = rng.randint(2, 300), _log_int(rng, 3000, 300_000_000)
        elif layout == "layers":
            n, numel = rng.randint(1, 24), 64 * rng.randint(1, 20)
        c = _grads("", op, layout, n, numel, dtype, rng.choice(["bf16", "f32"]) if op == "clip" else "",
                   odd=rng.random() < 0.4, divisor=rng.choice([0, 0, 1000]), max_norm=rng.choice([0.5, 1.0, 1e6]))
    del c["name"]
    return c


# ---- inputs ------------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _numels(case):
    """The tensors' sizes, the same for every seed."""
    n, numel = case["n"], case["numel"]
    if case["layout"] == "flat":
        return [numel]
    if case["layout"] == "random":  # spread over two orders of magnitude
        r = torch.rand(n, generator=torch.Generator().manual_seed(n)).mul(4.6).exp()
        return [max(1, int(v)) for v in (r / r.sum() * numel).tolist()]
    d = numel  # layers of width d: the attention's and the MLP's matrices, two norms, then both embeddings
    layer = [d * d, d * d // 4, d * d // 4, d * d, d * d * 11 // 4, d * d * 11 // 4, d * d * 11 // 4, d, d]
    return layer * n + [V_QWEN * d // 4, V_QWEN * d // 4, d]


def _places(case):
    """Each tensor's (first element, size) in its buffer: multiples of 64, or with gaps of odd length."""
    at, got = 0, []
    for k, size in enumerate(_numels(case)):
        if case["odd"]:
            at += 1 + 2 * (k % 5)
        got.append((at, size))
        at += size if case["odd"] else -(-size // 64) * 64
    return got, at


def _normal(n, dtype, std, g):
    buf = torch.empty(n, dtype=dtype, device="cuda")
    step = 1 << 28
    for a in range(0, n, step):
        b = min(n, a + step)
        buf[a:b].copy_(torch.randn(b - a, generator=g, device="cuda") * std)
    return buf


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "ce":
        T, V, H = case["T"], case["V"], case["H"]
        # hidden states and an embedding whose logits have a deviation of about 3; the targets mostly
        # have a larger logit, as a trained model's do
        s["W"] = (torch.randn((V, H), generator=g, device="cuda") * (3.0 / math.sqrt(H))).to(torch.bfloat16)
        s["target"] = torch.randint(V, (T,), generator=g, device="cuda").to(torch.int32)
        towards = s["W"][s["target"].long()].float() * (torch.rand((T, 1), generator=g, device="cuda") * 1.3)
        s["h"] = (torch.randn((T, H), generator=g, device="cuda") + towards).to(torch.bfloat16)
        s["mask"] = None
        if case["masked"]:
            s["mask"] = (torch.rand(T, generator=g, device="cuda") >= case["masked"]).to(torch.uint8)
            s["mask"][0] = 1
        s["w"] = torch.rand(T, generator=g, device="cuda") + 0.5 if case["weights"] else None
        s["scale"] = 1.0 / (T if s["mask"] is None else max(int(s["mask"].sum()), 1))
        s["loss"] = torch.empty(T, device="cuda")
        s["logp"] = torch.empty(T, device="cuda")
        s["d_h"] = torch.empty((T, H), dtype=torch.bfloat16, device="cuda") if case["grad"] else None
        s["dW"] = torch.empty((V, H), dtype=torch.bfloat16, device="cuda") if case["grad"] else None
        s["acc"] = torch.zeros(128, dtype=torch.uint8, device="cuda")  # the step accumulator
        return s
    places, total = _places(case)
    # sums over a step's tokens where the divisor is still to be applied, else gradients of its mean
    std = 2.0 / math.sqrt(total) * max(case["divisor"], 1)
    s["flat"] = _normal(total, _DTYPE[case["dtype"]], std * (0.5 + (seed % 8) / 8), g)
    s["grads"] = [s["flat"][a:a + n] for a, n in places]
    s["tensor_norms"] = torch.empty(len(places), device="cuda")
    s["result"] = torch.zeros(32, dtype=torch.uint8, device="cuda")
    s["acc"] = torch.zeros(128, dtype=torch.uint8, device="cuda")
    s["acc"].view(torch.int64)[5] = case["divisor"]  # as the step's finish leaves it
    if case["op"] == "clip":
        s["out_flat"] = torch.zeros(total, dtype=_DTYPE[case["out"]], device="cuda")
        s["out"] = [s["out_flat"][a:a + n] for a, n in places]
    return s


# ---- the plain forms ---------------------------------------------------------------------------

def _plain_ce(s):
    h, W, cap, eps = s["h"].float(), s["W"].float(), s["cap"], s["smoothing"]
    z = h @ W.T
    if cap:
        z = cap * torch.tanh(z / cap)
    top = z.max(1, keepdim=True).values
    e = (z - top).exp()
    tot = e.sum(1, keepdim=True)
    at = s["target"].long()[:, None]
    logp = (z.gather(1, at) - top) - tot.log()
    lse = top + tot.log()
    loss = -(1.0 - eps) * logp + s["z_loss"] * lse * lse
    if eps:
        loss = loss + eps * (lse - z.mean(1, keepdim=True))
    live = torch.ones_like(lse, dtype=torch.bool) if s["mask"] is None else (s["mask"] != 0)[:, None]
    outs = [torch.where(live, loss, 0.0)[:, 0], torch.where(live, logp, 0.0)[:, 0]]
    if not s["grad"]:
        return outs
    g = torch.where(live, s["scale"] * (1.0 if s["w"] is None else s["w"][:, None]), 0.0)
    dz = e.mul_((1.0 + 2.0 * s["z_loss"] * lse) / tot)
    dz.scatter_add_(1, at, torch.full_like(lse, -(1.0 - eps)))
    if eps:
        dz -= eps / s["V"]
    if cap:
        dz *= 1.0 - (z / cap).square()
    dz *= g
    return outs + [(dz @ W).to(torch.bfloat16), (dz.T @ h).to(torch.bfloat16)]


def _plain_norm(s):
    """The norm, the factor, and each tensor's norm."""
    scale = 1.0 / max(s["divisor"], 1)
    sums = torch.stack([g.float().square().sum(dtype=torch.float64) for g in s["grads"]])
    norm = scale * sums.sum().sqrt()
    coef = scale * torch.where(norm > s["max_norm"], s["max_norm"] / norm, torch.ones_like(norm))
    return [norm.float(), coef.float(), (scale * sums.sqrt()).float()]


def _plain(s):
    if s["op"] == "ce":
        return _plain_ce(s)
    outs = _plain_norm(s)
    if s["op"] == "clip":
        [d.copy_(g.float() * outs[1]) for d, g in zip(s["out"], s["grads"])]
        outs.append(s["out_flat"])
    return outs


# ---- the library's calls -----------------------------------------------------------------------

def _own(s):
    from rl_post_token_gb300 import _lib
    if s["op"] == "ce":
        ws = torch.empty(_lib.grpo_lmhead_ce_workspace_size(s["T"], s["V"], s["H"]), dtype=torch.uint8,
                         device="cuda")
        _lib.grpo_lmhead_ce_fwd_bwd(s["h"], s["W"], s["target"], s["mask"], s["scale"], s["d_h"], s["dW"], s["loss"],
                                    s["acc"], ws, label_smoothing=s["smoothing"], z_loss=s["z_loss"],
                                    soft_cap=s["cap"], w_tok=s["w"], logp_tok=s["logp"])
        return [s["loss"], s["logp"]] + ([s["d_h"], s["dW"]] if s["grad"] else [])
    ws = torch.empty(_lib.grpo_grad_norm_workspace_size(s["grads"]), dtype=torch.uint8, device="cuda")
    _lib.grpo_grad_norm(s["grads"], s["max_norm"], s["result"], ws, tensor_norms=s["tensor_norms"],
                        acc=s["acc"] if s["divisor"] else None, deferred=s["divisor"] > 0)
    norm, coef = s["result"].view(torch.float32)[2:4]
    outs = [norm, coef, s["tensor_norms"]]
    if s["op"] == "clip":
        _lib.grpo_grad_clip(s["grads"], s["result"], out=s["out"])
        outs.append(s["out_flat"])
    return outs


def run(state):
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without -------------------------------------------------------------

def work(case):
    if case["op"] == "ce":
        T, V, H = case["T"], case["V"], case["H"]
        live = T * (1.0 - case["masked"])
        if case["grad"]:
            return {"bytes": 4.0 * (T + V) * H + 17.0 * T, "flops": 6.0 * live * V * H}
        return {"bytes": 2.0 * (live + V) * H + 17.0 * T, "flops": 2.0 * live * V * H}
    numels = _numels(case)
    n = float(sum(numels))
    size = {"bf16": 2, "f32": 4, "": 0}
    return {"bytes": n * (size[case["dtype"]] + size[case["out"]]) + 4.0 * len(numels) + 8,
            "flops": n * (3.0 if case["op"] == "clip" else 2.0)}


# ---- the definitions in 64 bits ----------------------------------------------------------------

def _exact_ce(case, s):
    T, V = case["T"], case["V"]
    W = s["W"].double()
    live = torch.arange(T, device="cuda") if s["mask"] is None else s["mask"].nonzero()[:, 0]
    loss, logp = (torch.zeros(T, dtype=torch.float64, device="cuda") for _ in range(2))
    d_h, dW = torch.zeros_like(s["h"], dtype=torch.float64), torch.zeros_like(W)
    step = max(1, (1 << 27) // V)
    for a in range(0, live.numel(), step):
        t = live[a:a + step]
        x = s["h"][t].double() @ W.T
        x.requires_grad_(case["grad"])
        z = case["cap"] * torch.tanh(x / case["cap"]) if case["cap"] else x
        ls = torch.log_softmax(z, 1)
        lse = torch.logsumexp(z, 1)
        lp = ls.gather(1, s["target"][t].long()[:, None])[:, 0]
        rows = case["smoothing"] * -ls.mean(1) - (1.0 - case["smoothing"]) * lp + case["z_loss"] * lse ** 2
        loss[t], logp[t] = rows.detach(), lp.detach()
        if case["grad"]:
            g = s["scale"] * (1.0 if s["w"] is None else s["w"][t].double())
            (dx,) = torch.autograd.grad((rows * g).sum(), x)
            d_h[t] = dx @ W
            dW += dx.T @ s["h"][t].double()
    return [loss, logp] + ([d_h, dW] if case["grad"] else [])


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "ce":
        return _exact_ce(case, s)
    step = 1 << 26
    parts = [[(g[a:a + step].double() ** 2).sum() for a in range(0, g.numel(), step)] for g in s["grads"]]
    sums = torch.stack([torch.stack(p).sum() for p in parts]) / float(max(case["divisor"], 1)) ** 2
    norm = sums.sum().sqrt()
    factor = float(case["max_norm"] / norm) if float(norm) > case["max_norm"] else 1.0
    factor /= max(case["divisor"], 1)
    outs = [norm, torch.tensor(factor, dtype=torch.float64, device="cuda"), sums.sqrt()]
    if case["op"] == "clip":
        out = torch.zeros(s["flat"].numel(), dtype=torch.float64, device="cuda")
        for a, n in _places(case)[0]:
            out[a:a + n] = s["flat"][a:a + n].double() * factor
        outs.append(out)
    return outs
