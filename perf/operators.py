"""Cases of the operators around the transformer block that are timed and compared: the softmax
cross entropy of a language model's head, layer norm, and rotary positions, forward and backward.

``run`` computes an operator in its plain form (elementary torch operations in 32 bits, angles in
64) where ``own`` is false, and calls the framework's entry points where it is true.  Both return
the same outputs of the same inputs.  Sizes are those of this repository's workloads (widths 2048,
3584 and 5120, 4096 to 16384 tokens, 40 query and 8 key heads of 128), or generic.
"""

import math
import random

import torch

own = False

IGNORE = -100
LN_EPS = 1e-5
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # scoring a few short answers: the head's weights are read once for a handful of tokens
        {"name": "ce_fwd_answers", "op": "ce_fwd", "T": 24, "d": 2048, "V": 32000},
        # the loss of a held-out batch, a vocabulary that fills no tile
        {"name": "ce_fwd_heldout", "op": "ce_fwd", "T": 4096, "d": 3584, "V": 50257},
        # the head's gradients for a short, ragged micro-batch, with a weight for each token
        {"name": "ce_bwd_ragged", "op": "ce_bwd", "T": 1003, "d": 2048, "V": 50257, "mean": False},
        # the head's gradients in the 7B-class training step
        {"name": "ce_bwd_7b", "op": "ce_bwd", "T": 8192, "d": 3584, "V": 32000, "mean": True},
        # the norm of a few new tokens: latency
        {"name": "ln_fwd_tokens", "op": "ln_fwd", "T": 8, "d": 2048, "dtype": "bf16"},
        # the norm of a whole training batch at the 32B class's width
        {"name": "ln_fwd_32b", "op": "ln_fwd", "T": 16384, "d": 5120, "dtype": "bf16"},
        # its backward at the 7B class's sizes, with the residual branch's gradient
        {"name": "ln_bwd_7b", "op": "ln_bwd", "T": 8192, "d": 3584, "dtype": "bf16", "dres": True},
        # an fp32 residual stream whose width is no multiple of anything
        {"name": "ln_bwd_odd", "op": "ln_bwd", "T": 2047, "d": 1409, "dtype": "f32", "dres": False},
        # one new token for each of 16 running sequences, at far positions
        {"name": "rope_fwd_tokens", "op": "rope_fwd", "T": 16, "hq": 40, "hkv": 8, "dh": 128, "rot": 128,
         "sections": "64", "interleaved": False, "far": 1000000},
        # the 32B class's step: packed sequences of text
        {"name": "rope_fwd_32b", "op": "rope_fwd", "T": 16384, "hq": 40, "hkv": 8, "dh": 128, "rot": 128,
         "sections": "64", "interleaved": False, "far": 0},
        # gradient of images and video between text: positions of time, height and width
        {"name": "rope_bwd_video", "op": "rope_bwd", "T": 9001, "hq": 28, "hkv": 4, "dh": 128, "rot": 128,
         "sections": "16,24,24", "interleaved": False, "far": 0},
        # gradient of a narrow model that rotates half of each head, neighbouring pairs
        {"name": "rope_bwd_partial", "op": "rope_bwd", "T": 4095, "hq": 12, "hkv": 12, "dh": 64, "rot": 32,
         "sections": "16", "interleaved": True, "far": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(["ce_fwd", "ce_bwd", "ln_fwd", "ln_bwd", "rope_fwd", "rope_bwd"])
    if op in ("ce_fwd", "ce_bwd"):
        most = 8192 * 3584 * 32000 // (1 if op == "ce_bwd" else 2)
        while True:
            c = {"op": op, "T": _log(rng, 1, 8192), "d": 8 * _log(rng, 32, 640), "V": _log(rng, 1000, 100000)}
            if c["T"] * c["d"] * c["V"] <= most:
                break
        if op == "ce_bwd":
            c["mean"] = rng.random() < 0.6
        return c
    if op in ("ln_fwd", "ln_bwd"):
        d = 8 * _log(rng, 8, 1024) if rng.random() < 0.7 else _log(rng, 3, 8192)
        c = {"op": op, "T": _log(rng, 1, 16384), "d": d, "dtype": rng.choice(["bf16", "bf16", "f32"])}
        if op == "ln_bwd":
            c["dres"] = rng.random() < 0.5
        return c
    dh = rng.choice([64, 96, 128, 128])
    rot = rng.choice([dh, dh, dh // 2])
    hkv = rng.choice([1, 2, 4, 8])
    half = rot // 2
    if rng.random() < 0.5:
        sections = [half]
    else:
        a = rng.randrange(1, half - 1)
        b = rng.randrange(1, half - a)
        sections = [a, b, half - a - b]
    return {"op": op, "T": _log(rng, 1, 16384), "hq": hkv * rng.choice([1, 2, 5]), "hkv": hkv, "dh": dh, "rot": rot,
            "sections": ",".join(str(s) for s in sections if s), "interleaved": rng.random() < 0.3,
            "far": rng.choice([0, 0, 4000000])}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 13)


def _normal(shape, g, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std


def _ce_inputs(case, seed):
    """Hidden states of unit size that lean toward their target's row by a strength of their own (a
    model part of the way through its training), targets of a few frequent and many rare words, a
    tenth of them ignored."""
    T, d, V = case["T"], case["d"], case["V"]
    g = _gen(seed)
    W = _normal((V, d), g, 0.02).to(torch.bfloat16)
    u = torch.rand((T,), generator=g, device="cuda")
    targets = (torch.exp(u * math.log(V)) - 1).to(torch.int64).clamp_(0, V - 1)
    lean = torch.rand((T, 1), generator=g, device="cuda") * 12.0
    x = _normal((T, d), g)
    x += lean * W[targets].float() / (0.02 * math.sqrt(d))
    x = x.to(torch.bfloat16)
    ignored = torch.rand((T,), generator=g, device="cuda") < 0.1
    ignored[0] = False
    targets[ignored] = IGNORE
    return x, W, targets, g


def _sections(case):
    return [int(s) for s in case["sections"].split(",")]


def _inv_freq(rot):
    return [10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)]


def _positions(case, g):
    """[axes, T] int32: packed sequences of text (one axis), or text and grids of patches (several)."""
    T, axes = case["T"], len(_sections(case))
    t = torch.arange(T, device="cuda", dtype=torch.int64)
    if axes == 1:
        seq = max(1, min(4096, T))
        pos = (t % seq)[None]
    else:
        w, h = 24, 16
        frame = t // (w * h)
        axis = [frame, (t // w) % h + frame, t % w + frame]
        pos = torch.stack(axis[:axes])
    if case["far"]:
        pos = pos + torch.randint(0, case["far"], (1, T), generator=g, device="cuda")
    return pos.to(torch.int32).contiguous()


def prepare(case, seed):
    op = case["op"]
    if op in ("ce_fwd", "ce_bwd"):
        x, W, targets, g = _ce_inputs(case, seed)
        T, d, V = case["T"], case["d"], case["V"]
        s = {"case": case, "x": x, "W": W, "targets": targets}
        if op == "ce_bwd":
            lse = torch.empty(T, device="cuda")
            Wf = W.float()
            step = max(1, (1 << 28) // V)
            for i in range(0, T, step):
                lse[i:i + step] = torch.logsumexp(x[i:i + step].float() @ Wf.t(), dim=1)
            valid = targets >= 0
            weight = torch.full((T,), 1.0, device="cuda")
            if not case["mean"]:
                weight = 0.25 + 1.5 * torch.rand((T,), generator=g, device="cuda")
            s["lse"] = lse
            s["dloss"] = weight / valid.sum()
        if own:
            import fp8_absmax_reduce_gb300 as fq
            need = (fq.linear_cross_entropy_fwd_workspace_size if op == "ce_fwd"
                    else fq.linear_cross_entropy_bwd_workspace_size)(T, d, V)
            s["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda")
        return s
    g = _gen(seed)
    if op in ("ln_fwd", "ln_bwd"):
        T, d, dt = case["T"], case["d"], _DT[case["dtype"]]
        # a residual stream: a few wide channels, a mean of its own for each token
        chan = torch.where(torch.rand((d,), generator=g, device="cuda") < 0.01, 20.0, 1.0)
        x = (_normal((T, d), g) * chan + 0.5 * _normal((T, 1), g)).to(dt)
        s = {"case": case, "x": x, "g": (1.0 + 0.1 * _normal((d,), g)).to(dt), "b": (0.1 * _normal((d,), g)).to(dt)}
        if op == "ln_bwd":
            x64 = x.double()
            mean = x64.mean(dim=1)
            var = ((x64 - mean[:, None]) ** 2).mean(dim=1)
            s["mean"], s["rstd"] = mean.float(), (1.0 / torch.sqrt(var + LN_EPS)).float()
            s["dY"] = _normal((T, d), g, 1e-2).to(dt)
            s["dres"] = _normal((T, d), g, 1e-2).to(dt) if case["dres"] else None
            if own:
                import fp8_absmax_reduce_gb300 as fq
                s["ws"] = torch.empty(fq.layernorm_bwd_workspace_size(T, d), dtype=torch.uint8, device="cuda")
        return s
    heads = case["hq"] + 2 * case["hkv"]
    std = 0.7 if op == "rope_fwd" else 1e-3
    s = {"case": case, "qkv": _normal((case["T"], heads * case["dh"]), g, std).to(torch.bfloat16),
         "pos": _positions(case, g)}
    # the angles' plan, made once by a program: each pair's axis and frequency
    if own:
        import fp8_absmax_reduce_gb300 as fq
        s["rope"] = fq.Rope.make(head_dim=case["dh"], rot_dim=case["rot"], base=10000.0, sections=_sections(case),
                                 interleaved=case["interleaved"])
    else:
        s["axis"] = torch.tensor([a for a, k in enumerate(_sections(case)) for _ in range(k)], device="cuda")
        s["freq"] = torch.tensor(_inv_freq(case["rot"]), dtype=torch.float64, device="cuda")
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def _plain_ce_fwd(s):
    z = s["x"].float() @ s["W"].float().t()
    m = z.max(dim=1, keepdim=True).values
    lse = (m + torch.log(torch.exp(z - m).sum(dim=1, keepdim=True)))[:, 0]
    valid = s["targets"] >= 0
    picked = z.gather(1, s["targets"].clamp(min=0)[:, None])[:, 0]
    loss = torch.where(valid, lse - picked, torch.zeros_like(lse))
    return loss, lse


def _plain_ce_bwd(s):
    x, W = s["x"].float(), s["W"].float()
    p = x @ W.t()
    p -= s["lse"][:, None]
    p = torch.exp_(p)
    valid = s["targets"] >= 0
    rows = torch.arange(p.shape[0], device=p.device)
    p[rows, s["targets"].clamp(min=0)] -= 1.0
    p *= torch.where(valid, s["dloss"], torch.zeros_like(s["dloss"]))[:, None]
    return (p @ W).to(torch.bfloat16), (p.t() @ x).to(torch.bfloat16)


def _plain_ln_fwd(s):
    x = s["x"].float()
    mean = x.mean(dim=1, keepdim=True)
    c = x - mean
    rstd = 1.0 / torch.sqrt((c * c).mean(dim=1, keepdim=True) + LN_EPS)
    y = c * rstd * s["g"].float() + s["b"].float()
    return y.to(s["x"].dtype), mean[:, 0], rstd[:, 0]


def _plain_ln_bwd(s):
    x, dY, g = s["x"].float(), s["dY"].float(), s["g"].float()
    rstd = s["rstd"][:, None]
    xh = (x - s["mean"][:, None]) * rstd
    u = dY * g
    dX = rstd * (u - u.mean(dim=1, keepdim=True) - xh * (u * xh).mean(dim=1, keepdim=True))
    if s["dres"] is not None:
        dX = dX + s["dres"].float()
    return dX.to(s["x"].dtype), (dY * xh).sum(dim=0), dY.sum(dim=0)


def _plain_rope(s, sign):
    case, qkv = s["case"], s["qkv"]
    T, dh, rot = case["T"], case["dh"], case["rot"]
    n = (case["hq"] + case["hkv"]) * dh
    angle = s["pos"].double().t()[:, s["axis"]] * s["freq"]
    cos, sin = torch.cos(angle).float()[:, None, :], (sign * torch.sin(angle)).float()[:, None, :]
    x = qkv[:, :n].float().view(T, -1, dh)
    out = x.clone()
    if case["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        out[..., 0:rot:2], out[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        out[..., :rot // 2], out[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
    return torch.cat([out.view(T, n).to(qkv.dtype), qkv[:, n:]], dim=1)


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if own:
        import fp8_absmax_reduce_gb300 as fq
        if op == "ce_fwd":
            return fq.linear_cross_entropy_fwd(s["x"], s["W"], s["targets"], ignore_index=IGNORE, ws=s["ws"])
        if op == "ce_bwd":
            return fq.linear_cross_entropy_bwd(s["x"], s["W"], s["targets"], s["lse"], s["dloss"], ignore_index=IGNORE,
                                               dw_dtype=torch.bfloat16, ws=s["ws"])
        if op == "ln_fwd":
            return fq.layernorm_fwd(s["x"], s["g"], s["b"], eps=LN_EPS)
        if op == "ln_bwd":
            return fq.layernorm_bwd(s["dY"], s["x"], s["g"], s["mean"], s["rstd"], dres=s["dres"], ws=s["ws"])
        rope = fq.rope_fwd if op == "rope_fwd" else fq.rope_bwd
        return rope(s["qkv"], s["pos"], s["rope"], case["hq"], case["hkv"])
    if op == "ce_fwd":
        return _plain_ce_fwd(s)
    if op == "ce_bwd":
        return _plain_ce_bwd(s)
    if op == "ln_fwd":
        return _plain_ln_fwd(s)
    if op == "ln_bwd":
        return _plain_ln_bwd(s)
    return _plain_rope(s, 1.0 if op == "rope_fwd" else -1.0)


def work(case):
    op = case["op"]
    T = case["T"]
    if op in ("ce_fwd", "ce_bwd"):
        d, V = case["d"], case["V"]
        if op == "ce_fwd":  # x, W, targets in; loss and lse out; the logits
            return {"bytes": 2 * T * d + 2 * V * d + 8 * T + 8 * T, "flops": 2 * T * V * d}
        # x, W, targets, lse, dloss in; dX, dW out; the logits again and the two products of their gradient
        return {"bytes": 4 * T * d + 4 * V * d + 8 * T + 8 * T, "flops": 6 * T * V * d}
    if op in ("ln_fwd", "ln_bwd"):
        d, e = case["d"], 2 if case["dtype"] == "bf16" else 4
        if op == "ln_fwd":
            return {"bytes": 2 * T * d * e + 2 * d * e + 8 * T, "flops": 8 * T * d}
        return {"bytes": (4 if case["dres"] else 3) * T * d * e + d * e + 8 * T + 8 * d, "flops": 16 * T * d}
    heads = case["hq"] + 2 * case["hkv"]
    axes = len(_sections(case))
    return {"bytes": 2 * 2 * T * heads * case["dh"] + 4 * axes * T,
            "flops": 3 * T * (case["hq"] + case["hkv"]) * case["rot"]}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    op = case["op"]
    if op in ("ce_fwd", "ce_bwd") and 6 * case["T"] * case["V"] * case["d"] > 8e12:
        return None
    s = prepare(case, seed)
    if op == "ce_fwd":
        W = s["W"].double()
        loss, lse = [], []
        for xs, ts in zip(s["x"].split(512), s["targets"].split(512)):
            z = torch.einsum("td,vd->tv", xs.double(), W)
            l = torch.logsumexp(z, dim=1)
            own_z = (xs.double() * W[ts.clamp(min=0)]).sum(dim=1)
            loss.append((l - own_z).masked_fill(ts < 0, 0.0))
            lse.append(l)
        return torch.cat(loss), torch.cat(lse)
    if op == "ce_bwd":
        W = s["W"].double()
        dX = torch.zeros_like(s["x"], dtype=torch.float64)
        dW = torch.zeros_like(W)
        for i in range(0, case["T"], 1024):
            xs, ts = s["x"][i:i + 1024].double(), s["targets"][i:i + 1024]
            keep = (ts >= 0).double() * s["dloss"][i:i + 1024].double()
            q = torch.exp(torch.einsum("td,vd->tv", xs, W) - s["lse"][i:i + 1024].double()[:, None]) * keep[:, None]
            q.scatter_add_(1, ts.clamp(min=0)[:, None], -keep[:, None])
            dX[i:i + 1024] = torch.einsum("tv,vd->td", q, W)
            dW += torch.einsum("tv,td->vd", q, xs)
        return dX, dW
    if op == "ln_fwd":
        x = s["x"].double()
        mean = x.sum(dim=1) / case["d"]
        var = ((x - mean[:, None]) ** 2).sum(dim=1) / case["d"]
        rstd = (var + LN_EPS) ** -0.5
        return torch.addcmul(s["b"].double(), (x - mean[:, None]) * rstd[:, None], s["g"].double()), mean, rstd
    if op == "ln_bwd":
        d = case["d"]
        xh = (s["x"].double() - s["mean"].double()[:, None]) * s["rstd"].double()[:, None]
        dY = s["dY"].double()
        u = dY * s["g"].double()
        su, sux = u.sum(dim=1, keepdim=True), (u * xh).sum(dim=1, keepdim=True)
        dX = (d * u - su - xh * sux) * (s["rstd"].double()[:, None] / d)
        if s["dres"] is not None:
            dX += s["dres"].double()
        return dX, torch.einsum("td,td->d", dY, xh), dY.sum(dim=0)
    sign = 1.0 if op == "rope_fwd" else -1.0
    out = s["qkv"].double()
    heads, dh, rot, half = case["hq"] + case["hkv"], case["dh"], case["rot"], case["rot"] // 2
    first = 0
    for a, count in enumerate(_sections(case)):
        for i in range(first, first + count):
            angle = sign * s["pos"][a].double() * 10000.0 ** (-2.0 * i / rot)
            z = torch.polar(torch.ones_like(angle), angle)[:, None]
            lo, hi = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
            v = out[:, :heads * dh].view(case["T"], heads, dh)
            w = torch.complex(v[:, :, lo].contiguous(), v[:, :, hi].contiguous()) * z
            v[:, :, lo], v[:, :, hi] = w.real, w.imag
        first += count
    return out
