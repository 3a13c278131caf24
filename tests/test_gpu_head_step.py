"""The operators around the block together, as a training step uses them: rotary positions, the
attention core, layer norm, the head's cross entropy, and back.  Against 64-bit automatic
differentiation; eager, captured and replayed, from two graphs with workspaces of their own.

Tolerance: the chain rounds to bf16 eleven times between its inputs and dqkv (rope, P, att, y; G, dX of
the head, dX of the norm, P, dS, dqkv, rope back), each by at most 2^-8 of its values, so 11 2^-8 of the
result's norm bounds what arrives (the roundings are independent, and the norm only removes components)."""

import pytest
import torch

import fp8_absmax_reduce_gb300 as fq

pytestmark = pytest.mark.gpu

S, HQ, HKV, V, IGN = 256, 4, 2, 1237, -100
T, D = 2 * S, HQ * 128


def inputs(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")
    t = torch.randint(0, V, (T,), generator=g, device="cuda")
    t[::9] = IGN
    return dict(qkv=(0.7 * n(T, (HQ + 2 * HKV) * 128)).bfloat16(), g=(1 + 0.1 * n(D)).bfloat16(), b=(0.1 * n(D)).bfloat16(),
                W=(0.05 * n(V, D)).bfloat16(), t=t, dl=torch.where(t == IGN, 0.0, 1.0 / (t != IGN).sum()),
                pos=torch.stack([torch.arange(T, device="cuda") % S, torch.arange(T, device="cuda") // 16]).int())


class Step:
    """One step's buffers and workspaces, kept as a program keeps them."""

    def __init__(self, i):
        self.i = i
        self.plan = fq.Rope.make(sections=[40, 24])
        e = lambda *s, dt=torch.bfloat16: torch.empty(*s, dtype=dt, device="cuda")
        self.ws_f = e(fq.linear_cross_entropy_fwd_workspace_size(T, D, V), dt=torch.uint8)
        self.ws_b = e(fq.linear_cross_entropy_bwd_workspace_size(T, D, V), dt=torch.uint8)
        self.ws_n = e(fq.layernorm_bwd_workspace_size(T, D), dt=torch.uint8)
        self.ws_a = e(fq.lib.attention_bwd_workspace_size(T, HQ), dt=torch.uint8)

    def run(self):
        i = self.i
        r = fq.rope_fwd(i["qkv"], i["pos"], self.plan, HQ, HKV)
        att, alse = fq.attention_fwd(r, S, HQ, HKV)
        y, mean, rstd = fq.layernorm_fwd(att, i["g"], i["b"])
        loss, lse = fq.linear_cross_entropy_fwd(y, i["W"], i["t"], ws=self.ws_f)
        dy, dW = fq.linear_cross_entropy_bwd(y, i["W"], i["t"], lse, i["dl"], ws=self.ws_b)
        datt, dg, db = fq.layernorm_bwd(dy, att, i["g"], mean, rstd, ws=self.ws_n)
        dr = fq.attention_bwd(r, att, alse, datt, S, HQ, HKV, ws=self.ws_a)
        dqkv = fq.rope_bwd(dr, i["pos"], self.plan, HQ, HKV, dqkv=dr)
        return loss, dW, dg, db, dqkv


def reference(i, plan):
    x = i["qkv"].double().requires_grad_()
    g, b, W = (i[k].double().requires_grad_() for k in ("g", "b", "W"))
    ang = i["pos"].double()[list(plan.axis)].t() * torch.tensor(plan.inv_freq, dtype=torch.float64, device="cuda")
    c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
    h = x.view(T, -1, 128)
    a, bb = h[:, :HQ + HKV, :64], h[:, :HQ + HKV, 64:]
    h = torch.cat([torch.cat([a * c - bb * s, bb * c + a * s], 2), h[:, HQ + HKV:]], 1)
    outs = []
    mask = torch.ones(S, S, dtype=torch.bool, device="cuda").tril()
    for q0 in range(0, T, S):
        q, k, v = h[q0:q0 + S, :HQ], h[q0:q0 + S, HQ:HQ + HKV], h[q0:q0 + S, HQ + HKV:]
        k, v = k.repeat_interleave(HQ // HKV, 1), v.repeat_interleave(HQ // HKV, 1)
        p = torch.softmax((torch.einsum("qhd,khd->hqk", q, k) * 128 ** -0.5).masked_fill(~mask, float("-inf")), 2)
        outs.append(torch.einsum("hqk,khd->qhd", p, v).reshape(S, D))
    att = torch.cat(outs)
    m = att.mean(1, keepdim=True)
    y = (att - m) / torch.sqrt(((att - m) ** 2).mean(1, keepdim=True) + 1e-5) * g + b
    z = y @ W.t()
    keep = i["t"] != IGN
    loss = torch.where(keep, torch.logsumexp(z, 1) - z.gather(1, i["t"].clamp(min=0)[:, None])[:, 0], 0.0)
    (loss * i["dl"].double()).sum().backward()
    return [v.detach() for v in (loss, W.grad, g.grad, b.grad, x.grad)]


def test_step_matches_automatic_differentiation():
    fq.get_status(clear=True)
    step = Step(inputs(0))
    got = step.run()
    torch.cuda.synchronize()
    assert fq.get_status() == 0
    for a, w in zip(got, reference(step.i, step.plan)):
        assert float((a.double() - w).norm() / w.norm()) < 11 * 2.0 ** -8


def test_two_captured_steps_replay_like_eager_ones():
    steps = [Step(inputs(1)), Step(inputs(2))]
    eager = [[t.clone() for t in s.run()] for s in steps]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs, outs = [], []
    with torch.cuda.stream(side):
        for s in steps:
            s.run()
    torch.cuda.current_stream().wait_stream(side)
    for s in steps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(s.run())
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):  # both at once, each with its own workspaces
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for o, e in zip(outs, eager):
        for a, b in zip(o, e):
            assert torch.equal(a, b)


def test_launches_are_traced():
    import ctypes
    step = Step(inputs(3))
    step.run()
    assert fq.lib.fp8q_trace_start(256) == 0
    step.run()
    fq.lib.fp8q_trace_stop()
    torch.cuda.synchronize()
    ms, kinds = (ctypes.c_float * 256)(), (ctypes.c_int * 256)()
    n = fq.lib.fp8q_trace_read(ms, kinds, 256)
    names = [fq.lib.fp8q_kernel_name(kinds[k]).decode() for k in range(n)]
    for want in ("rope", "layernorm_fwd", "layernorm_bwd", "ce_fwd", "ce_bwd"):
        assert want in names
    assert names.count("rope") == 2 and all(ms[k] > 0 for k in range(n))
