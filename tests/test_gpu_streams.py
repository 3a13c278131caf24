"""Calls on another stream than the current one (``stream=``), with everything that a call can allocate left to it.

Each entry point is called on a stream that is still busy, so that its kernels run after the call has returned and the
current stream has gone on: memory that the call took or dropped must not be handed out by either stream's allocator while
the other still uses it.  Inputs are ready before, outputs are waited for, as the documentation asks."""

import pytest
import torch

import fp8_absmax_reduce_gb300 as fq

pytestmark = pytest.mark.gpu

BUSY = 20_000_000  # clock cycles, about 10 ms


def _tensors(out):
    if isinstance(out, torch.Tensor):
        return [out]
    return [t for o in out if o is not None for t in _tensors(o)]


def _calls():
    g = torch.Generator(device="cuda").manual_seed(5)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")
    T, d, V = 256, 512, 3001
    x, dY, gain, bias = n(T, d).bfloat16(), n(T, d).bfloat16(), n(d).bfloat16(), n(d).bfloat16()
    W = (0.05 * n(V, d)).bfloat16()
    t = torch.randint(0, V, (T,), generator=g, device="cuda")
    dl = torch.full((T,), 1.0 / T, device="cuda")
    q, scal = fq.fp8_quantize_absmax(x)
    qw, sw = fq.fp8_quantize_absmax(W[:512].contiguous())
    (qr, sr), _ = fq.mx_quantize(x)
    _, _, rr = fq.rmsnorm_quant(x, gain)
    _, mean, rstd = fq.layernorm_fwd(x, gain, bias)
    _, lse = fq.linear_cross_entropy_fwd(x, W, t)
    dN = n(T, d)
    qkv, pos, plan = n(T, 8 * 128).bfloat16(), torch.arange(T, device="cuda").int(), fq.Rope.make()
    att, alse = fq.attention_fwd(qkv, T, 4, 2)
    datt = n(T, 4 * 128).bfloat16()
    H = n(T, 2 * d).bfloat16()
    return {
        "fp8_quantize_absmax": lambda **k: fq.fp8_quantize_absmax(x, **k),
        "fp8_gemm_scaled": lambda **k: fq.fp8_gemm_scaled(fq.NT, q, fq.E4M3, qw, fq.E4M3, scal[2:3], sw[2:3], **k),
        "mx_quantize": lambda **k: fq.mx_quantize(x, **k),
        "fp8_gemm_mx": lambda **k: fq.fp8_gemm_mx(fq.NT, qr, fq.E4M3, sr, qr, fq.E4M3, sr, **k),
        "rmsnorm_quant": lambda **k: fq.rmsnorm_quant(x, gain, **k),
        "rmsnorm_bwd": lambda **k: fq.rmsnorm_bwd(dN, x, dY, gain, rr, **k),
        "swiglu_quant": lambda **k: fq.swiglu_quant(H, **k),
        "attention_fwd": lambda **k: fq.attention_fwd(qkv, T, 4, 2, **k),
        "attention_bwd": lambda **k: fq.attention_bwd(qkv, att, alse, datt, T, 4, 2, **k),
        "rope_fwd": lambda **k: fq.rope_fwd(qkv, pos, plan, 4, 2, **k),
        "rope_bwd": lambda **k: fq.rope_bwd(qkv, pos, plan, 4, 2, **k),
        "layernorm_fwd": lambda **k: fq.layernorm_fwd(x, gain, bias, **k),
        "layernorm_bwd": lambda **k: fq.layernorm_bwd(dY, x, gain, mean, rstd, dres=dY, **k),
        "linear_cross_entropy_fwd": lambda **k: fq.linear_cross_entropy_fwd(x, W, t, **k),
        "linear_cross_entropy_bwd": lambda **k: fq.linear_cross_entropy_bwd(x, W, t, lse, dl, **k),
    }, {"fp8_quantize_absmax": fq.lib.fp8_quantize_absmax_workspace_size(T * d), "rmsnorm_quant": fq.lib.rmsnorm_quant_workspace_size(T, d),
        "rmsnorm_bwd": fq.lib.rmsnorm_bwd_workspace_size(T, d), "swiglu_quant": fq.lib.swiglu_quant_workspace_size(T, d),
        "attention_bwd": fq.lib.attention_bwd_workspace_size(T, 4), "layernorm_bwd": fq.layernorm_bwd_workspace_size(T, d),
        "linear_cross_entropy_fwd": fq.linear_cross_entropy_fwd_workspace_size(T, d, V),
        "linear_cross_entropy_bwd": fq.linear_cross_entropy_bwd_workspace_size(T, d, V)}


NAMES = ["fp8_quantize_absmax", "fp8_gemm_scaled", "mx_quantize", "fp8_gemm_mx", "rmsnorm_quant", "rmsnorm_bwd", "swiglu_quant",
         "attention_fwd", "attention_bwd", "rope_fwd", "rope_bwd", "layernorm_fwd", "layernorm_bwd", "linear_cross_entropy_fwd",
         "linear_cross_entropy_bwd"]


@pytest.fixture(scope="module")
def calls():
    c = _calls()
    torch.cuda.synchronize()
    assert sorted(c[0]) == sorted(NAMES)
    return c


def _busy(s):
    with torch.cuda.stream(s):
        torch.cuda._sleep(BUSY)


@pytest.mark.parametrize("name", NAMES)
def test_what_a_call_allocates_belongs_to_its_stream(calls, name):
    call, ws = calls[0][name], calls[1].get(name, 0)
    want = [t.clone() for t in _tensors(call())]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    _busy(s)
    out = _tensors(call(stream=s))
    # the current stream goes on at once, with memory of the sizes that the call has dropped
    junk = [torch.full((ws,), 0xA5, dtype=torch.uint8, device="cuda") for _ in range(3) if ws]
    torch.cuda.synchronize()
    assert all(bool((j == 0xA5).all()) for j in junk)
    assert len(out) == len(want) and all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("name", NAMES)
def test_outputs_may_be_dropped_while_the_current_stream_reads_them(calls, name):
    call = calls[0][name]
    want = [t.clone() for t in _tensors(call())]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = _tensors(call(stream=s))
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(BUSY)
    copies = [t.clone() for t in out]
    sizes = [t.nbytes for t in out]
    del out
    with torch.cuda.stream(s):
        junk = [torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda") for n in sizes]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(copies, want)) and len(junk) == len(want)


@pytest.mark.parametrize("name", NAMES)
def test_memory_that_the_current_stream_still_reads_is_not_taken(calls, name):
    call, ws = calls[0][name], calls[1].get(name, 0)
    want = [t.clone() for t in _tensors(call())]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    held = [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda") for n in [t.nbytes for t in want] + [max(ws, 1)]]
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    copies = [h.clone() for h in held]  # after the sleep; the originals are free for the current stream's allocator
    del held
    out = _tensors(call(stream=s))
    torch.cuda.synchronize()
    assert all(bool((c == 0x5A).all()) for c in copies)
    assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_the_current_stream_given_as_such():
    x = torch.randn(64, 512, device="cuda").bfloat16()
    g = torch.ones(512, device="cuda").bfloat16()
    want = fq.layernorm_fwd(x, g)
    got = fq.layernorm_fwd(x, g, stream=torch.cuda.current_stream())
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", NAMES)
def test_captured_on_a_side_stream_and_replayed(calls, name):
    call = calls[0][name]
    want = [t.clone() for t in _tensors(call())]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        out = _tensors(call(stream=side))
        torch.cuda.current_stream().wait_stream(side)
    for o in out:
        o.zero_()
    for _ in range(2):
        graph.replay()
    junk = [torch.full((t.nbytes,), 0xA5, dtype=torch.uint8, device="cuda") for t in want]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want)) and all(bool((j == 0xA5).all()) for j in junk)
