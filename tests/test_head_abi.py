"""Refusals of layer norm, rotary positions and the head's cross entropy, without a GPU: the C entry
points return the documented codes before they touch the device, and the Python entry points raise."""

import copy
import ctypes
import dataclasses
import fractions
import os
import pickle
import shutil
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 6
FAKE, ODD = 1 << 20, (1 << 20) + 2
BF16, F32 = 0, 1


@pytest.fixture(scope="module")
def fq():
    import fp8_absmax_reduce_gb300 as fq
    from fp8_absmax_reduce_gb300 import build as b
    b.build()
    fq.load_library()
    return fq


def test_layernorm_refuses(fq):
    def fwd(x=FAKE, dt=BF16, g=FAKE, b=FAKE, T=4, d=24, eps=1e-5, y=FAKE, mean=FAKE, rstd=FAKE):
        return fq.lib.layernorm_fwd(x, dt, g, b, T, d, eps, y, mean, rstd, None)
    for bad in (dict(x=None), dict(x=ODD), dict(g=None), dict(b=ODD), dict(y=ODD), dict(mean=None), dict(rstd=ODD), dict(T=0),
                dict(T=(1 << 28) + 1), dict(d=0), dict(d=16385), dict(dt=2), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf"))):
        assert fwd(**bad) == INVALID, bad
    need = fq.layernorm_bwd_workspace_size(4, 24)
    assert need > 0 and need % 256 == 0 and fq.layernorm_bwd_workspace_size(0, 24) == 0

    def bwd(dY=FAKE, x=FAKE, dt=BF16, g=FAKE, mean=FAKE, rstd=FAKE, dres=None, T=4, d=24, dX=FAKE, dg=FAKE, db=FAKE, ws=FAKE,
            n=need):
        return fq.lib.layernorm_bwd(dY, x, dt, g, mean, rstd, dres, T, d, dX, dg, db, ws, n, None)
    for bad in (dict(dY=ODD), dict(x=None), dict(g=ODD), dict(mean=ODD), dict(rstd=None), dict(dres=ODD), dict(T=0), dict(d=16385),
                dict(dX=None), dict(dg=None), dict(db=ODD), dict(dt=7)):
        assert bwd(**bad) == INVALID, bad
    for bad in (dict(ws=None), dict(ws=FAKE + 16), dict(n=need - 1)):
        assert bwd(**bad) == WORKSPACE, bad


def test_rope_refuses(fq):
    def call(x=FAKE, dt=BF16, T=4, hq=2, hkv=1, pos=FAKE, out=1 << 24, null=False, **kw):
        r = fq.FP8QRope(head_dim=64, rot_dim=32, n_axes=2, interleaved=0)
        r.inv_freq[:16] = [1.0] * 16
        r.axis[:16] = [0] * 8 + [1] * 8
        for k, v in kw.items():
            if k in ("inv_freq", "axis"):
                getattr(r, k)[15] = v
            else:
                setattr(r, k, v)
        got = [f(x, dt, T, hq, hkv, None if null else ctypes.byref(r), pos, out, None)
               for f in (fq.lib.rope_fwd, fq.lib.rope_bwd)]
        assert got[0] == got[1]
        return got[0]
    for bad in (dict(x=None), dict(x=ODD), dict(out=ODD), dict(pos=None), dict(pos=ODD), dict(dt=3), dict(T=0), dict(hq=0),
                dict(hkv=-1), dict(hq=1025), dict(null=True), dict(rot_dim=31), dict(rot_dim=66), dict(rot_dim=0),
                dict(n_axes=0), dict(n_axes=1), dict(inv_freq=float("nan")), dict(inv_freq=float("inf")), dict(axis=2),
                dict(out=FAKE + 16), dict(out=FAKE - 16)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(head_dim=4), dict(head_dim=60), dict(head_dim=264)):
        assert call(**bad) == UNSUPPORTED, bad


def test_rope_plan_refuses(fq):
    for bad in (dict(head_dim=60), dict(head_dim=512), dict(rot_dim=3), dict(rot_dim=256), dict(sections=[63]),
                dict(sections=[70, -6]), dict(sections=[64], axis=[0] * 64), dict(axis=[-1] + [0] * 63),
                dict(inv_freq=[1.0] * 63), dict(inv_freq=[float("nan")] * 64), dict(axis=[300] * 64)):
        with pytest.raises(ValueError):
            fq.Rope.make(**bad)
    r = fq.Rope.make(sections=[16, 24, 24])
    assert r.n_axes == 3 and r.axis[15:17] == (0, 1) and r.inv_freq[0] == 1.0 and r == fq.Rope.make(sections=[16, 24, 24])


def test_a_changed_or_copied_rope_plan_is_its_own(fq):
    r = fq.Rope.make(head_dim=64, sections=[16, 16])
    for c in (copy.deepcopy(r), pickle.loads(pickle.dumps(r))):
        assert c == r and c._ref._obj is not r._ref._obj and list(c._ref._obj.axis) == list(r._ref._obj.axis)
    wide = dataclasses.replace(r, head_dim=128)
    assert (wide._ref._obj.head_dim, wide._ref._obj.rot_dim, r._ref._obj.head_dim) == (128, 64, 64)
    with pytest.raises(ValueError):
        dataclasses.replace(r, head_dim=32)
    with pytest.raises(ValueError):
        dataclasses.replace(r, n_axes=1)


def test_cross_entropy_refuses(fq):
    T, d, V = 5, 64, 100
    nf, nb = fq.linear_cross_entropy_fwd_workspace_size(T, d, V), fq.linear_cross_entropy_bwd_workspace_size(T, d, V)
    assert nf > 0 and nb > 0 and fq.linear_cross_entropy_fwd_workspace_size(T, 60, V) == 0

    def fwd(x=FAKE, W=FAKE, t=FAKE, T=T, d=d, V=V, loss=FAKE, lse=FAKE, ws=FAKE, n=nf):
        return fq.lib.linear_cross_entropy_fwd(x, W, t, T, d, V, -100, loss, lse, ws, n, None)

    def bwd(x=FAKE, W=FAKE, t=FAKE, lse=FAKE, dl=FAKE, T=T, d=d, V=V, dX=FAKE, dW=FAKE, dt=BF16, ws=FAKE, n=nb):
        return fq.lib.linear_cross_entropy_bwd(x, W, t, lse, dl, T, d, V, -100, dX, dW, dt, ws, n, None)
    for bad in (dict(x=None), dict(W=ODD), dict(t=FAKE + 4), dict(T=0), dict(T=(1 << 24) + 1), dict(V=0), dict(V=(1 << 24) + 1),
                dict(d=0), dict(d=60), dict(d=65544), dict(lse=ODD)):
        assert fwd(**bad) == INVALID and bwd(**bad) == INVALID, bad
    assert fwd(loss=None) == INVALID
    assert fwd(T=1 << 24, V=1 << 24) == INVALID and fq.linear_cross_entropy_fwd_workspace_size(1 << 24, 64, 1 << 24) == 0
    for bad in (dict(dl=ODD), dict(dX=ODD), dict(dW=None), dict(dt=2)):
        assert bwd(**bad) == INVALID, bad
    for f, n in ((fwd, nf), (bwd, nb)):
        for bad in (dict(ws=None), dict(ws=FAKE + 16), dict(n=n - 1)):
            assert f(**bad) == WORKSPACE, bad


def test_python_entry_points_refuse_host_tensors(fq):
    x, g, t = torch.zeros(4, 16), torch.ones(16), torch.zeros(4, dtype=torch.int64)
    f = torch.zeros(4)
    for call in (lambda: fq.layernorm_fwd(x, g), lambda: fq.layernorm_bwd(x, x, g, f, f),
                 lambda: fq.rope_fwd(x, t.int(), fq.Rope.make(head_dim=16), 1, 0),
                 lambda: fq.linear_cross_entropy_fwd(x.bfloat16(), x.bfloat16(), t),
                 lambda: fq.linear_cross_entropy_bwd(x.bfloat16(), x.bfloat16(), t, f, f)):
        with pytest.raises(ValueError):
            call()


def test_rope_struct_matches_the_header(fq, tmp_path):
    if not shutil.which("gcc"):
        pytest.skip("gcc not available")
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "fp8q.h"\nint main(void) { printf("%zu %zu %zu\\n", '
                   "sizeof(fp8q_rope), offsetof(fp8q_rope, inv_freq), offsetof(fp8q_rope, axis)); return 0; }\n")
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "layout")], check=True)
    got = subprocess.run([str(tmp_path / "layout")], check=True, capture_output=True, text=True).stdout.split()
    r = fq.FP8QRope
    assert [int(v) for v in got] == [ctypes.sizeof(r), r.inv_freq.offset, r.axis.offset]


def test_rope_frequencies_in_turns(tmp_path):
    """The fixed-point fraction of a turn per position against exact arithmetic: half a unit of 2^-64, and the
    division's and the constant's roundings, below 2^-52 of the turns (the fraction is taken without error)."""
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("g++ not available")
    freqs = [s * f for s in (1.0, -1.0) for f in
             (0.0, 1e-300, 1e-20, 3.1e-19, 4.7e-13, 1e-10, 3.1e-10, 1e-8, 3.1e-7, 1e-4, 0.1, 0.5, 1.0, 3.0, 6.283185307179586,
              6.28318530717958, 7.0, 12345.678, 1e9, 2.0 ** 52 + 0.5)] + [10000.0 ** (-i / 64) for i in range(64)]
    src = tmp_path / "turn.cpp"
    src.write_text('#include "fp8q_turn.h"\n#include <cstdio>\n#include <cstdlib>\nint main(int n, char** v) { for (int i = 1; i < n; ++i) '
                   'std::printf("%llu\\n", (unsigned long long)fp8q::rope_turn(std::strtod(v[i], nullptr))); }\n')
    subprocess.run([cxx, "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover=undefined", "-I",
                    os.path.join(ROOT, "fp8_absmax_reduce_gb300", "csrc"), str(src), "-o", str(tmp_path / "turn")], check=True)
    got = subprocess.run([str(tmp_path / "turn"), *[f.hex() for f in freqs]], check=True, capture_output=True, text=True).stdout.split()
    two_pi = fractions.Fraction("6.28318530717958647692528676655900576839433879875021164194988918461563281257")
    one = fractions.Fraction(2) ** 64
    for f, u in zip(freqs, got):
        turns = fractions.Fraction(f) / two_pi
        off = (int(u) - turns * one) % one
        off = min(off, one - off)
        assert off <= fractions.Fraction(1, 2) + abs(turns) * 2 ** 12, (f, float(off))


@pytest.mark.parametrize("T", [1, 2, 32, 33, 64, 65, 128, 129, 1000, 8192, 131072])
def test_backward_pieces_of_any_vocabulary_fit_their_limit(fq, T):
    """What a larger vocabulary adds to the backward's workspace stops at G's 256 MB (d = 8: the parts of dX, of dW and of the
    logits are at most 32 Tp d, 32 MB and 256 MB), whatever the tokens."""
    size = lambda V: fq.linear_cross_entropy_bwd_workspace_size(T, 8, V)
    rows = 2 * ((T + 31) // 32 * 32) if T <= 64 else T
    other = rows * 8 * (2 + 32 * 4) + T * 16 + (rows + 256) * 8 * 4 * 32 + 4096
    for V in (1 << 20, 3_000_000, 5_000_001, (1 << 24) - 3, 1 << 24):
        assert 0 < size(V) <= (256 << 20) + (256 << 20) + other, V


@pytest.mark.parametrize("d,rows", [(8, 4 * 152), (256, 4 * 152), (264, 152), (512, 152), (1024, 152), (4096, 152), (5120, 152), (8192, 152),
                                    (8200, 152), (16384, 152)])
def test_layernorm_workspace_is_what_the_widths_use(fq, d, rows):
    """Partial rows of dg and db for one block an SM, four where rows are narrow (152 SMs), not for shapes that a width no
    longer takes; fewer tokens need no more rows than tokens."""
    pad = lambda n: (n + 255) // 256 * 256
    assert fq.layernorm_bwd_workspace_size(100000, d) == pad(rows * 2 * d * 4)
    assert fq.layernorm_bwd_workspace_size(5, d) == pad(5 * 2 * d * 4)


def test_head_wait_limit_is_validated(fq):
    T, d, V = 5, 64, 100
    n = max(fq.linear_cross_entropy_fwd_workspace_size(T, d, V), fq.linear_cross_entropy_bwd_workspace_size(T, d, V))

    def call(back, limit=1, x=FAKE, ws=FAKE, n=n):
        return fq.lib.fp8q_selftest_linear_cross_entropy_wait_limit(back, x, FAKE, FAKE, FAKE, T, d, V, -100, FAKE, FAKE, FAKE,
                                                                    FAKE, F32, ws, n, limit, None)
    for back in (0, 1):
        for bad in (dict(limit=10 ** 10 + 1), dict(limit=0), dict(limit=-5), dict(x=ODD)):
            assert call(back, **bad) == INVALID, bad
        assert call(back, ws=None) == WORKSPACE and call(back, n=16) == WORKSPACE
