"""Refusals of the 8-bit key/value cache's entry points, without a GPU: the C entry points return the documented codes before
they touch the device, and the Python entry points raise."""

import ctypes
import os
import shutil
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 6
FAKE, ODD = 1 << 20, (1 << 20) + 2
BF16 = 0


@pytest.fixture(scope="module")
def fq():
    import fp8_absmax_reduce_gb300 as fq
    from fp8_absmax_reduce_gb300 import build as b
    b.build()
    fq.load_library()
    return fq


def cache(fq, **kw):
    f = dict(n_pages=10, page_size=64, n_kv_heads=2, head_dim=128, fmt=0, k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE)
    return fq.FP8QKvCache(**{**f, **kw})


def calls(fq):
    need = fq.lib.attention_cached_workspace_size(cache(fq), 4, 2, 4)

    def append(c, pages=FAKE, n=2, most=3, lens=FAKE, start=None, qkv=FAKE, dt=BF16, T=4, hq=4):
        return fq.lib.kv_cache_append(c, pages, n, most, lens, start, qkv, dt, T, hq, None)

    def read(c, pages=FAKE, n=2, most=3, lens=FAKE, start=None, kv=FAKE, dt=BF16, T=4):
        return fq.lib.kv_cache_read(c, pages, n, most, lens, start, T, kv, dt, None)

    def attend(c, pages=FAKE, n=2, most=3, lens=FAKE, start=None, qkv=FAKE, T=4, hq=4, att=FAKE, lse=FAKE, ws=FAKE, size=need):
        return fq.lib.attention_cached(c, pages, n, most, lens, start, qkv, T, hq, att, lse, ws, size, None)
    return append, read, attend


def test_what_they_share_is_refused(fq):
    for f in calls(fq):
        assert f(None) == INVALID
        for bad in (dict(n_pages=0), dict(n_pages=1 << 31), dict(n_kv_heads=0), dict(n_kv_heads=1025), dict(fmt=2), dict(k=None),
                    dict(k=FAKE + 8), dict(v=None), dict(v=ODD), dict(k_scale=None), dict(v_scale=None)):
            assert f(cache(fq, **bad)) == INVALID, bad
        for bad in (dict(page_size=0), dict(page_size=8), dict(page_size=48), dict(page_size=256), dict(head_dim=32), dict(head_dim=80),
                    dict(head_dim=256), dict(head_dim=0), dict(page_size=-64)):
            assert f(cache(fq, **bad)) == UNSUPPORTED, bad
        for bad in (dict(pages=None), dict(pages=ODD), dict(lens=None), dict(lens=ODD), dict(start=ODD), dict(n=0), dict(n=(1 << 20) + 1),
                    dict(n=3), dict(most=0), dict(most=-1), dict(most=(1 << 30) // 64 + 1), dict(T=0), dict(T=(1 << 28) + 1), dict(T=-4)):
            assert f(cache(fq), **bad) == INVALID, bad


def test_own_arguments_are_refused(fq):
    append, read, attend = calls(fq)
    for bad in (dict(qkv=None), dict(qkv=FAKE + 8), dict(dt=2), dict(hq=-2), dict(hq=3), dict(hq=1026)):
        assert append(cache(fq), **bad) == INVALID, bad
    for bad in (dict(kv=None), dict(kv=ODD), dict(dt=5)):
        assert read(cache(fq), **bad) == INVALID, bad
    for bad in (dict(qkv=None), dict(qkv=ODD), dict(att=None), dict(att=FAKE + 8), dict(lse=None), dict(lse=ODD), dict(hq=0), dict(hq=3),
                dict(hq=1026)):
        assert attend(cache(fq), **bad) == INVALID, bad
    for bad in (dict(ws=None), dict(ws=FAKE + 16), dict(size=0)):
        assert attend(cache(fq), **bad) == WORKSPACE, bad


def test_workspace_sizes(fq):
    size = fq.lib.attention_cached_workspace_size
    assert size(cache(fq), 4, 2, 4) > 0 and size(cache(fq), 4, 2, 4) % 256 == 0
    for args in ((cache(fq, head_dim=80), 4, 2, 4), (cache(fq), 0, 2, 4), (cache(fq), 4, 0, 4), (cache(fq), 4, 2, 3), (None, 4, 2, 4)):
        assert size(*args) == 0
    # tokens of one batch: what it holds does not grow without end
    assert 0 < size(cache(fq), 1 << 28, 1 << 20, 4) <= 1 << 28 and size(cache(fq), 1 << 28, 1 << 20, 8) == 0


def test_python_entry_points_refuse_host_tensors(fq):
    z = torch.zeros(2, 2, 16, 64, dtype=torch.uint8)
    with pytest.raises(ValueError):
        fq.KvCache(z, z, z[:, :, 0, 0].contiguous(), z[:, :, 0, 0].contiguous())
    with pytest.raises(ValueError):
        fq.KvCache(None, z, z, z)


def test_cache_struct_matches_the_header(fq, tmp_path):
    if not shutil.which("gcc"):
        pytest.skip("gcc not available")
    names = [n for n, _ in fq.FP8QKvCache._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "fp8q.h"\nint main(void) {\n  printf("%zu\\n", sizeof(fp8q_kv_cache));\n'
                   + "".join(f'  printf("%zu\\n", offsetof(fp8q_kv_cache, {n}));\n' for n in names) + "  return 0;\n}\n")
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "layout")], check=True)
    got = subprocess.run([str(tmp_path / "layout")], check=True, capture_output=True, text=True).stdout.split()
    assert [int(v) for v in got] == [ctypes.sizeof(fq.FP8QKvCache)] + [getattr(fq.FP8QKvCache, n).offset for n in names]


def test_wait_limit_is_validated(fq):
    need = fq.lib.attention_cached_workspace_size(cache(fq), 4, 2, 4)

    def call(limit, ws=FAKE, **kw):
        return fq.lib.fp8q_selftest_attention_cached_wait_limit(cache(fq, **kw), FAKE, 2, 3, FAKE, None, FAKE, 4, 4, FAKE, FAKE, ws, need, limit, None)
    for limit in (0, -1, 10 ** 10 + 1):
        assert call(limit) == INVALID
    assert call(1, ws=None) == WORKSPACE and call(1, fmt=1) == UNSUPPORTED and call(1, head_dim=64) == UNSUPPORTED
