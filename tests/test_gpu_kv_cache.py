"""The 8-bit key/value cache against its definition in 64 bits: writing, reading back, and attention over it.

Codes, scales and values read back are equal to the definition's.  Attention: an output is off by at most
  2^-8 |att|                                     its rounding to bf16,
  (2^-11 + 2 e + (keys + 16) 2^-22) size         the probabilities as fp16 (half a step, 2^-11 of each); their exponents' errors e;
                                                 fp32 sums over the keys,
with size = sum p |v| / sum p and e = (dh + 16) 2^-23 max sum |q| |k| / sqrt(dh): a score is an fp32 sum of dh products that
the tensor core may cut at 2^-23 of its terms, and its scaling, subtraction and 2^x each add a rounding of the same size.
lse: e + (keys + 16) 2^-22 for the sum's logarithm, and 2^-22 |lse|."""

import copy
import pickle

import numpy as np
import pytest
import torch

import _kv_ref as ref
import fp8_absmax_reduce_gb300 as fq
from _gpu import fp8_table

pytestmark = pytest.mark.gpu

TABLE = [fp8_table(0), fp8_table(1)]


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class World:
    """A cache, sequences in it, and the same in the reference.  Slots that no token was written to hold NaN codes."""

    def __init__(self, fmt=0, dh=128, P=64, hq=4, hkv=2, lens=(1,), rows=1, ragged=None, seed=0, extra=2, behind=0, wide=True):
        self.fmt, self.dh, self.P, self.hq, self.hkv = fmt, dh, P, hq, hkv
        self.rng = np.random.default_rng(seed)
        need = [-(-n // P) for n in lens]
        n_pages = sum(need) + extra
        order = self.rng.permutation(n_pages)
        width = max(1, max(need))
        self.pages = np.full((len(lens), width), -1, np.int64)
        at = 0
        for s, k in enumerate(need):
            self.pages[s, :k] = order[at:at + k]
            at += k
        self.lens = list(lens)
        self.row_start = None
        if ragged is not None:
            self.row_start = [0]
            for r in ragged:
                self.row_start.append(self.row_start[-1] + r)
        self.T = (len(lens) * rows if ragged is None else self.row_start[-1]) + behind
        self.rows = ref.rows_of(len(lens), self.T, self.row_start)
        self.cache = fq.KvCache.allocate(n_pages, hkv, dh, P, fmt)
        self.cache.k.fill_(0x7F)
        self.cache.v.fill_(0xFF)
        self.ref = {n: np.full((n_pages, hkv, P, dh), np.nan) for n in "kv"} | {n: np.full((n_pages, hkv), -127) for n in ("kx", "vx")}
        self.wide = np.where(self.rng.random(dh) < 0.05, 6.0, 1.0) if wide else np.ones(dh)

    def args(self):
        return i32(self.pages), i32(self.lens)

    def start(self):
        return None if self.row_start is None else i32(self.row_start)

    def qkv(self, dtype=torch.bfloat16, std=1.0):
        x = self.rng.standard_normal((self.T, self.hq + 2 * self.hkv, self.dh)) * std * np.exp2(self.rng.integers(-2, 3, (self.T, 1, 1)))
        x[:, self.hq:self.hq + self.hkv] *= self.wide
        t = torch.tensor(x, dtype=torch.float32).to(dtype).cuda()
        return t.reshape(self.T, -1), t.double().cpu().numpy()

    def fill(self):
        """Every sequence's tokens before this call's, written by the framework and by the reference."""
        before = [max(0, n - r) for n, (_, r) in zip(self.lens, self.rows)]
        if not any(before):
            return
        start = np.concatenate([[0], np.cumsum(before)]).tolist()
        rows = ref.rows_of(len(before), start[-1], start)
        x = self.rng.standard_normal((start[-1], 2 * self.hkv, self.dh)) * np.exp2(self.rng.integers(-2, 3, (start[-1], 1, 1)))
        x[:, :self.hkv] *= self.wide
        t = torch.tensor(x, dtype=torch.float32).cuda()
        fq.kv_cache_append(self.cache, t.reshape(start[-1], -1), i32(self.pages), i32(before), 0, row_start=i32(start))
        ref.append(self.ref, self.fmt, self.P, self.pages, before, rows, t.double().cpu().numpy().reshape(-1, 2, self.hkv, self.dh))

    def append(self, dtype=torch.bfloat16, **kw):
        t, x = self.qkv(dtype)
        fq.kv_cache_append(self.cache, t, *self.args(), self.hq, row_start=self.start(), **kw)
        ref.append(self.ref, self.fmt, self.P, self.pages, self.lens, self.rows, x[:, self.hq:].reshape(-1, 2, self.hkv, self.dh))
        return t, x

    def check_cache(self):
        torch.cuda.synchronize()
        for n, c, x in (("k", self.cache.k, self.cache.k_scale), ("v", self.cache.v, self.cache.v_scale)):
            got = TABLE[self.fmt][c.cpu().numpy()]
            assert np.array_equal(np.isnan(got), np.isnan(self.ref[n])), n
            assert np.array_equal(np.nan_to_num(got), np.nan_to_num(self.ref[n])), n
            wrote = ~np.isnan(self.ref[n]).all(axis=(2, 3))
            assert np.array_equal(x.cpu().numpy().astype(int)[wrote] - 127, self.ref[n + "x"][wrote]), n

    def check_attention(self, att, lse, q, below=0.0):
        torch.cuda.synchronize()
        want, size, wlse, mag = ref.attend(self.ref, self.P, self.pages, self.lens, self.rows, q)
        owned = ~np.isnan(wlse[0])
        assert owned.any()
        got, glse = att.double().cpu().numpy().reshape(want.shape), lse.double().cpu().numpy()
        keys = max(1, max(self.lens))
        e = (self.dh + 16) * 2.0 ** -23 * mag.T[:, :, None]
        tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2 * e + (keys + 16) * 2.0 ** -22) * size + below
        worst = np.max((np.abs(got - want) - tol)[owned])
        assert worst <= 0, f"att off by {worst} more than allowed"
        empty = np.isneginf(wlse)
        assert np.array_equal(np.isneginf(glse)[:, owned], empty[:, owned])
        seen = owned[None] & ~empty
        glse, wlse = np.where(seen, glse, 0), np.where(seen, wlse, 0)
        tol = e[:, :, 0].T + (keys + 16) * 2.0 ** -22 + 2.0 ** -22 * np.abs(wlse)
        assert (np.abs(glse - wlse)[seen] <= tol[seen]).all()

    def attend(self, t, x, **kw):
        att, lse = fq.attention_cached(self.cache, t, *self.args(), self.hq, row_start=self.start(), **kw)
        self.check_attention(att, lse, x[:, :self.hq])
        return att, lse


SHAPES = [  # dh, P, hq, hkv
    (128, 64, 4, 2), (128, 128, 7, 1), (64, 16, 3, 3), (96, 32, 10, 2), (128, 16, 16, 1), (64, 128, 40, 2), (96, 64, 1, 1)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("dh,P,hq,hkv", SHAPES)
def test_append_prompts_then_tokens(fmt, dtype, dh, P, hq, hkv):
    """New sequences of one token to several pages, then one more token each, then a few; read back at each step."""
    fq.get_status(clear=True)
    lens = [1, P - 1, P, P + 1, 3 * P + 5]
    w = World(fmt, dh, P, hq, hkv, [n + 8 for n in lens], seed=dh + P + fmt)
    for n_rows, upto in ((lens, lens), ([1] * 5, [n + 1 for n in lens]), ([7, 0, 3, 7, 1], [n + k for n, k in zip(lens, (8, 1, 4, 8, 2))])):
        w.lens, w.row_start = upto, np.concatenate([[0], np.cumsum(n_rows)]).tolist()
        w.T = w.row_start[-1]
        w.rows = ref.rows_of(5, w.T, w.row_start)
        w.append(dtype)
        w.check_cache()
        for out in (torch.float32, torch.bfloat16):
            # every token of every sequence
            full = np.concatenate([[0], np.cumsum(upto)]).tolist()
            got = fq.kv_cache_read(w.cache, *w.args(), full[-1], row_start=i32(full), dtype=out)
            want = ref.read(w.ref, P, w.pages, upto, ref.rows_of(5, full[-1], full), full[-1])
            assert np.array_equal(got.double().cpu().numpy(), want)
    assert fq.get_status() == 0


@pytest.mark.parametrize("n,rows", [(1, 1), (3, 2), (70, 1), (2, 130), (5, 33)])
def test_append_of_equal_rows(n, rows):
    w = World(0, 64, 32, 2, 2, [rows + (37 * s) % 101 for s in range(n)], rows=rows, seed=n)
    w.fill()
    w.append()
    w.check_cache()
    got = fq.kv_cache_read(w.cache, *w.args(), w.T, dtype=torch.float32)
    assert np.array_equal(got.double().cpu().numpy(), ref.read(w.ref, w.P, w.pages, w.lens, w.rows, w.T))


def test_append_of_many_ragged_sequences():
    """Sequences with no rows between others, in blocks of rows that begin inside pages; a batch longer than a search of one step."""
    rng = np.random.default_rng(4)
    ragged = rng.integers(0, 6, 1100).tolist()
    ragged[500] = 200
    lens = [r + int(rng.integers(0, 40)) for r in ragged]
    w = World(0, 64, 16, 1, 1, lens, ragged=ragged, seed=5, behind=9)
    w.fill()
    w.append()
    w.check_cache()
    kv = torch.full((w.T, 2 * 64), 7.0, device="cuda")
    fq.kv_cache_read(w.cache, *w.args(), w.T, row_start=w.start(), kv=kv)
    want = ref.read(w.ref, w.P, w.pages, w.lens, w.rows, w.T)
    assert np.array_equal(kv.double().cpu().numpy(), np.where(np.isnan(want), 7.0, want))


def test_scales_grow_and_small_values_follow():
    """A page whose later tokens are larger by powers of two from 1 to 2^40, then by none."""
    for fmt in (0, 1):
        w = World(fmt, 64, 16, 0, 1, [16], seed=9)
        for t, grow in enumerate([0, 1, 1, 3, 8, 8, 9, 17, 40, 40, 0, 2]):
            w.lens = [t + 1]
            x = w.rng.standard_normal((1, 2, 64)) * 2.0 ** grow
            d = torch.tensor(x, dtype=torch.float32).cuda()
            fq.kv_cache_append(w.cache, d.reshape(1, -1), i32(w.pages), i32(w.lens), 0)
            ref.append(w.ref, fmt, 16, w.pages, w.lens, [(0, 1)], d.double().cpu().numpy().reshape(1, 2, 1, 64))
            w.check_cache()


@pytest.mark.parametrize("fmt", [0, 1])
def test_scale_rule_at_its_borders(fmt):
    """amax on, just above and just below fmax 2^X, the largest and smallest fp32 values, zero."""
    f = np.float32(ref.FMAX[fmt])
    vals = [f, np.nextafter(f, np.float32(np.inf)), np.nextafter(f, np.float32(0)), f / 2, np.float32(1.75), np.float32(0),
            np.finfo(np.float32).max, np.float32(2.0 ** -149), np.float32(2.0 ** -126), np.float32(3e-39), np.float32(1e-30)]
    n = len(vals)
    w = World(fmt, 64, 16, 0, 1, [1] * n, seed=1)
    x = np.zeros((n, 2, 1, 64), np.float32)
    x[:, 0, 0, 3], x[:, 1, 0, 60] = vals, [-v for v in vals]
    fq.kv_cache_append(w.cache, torch.tensor(x).cuda().reshape(n, -1), i32(w.pages), i32(w.lens), 0)
    ref.append(w.ref, fmt, 16, w.pages, w.lens, w.rows, x.astype(float))
    w.check_cache()


def test_values_that_are_not_finite_are_marked_and_spoil_no_other():
    fq.get_status(clear=True)
    w = World(0, 64, 16, 2, 2, [20, 5], rows=4, seed=3)
    w.fill()
    t, x = w.qkv()
    t[1, 2 * 64 + 5] = float("inf")     # first K head, second row
    t[2, 5 * 64 + 1] = float("nan")     # second V head, third row
    t[5, 3 * 64:4 * 64] = float("nan")  # a whole K head of a row
    fq.kv_cache_append(w.cache, t, *w.args(), 2)
    x = t.double().cpu().numpy().reshape(8, 6, 64)
    ref.append(w.ref, 0, 16, w.pages, w.lens, w.rows, x[:, 2:].reshape(-1, 2, 2, 64))
    w.check_cache()
    assert fq.get_status(clear=True) == fq.STATUS_NONFINITE
    # rows before the NaN tokens, and heads without one, are what they were
    att, lse = fq.attention_cached(w.cache, t, *w.args(), 2)
    torch.cuda.synchronize()
    a = att.float().view(8, 2, 64)
    assert torch.isfinite(a[0]).all() and torch.isfinite(a[4]).all()
    assert torch.isnan(a[1:4, 0]).all() and torch.isfinite(a[1, 1]).all()  # K head 0 holds a NaN in token 17
    assert torch.isnan(a[2:4, 1, 1]).all() and torch.isfinite(a[2:4, 1, 2:]).all()  # V head 1: one column
    assert torch.isnan(a[5:, 1]).all() and torch.isfinite(a[5:, 0]).all()


ATTEND = [  # dh, P, hq, hkv, lens, rows, ragged
    (128, 64, 4, 2, [1], 1, None),
    (128, 64, 40, 8, [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 500], 1, None),
    (128, 128, 28, 4, [1000, 1, 0, 257, 0], 1, None),
    (64, 16, 12, 12, [5, 100, 17, 333], None, [3, 0, 1, 6]),
    (96, 32, 10, 2, [40, 7, 200], 7, None),
    (128, 16, 16, 1, [300, 3, 4], 4, None),          # 64 rows of a head; a sequence shorter than its rows
    (64, 128, 40, 2, [70, 130], 3, None),            # 60 rows of a head
    (128, 64, 5, 1, [260, 90], None, [150, 90]),     # a piece of a prompt, a whole prompt
    (96, 64, 1, 1, [1030], 1, None),
    (64, 32, 6, 6, [2100, 1, 900], None, [1, 1, 130]),
    (128, 32, 33, 1, [129, 64], 2, None),
]


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("case", range(len(ATTEND)))
def test_attention_matches_its_definition(case, fmt):
    dh, P, hq, hkv, lens, rows, ragged = ATTEND[case]
    fq.get_status(clear=True)
    w = World(fmt, dh, P, hq, hkv, lens, rows=rows, ragged=ragged, seed=case, behind=0 if ragged is None else 3)
    w.fill()
    t, x = w.append()
    w.check_cache()
    w.attend(t, x)
    assert fq.get_status() == 0


MANY = [  # more than 64 (token, query head) pairs of a K/V head: the kernel on tensor memory
    (128, 64, 5, 1, [700, 512, 130], 130, None),
    (96, 16, 10, 2, [300, 0, 45], 40, None),
    (64, 128, 6, 6, [1000, 90], None, [90, 90]),
    (128, 16, 8, 1, [257, 1024, 33], None, [257, 64, 1]),
    (96, 128, 3, 1, [2000], None, [100]),
    (128, 32, 70, 1, [5, 300], 1, None),             # 70 heads of one token
    (64, 64, 2, 2, [400] * 5, None, [399, 1, 0, 257, 128]),
    (128, 128, 4, 4, [129] * 40, 128, None),         # more units than SMs
    (128, 64, 1, 1, [9000], 300, None),              # a unit cut over many CTAs
]


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("case", range(len(MANY)))
def test_attention_of_many_rows_matches_its_definition(case, fmt):
    dh, P, hq, hkv, lens, rows, ragged = MANY[case]
    fq.get_status(clear=True)
    w = World(fmt, dh, P, hq, hkv, lens, rows=rows, ragged=ragged, seed=100 + case, behind=0 if ragged is None else 2)
    w.fill()
    t, x = w.append()
    first = w.attend(t, x)
    again = fq.attention_cached(w.cache, t, *w.args(), hq, row_start=w.start())
    torch.cuda.synchronize()
    n = w.T if w.row_start is None else w.row_start[-1]
    assert torch.equal(first[0][:n], again[0][:n]) and torch.equal(first[1][:, :n], again[1][:, :n])
    assert fq.get_status() == 0


@pytest.mark.parametrize("idle", [1, 2, 3, 7])
def test_many_rows_with_idle_slots_between_sequences_of_different_sizes(idle):
    """Sequences of one or two blocks, V 2^20 apart, with empty slots between them: a CTA has many of both."""
    n = 1500
    lens = [(200 if s % 8 else 120) if s % (idle + 1) == 0 else 0 for s in range(n)]
    w = World(0, 64, 64, 9, 1, lens, rows=8, seed=40 + idle, wide=False)
    before = [max(0, k - 8) for k in lens]
    start = np.concatenate([[0], np.cumsum(before)]).tolist()
    x = w.rng.standard_normal((start[-1], 2, 1, 64))
    x[:, 1] *= np.repeat(np.exp2(w.rng.integers(-10, 11, n)), before)[:, None, None]
    d = torch.tensor(x, dtype=torch.float32).cuda()
    fq.kv_cache_append(w.cache, d.reshape(start[-1], -1), i32(w.pages), i32(before), 0, row_start=i32(start))
    ref.append(w.ref, 0, 64, w.pages, before, ref.rows_of(n, start[-1], start), d.double().cpu().numpy())
    t, x = w.append()
    # A weight in a small page is p 2^dx 2^11 in fp16, dx the page's exponent below the sequence's largest page: where that is subnormal
    # it is off by up to 2^-25, which multiplies a code of up to 448 in units of the largest page's 2^X <= 2 max |v| / 448.  A sum of
    # weights is 1 at least, so an output is off by keys 2^-25 2^-11 2 max |v| besides.
    below = np.zeros((w.T, 1, 1))
    for s, (first, m) in enumerate(w.rows):
        v, _ = ref.held(w.ref, 64, w.pages, s, lens[s], "v")
        below[first:first + m] = lens[s] * 2.0 ** -35 * np.abs(v).max(initial=0.0)
    att, lse = fq.attention_cached(w.cache, t, *w.args(), 9)
    w.check_attention(att, lse, x[:, :9], below)


def test_many_rows_see_values_that_are_not_finite_only_behind_them():
    w = World(0, 64, 32, 2, 2, [300, 300], rows=200, seed=30)
    w.fill()
    t, _ = w.qkv()
    t[120, 2 * 64 + 5] = float("inf")   # K head 0 of the first sequence's token 220
    t[150, 5 * 64 + 7] = float("nan")   # V head 1, column 7, of its token 250
    fq.kv_cache_append(w.cache, t, *w.args(), 2)
    x = t.double().cpu().numpy().reshape(400, 6, 64)
    ref.append(w.ref, 0, 32, w.pages, w.lens, w.rows, x[:, 2:].reshape(-1, 2, 2, 64))
    w.check_cache()
    att, lse = fq.attention_cached(w.cache, t, *w.args(), 2)
    torch.cuda.synchronize()
    a = att.float().view(400, 2, 64)
    assert torch.isnan(a[120:200, 0]).all() and torch.isfinite(a[:120, 0]).all() and torch.isfinite(a[200:]).all()
    assert torch.isnan(a[150:200, 1, 7]).all()
    a[150:200, 1, 7] = 0
    assert torch.isfinite(a[:, 1]).all()
    # what is finite is what it was: rows before, and the other columns
    fine = {k: np.nan_to_num(v) if k in "kv" else v for k, v in w.ref.items()}
    want, size, _, _ = ref.attend(fine, 32, w.pages, w.lens, w.rows, x[:, :2])
    got = att.double().cpu().numpy().reshape(400, 2, 64)
    rows = [r for r in range(400) if not 120 <= r < 200]
    assert np.abs(got[rows, 0] - want[rows, 0]).max() < 0.02 * size.max()
    others = [c for c in range(64) if c != 7]
    assert np.abs(got[:, 1][:, others] - want[:, 1][:, others]).max() < 0.02 * size.max()


def test_rows_behind_the_last_sequence_are_left_as_they_were():
    w = World(0, 128, 32, 6, 2, [50, 9], ragged=[3, 2], behind=4, seed=2)
    w.fill()
    t, x = w.append()
    att = torch.full((w.T, 6 * 128), 3.0, device="cuda").bfloat16()
    lse = torch.full((6, w.T), 5.0, device="cuda")
    w.attend(t, x, att=att, lse=lse)
    assert (att[5:] == 3).all() and (lse[:, 5:] == 5).all()


def test_pages_of_very_different_sizes():
    """V pages 2^20 apart, and K so that the probable keys are those of the small pages: each keeps its own precision."""
    w = World(0, 64, 16, 2, 1, [200], rows=1, seed=11, wide=False)
    before = 199
    x = w.rng.standard_normal((before, 2, 1, 64))
    size = np.exp2(np.repeat(w.rng.integers(-10, 11, 13), 16)[:before])
    x[:, 1] *= size[:, None, None]
    d = torch.tensor(x, dtype=torch.float32).cuda()
    fq.kv_cache_append(w.cache, d.reshape(before, -1), i32(w.pages), i32([before]), 0)
    ref.append(w.ref, 0, 16, w.pages, [before], [(0, before)], d.double().cpu().numpy())
    t, q = w.append()
    w.attend(t, q)


def test_sharp_and_flat_probabilities():
    """Scores of +-60 (one key takes all), and of zero (every key alike); many keys far below the largest."""
    for std in (8.0, 0.0):
        w = World(0, 128, 64, 4, 2, [700, 65], rows=1, seed=12)
        w.fill()
        w.append()
        t, x = w.qkv(std=std)
        w.attend(t, x)
    # a first key 20 above 5000 equal ones
    w = World(0, 64, 64, 1, 1, [5000], rows=1, seed=13)
    k = np.zeros((5000, 2, 1, 64))
    k[0, 0, 0, 0] = 20.0
    k[:, 1] = w.rng.standard_normal((5000, 1, 64))
    d = torch.tensor(k, dtype=torch.float32).cuda()
    fq.kv_cache_append(w.cache, d.reshape(5000, -1), i32(w.pages), i32([5000]), 0)
    ref.append(w.ref, 0, 64, w.pages, [5000], [(0, 5000)], d.double().cpu().numpy())
    q = torch.zeros((1, 3 * 64), device="cuda").bfloat16()
    for big in (8.0, 4.0):
        q[0, 0] = big
        w.attend(q, q.double().cpu().numpy().reshape(1, 3, 64))


def test_q_of_any_size():
    """q from the smallest to the largest magnitudes of bf16, with small elements beside large ones; K so that scores stay finite."""
    for std in (2.0 ** -120, 2.0 ** -30, 2.0 ** 20, 2.0 ** 100):
        w = World(0, 64, 16, 2, 1, [40], rows=1, seed=14, wide=False)
        k = w.rng.standard_normal((40, 2, 1, 64))
        k[:, 0] /= std
        d = torch.tensor(k, dtype=torch.float32).cuda()
        fq.kv_cache_append(w.cache, d.reshape(40, -1), i32(w.pages), i32([40]), 0)
        ref.append(w.ref, 0, 16, w.pages, [40], [(0, 40)], d.double().cpu().numpy())
        x = w.rng.standard_normal((1, 4, 64)) * np.exp2(w.rng.integers(-12, 1, (1, 4, 64)).astype(float)) * std
        q = torch.tensor(x, dtype=torch.float64).to(torch.bfloat16).cuda()
        w.attend(q.reshape(1, -1), q.double().cpu().numpy())


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("dh,hq,rows", [(64, 8, 1), (128, 7, 1), (96, 12, 1), (128, 5, 6), (64, 4, 130), (128, 3, 140)])
def test_scores_of_any_size(dh, hq, rows, fmt):
    """Scores from 2^7 to 2^117, either sign, of which one is largest or many are alike, to the last bit; the others are further below than any
    weight reaches.  Then only the weights' rounding, the sums' and the output's are left: a score's own error is the same for all that count, but
    for the window's offset, which may go into a reference below 2^10, rounded to half a unit of 2^-14 there.
    lse: five roundings of the score (scale, product, sum, ln 2 and its product)."""
    n = 300
    for a in (10, 18, 22, 24, 25, 27, 31, 40, 90, 120):
        w = World(fmt, dh, 32, hq, 1, [n, n - 111], rows=rows, seed=a, wide=False)
        start = np.concatenate([[0], np.cumsum(w.lens)]).tolist()
        kv = w.rng.standard_normal((start[-1], 2, 1, dh))
        kv[:, 0] = 0
        kv[:, 0, 0, 3] = 0.5
        for s in range(2):
            kv[start[s] + 101, 0, 0, 3] = 1.0
        d = torch.tensor(kv, dtype=torch.float32).cuda()
        fq.kv_cache_append(w.cache, d.reshape(start[-1], -1), i32(w.pages), i32(w.lens), 0, row_start=i32(start))
        ref.append(w.ref, fmt, 32, w.pages, w.lens, ref.rows_of(2, start[-1], start), d.double().cpu().numpy())
        x = np.zeros((w.T, hq + 2, dh))
        x[:, :hq, 3] = w.rng.choice([-1, 1], (w.T, hq)) * w.rng.integers(128, 256, (w.T, hq)) * 2.0 ** (a - 7)
        q = torch.tensor(x).to(torch.bfloat16).cuda()
        att, lse = fq.attention_cached(w.cache, q.reshape(w.T, -1), *w.args(), hq)
        torch.cuda.synchronize()
        want, size, wlse, _ = ref.attend(w.ref, 32, w.pages, w.lens, w.rows, x[:, :hq])
        got, glse = att.double().cpu().numpy().reshape(want.shape), lse.double().cpu().numpy()
        assert np.isfinite(got).all() and np.isfinite(glse).all(), a
        off = np.abs(got - want) - (2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -15 + (n + 16) * 2.0 ** -22) * size)
        assert off.max() <= 0, (a, off.max())
        assert (np.abs(glse - wlse) <= 5 * 2.0 ** -24 * (1 + 2.0 ** -10) * np.abs(wlse) + (n + 16) * 2.0 ** -22).all(), a


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("dh,hq,rows,before", [(128, 2, 4, 45), (64, 4, 8, 60), (96, 8, 8, 1004), (128, 4, 30, 20), (64, 4, 130, 30), (96, 2, 200, 700),
                                               (128, 6, 150, 0), (128, 4, 300, 5000)])
def test_rows_do_not_depend_on_values_that_they_do_not_see(dh, hq, rows, before, fmt):
    """V of the pages of the call's later tokens from unit size to 2^100 of it: rows before those pages keep their bits, and are right; rows
    that see them lose at most what vanishes beside them, keys 2^-36 of the largest scale, which is at most twice max |v| over fmax, times fmax."""
    n, P = before + rows, 16
    border = -(-(before + rows // 2) // P) * P  # a page's first token, inside the call's
    outs = []
    for up in (0, 30, 40, 100):
        w = World(fmt, dh, P, hq, 2, [n], rows=rows, seed=60 + dh, wide=False)
        w.fill()
        q, x = w.qkv()
        v = q.view(rows, hq + 4, dh)[:, hq + 2:]
        v[max(0, border - before):] *= 2.0 ** up
        x = q.double().cpu().numpy().reshape(rows, hq + 4, dh)
        fq.kv_cache_append(w.cache, q, *w.args(), hq)
        ref.append(w.ref, fmt, P, w.pages, w.lens, w.rows, x[:, hq:].reshape(-1, 2, 2, dh))
        w.check_cache()
        att, lse = fq.attention_cached(w.cache, q, *w.args(), hq)
        seen = before + np.arange(rows) >= border
        big, _ = ref.held(w.ref, P, w.pages, 0, n, "v")
        w.check_attention(att, lse, x[:, :hq], below=(seen * n * 2.0 ** -35 * np.abs(big).max())[:, None, None])
        outs.append((att[:border - before], lse[:, :border - before]))
    assert 0 < border - before < rows
    for att, lse in outs[1:]:
        assert torch.equal(att, outs[0][0]) and torch.equal(lse, outs[0][1])


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("dh,hq,rows,before", [(128, 2, 4, 45), (64, 4, 8, 60), (96, 8, 8, 1004), (128, 4, 30, 20), (64, 4, 130, 30), (96, 2, 200, 700),
                                               (128, 6, 150, 0)])
def test_rows_keep_their_bits_whatever_keys_they_do_not_see(dh, hq, rows, before, fmt):
    """K of the pages of the call's later tokens of unit size, 2^20 and 2^60 of it (scores that are taken another way), and not finite, V too."""
    n, P = before + rows, 16
    border = -(-(before + rows // 2) // P) * P
    outs = []
    for up in (1.0, 2.0 ** 20, 2.0 ** 60, float("nan")):
        w = World(fmt, dh, P, hq, 2, [n], rows=rows, seed=70 + dh, wide=False)
        w.fill()
        q, _ = w.qkv()
        kv = q.view(rows, hq + 4, dh)[:, hq:]
        kv[border - before:, :2] *= up
        if up != up:
            kv[border - before:] = up
        fq.kv_cache_append(w.cache, q, *w.args(), hq)
        att, lse = fq.attention_cached(w.cache, q, *w.args(), hq)
        outs.append((att[:border - before], lse[:, :border - before]))
    torch.cuda.synchronize()
    fq.get_status(clear=True)
    assert 0 < border - before < rows and torch.isfinite(outs[0][0]).all() and torch.isfinite(outs[0][1]).all()
    for att, lse in outs[1:]:
        assert torch.equal(att, outs[0][0]) and torch.equal(lse, outs[0][1])


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("dh,rows", [(64, 1), (128, 1), (96, 9), (64, 130), (128, 130)])
def test_pages_of_the_smallest_scale(dh, rows, fmt):
    """K and V below fmax 2^-127, so that their scale has code 0, and q so that scores are of unit size; every kernel, units cut and whole.
    Outputs are near bf16's subnormal numbers, half a step of which (2^-134) is allowed besides, and as much for fp32's."""
    w = World(fmt, dh, 32, 4, 2, [1000, 150, 130], rows=rows, seed=50 + dh)
    start = np.concatenate([[0], np.cumsum(w.lens)]).tolist()
    x = w.rng.uniform(-1, 1, (start[-1], 4, dh)) * 2.0 ** -119
    d = torch.tensor(x, dtype=torch.float32).cuda()
    fq.kv_cache_append(w.cache, d.reshape(start[-1], -1), i32(w.pages), i32(w.lens), 0, row_start=i32(start))
    ref.append(w.ref, fmt, 32, w.pages, w.lens, ref.rows_of(3, start[-1], start), d.double().cpu().numpy().reshape(-1, 2, 2, dh))
    w.check_cache()
    assert (w.ref["kx"][w.pages[0]] == -127).all() and (w.ref["vx"][w.pages[0]] == -127).all()
    q, x = w.qkv(std=2.0 ** 117)
    att, lse = fq.attention_cached(w.cache, q, *w.args(), 4)
    w.check_attention(att, lse, x[:, :4], below=2.0 ** -133)


@pytest.mark.parametrize("n,length,hkv,hq", [(1, 20000, 1, 5), (1, 4000, 8, 8), (40, 700, 2, 2), (300, 40, 1, 1)])
def test_work_split_over_the_keys(n, length, hkv, hq):
    """Long sequences cut over many blocks, and more sequences than blocks."""
    w = World(0, 128, 64, hq, hkv, [max(1, length - 13 * s) for s in range(n)], rows=1, seed=n)
    w.fill()
    t, x = w.append()
    a1 = w.attend(t, x)
    a2 = fq.attention_cached(w.cache, t, *w.args(), hq)
    assert all(torch.equal(a, b) for a, b in zip(a1, a2))


def test_bad_pages_lengths_and_rows_are_reported_and_touch_nothing_else():
    """Invalid tables are turned into the status bit by the kernels' own checks."""
    w = World(0, 128, 32, 4, 2, [100, 70, 33], ragged=[2, 3, 1], seed=6)
    w.fill()
    t, x = w.append()
    good = fq.attention_cached(w.cache, t, *w.args(), 4, row_start=w.start())
    kv_good = fq.kv_cache_read(w.cache, *w.args(), w.T, row_start=w.start())
    torch.cuda.synchronize()
    keep = [c.clone() for c in (w.cache.k, w.cache.v, w.cache.k_scale, w.cache.v_scale)]
    fq.get_status(clear=True)
    for bad_page in (-5, w.cache.n_pages, 2 ** 31 - 1, -2 ** 31):
        p = w.pages.copy()
        p[0, 1] = bad_page                     # a page in the middle: its tokens are not seen
        p[1, 2] = bad_page                     # the page of the second sequence's rows (tokens 67 .. 69)
        fq.kv_cache_append(w.cache, t, i32(p), i32(w.lens), 4, row_start=w.start())
        att, lse = fq.attention_cached(w.cache, t, i32(p), i32(w.lens), 4, row_start=w.start())
        kv = fq.kv_cache_read(w.cache, i32(p), i32(w.lens), w.T, row_start=w.start())
        torch.cuda.synchronize()
        assert fq.get_status(clear=True) == fq.STATUS_BAD_CACHE
        assert all(torch.equal(a, b) for a, b in zip(keep, (w.cache.k, w.cache.v, w.cache.k_scale, w.cache.v_scale)))
        assert (kv[2:5] == 0).all() and torch.equal(kv[:2], kv_good[:2]) and torch.equal(kv[5:], kv_good[5:])
        assert torch.equal(att[5:], good[0][5:])
        saved, w.pages = w.pages, p
        w.check_attention(att, lse, x[:, :4])
        w.pages = saved
    for lens in ([100, -1, 33], [100, 32 * w.pages.shape[1] + 1, 33], [100, 2 ** 31 - 1, 33], [100, -2 ** 31, 33]):
        fq.kv_cache_append(w.cache, t, i32(w.pages), i32(lens), 4, row_start=w.start())
        att, lse = fq.attention_cached(w.cache, t, i32(w.pages), i32(lens), 4, row_start=w.start())
        kv = fq.kv_cache_read(w.cache, i32(w.pages), i32(lens), w.T, row_start=w.start())
        torch.cuda.synchronize()
        assert fq.get_status(clear=True) == fq.STATUS_BAD_CACHE
        assert (att[2:5] == 0).all() and torch.isneginf(lse[:, 2:5]).all() and (kv[2:5] == 0).all()
        assert torch.equal(att[:2], good[0][:2]) and torch.equal(att[5:], good[0][5:])
        assert all(torch.equal(a, b) for a, b in zip(keep, (w.cache.k, w.cache.v, w.cache.k_scale, w.cache.v_scale)))
    for start in ([0, 2, 9, 9], [-3, 2, 5, 6], [0, 2, 1, 6], [0, 2, 2 ** 31 - 1, -2 ** 31], [2 ** 31 - 1] * 4):
        fq.attention_cached(w.cache, t, i32(w.pages), i32(w.lens), 4, row_start=i32(start))
        fq.kv_cache_read(w.cache, i32(w.pages), i32(w.lens), w.T, row_start=i32(start))
        scratch = fq.KvCache(w.cache.k.clone(), w.cache.v.clone(), w.cache.k_scale.clone(), w.cache.v_scale.clone())
        fq.kv_cache_append(scratch, t, i32(w.pages), i32(w.lens), 4, row_start=i32(start))
        torch.cuda.synchronize()
        status = fq.get_status(clear=True)
        if start == [0, 2, 1, 6] or start[0] == 2 ** 31 - 1:  # decreasing rows may go unreported; no row of the call is anyone's
            assert status in (0, fq.STATUS_BAD_CACHE)
        else:
            assert status == fq.STATUS_BAD_CACHE


def test_pages_past_32_bits():
    """A cache of over 4 GB for K: the last pages are written, read and attended to."""
    n_pages = (1 << 32) // (64 * 128 * 4) + 5
    cache = fq.KvCache.allocate(n_pages, 4, 128, 64)
    pages = i32([[n_pages - 1, 3, n_pages - 2]])
    g = torch.Generator(device="cuda").manual_seed(1)
    qkv = torch.randn((150, 12 * 128), generator=g, device="cuda").bfloat16()
    fq.kv_cache_append(cache, qkv, pages, i32([150]), 4)
    small = fq.KvCache.allocate(3, 4, 128, 64)
    fq.kv_cache_append(small, qkv, i32([[0, 1, 2]]), i32([150]), 4)
    for a, b in ((cache.k, small.k), (cache.v, small.v), (cache.k_scale, small.k_scale), (cache.v_scale, small.v_scale)):
        assert torch.equal(a[pages[0].long()], b) and int(a[:3].count_nonzero()) == 0
    a1, a2 = (fq.attention_cached(c, qkv, p, i32([150]), 4) for c, p in ((cache, pages), (small, i32([[0, 1, 2]]))))
    assert torch.equal(a1[0], a2[0]) and torch.equal(a1[1], a2[1])
    assert torch.equal(fq.kv_cache_read(cache, pages, i32([150]), 150), fq.kv_cache_read(small, i32([[0, 1, 2]]), i32([150]), 150))


def test_sequences_may_share_pages_that_they_read():
    w = World(0, 64, 16, 2, 1, [40], rows=1, seed=8)
    w.fill()
    t, x = w.append()
    one = fq.attention_cached(w.cache, t, *w.args(), 2)
    two = fq.attention_cached(w.cache, t.repeat(3, 1), i32(np.repeat(w.pages, 3, 0)), i32([40] * 3), 2)
    assert all(torch.equal(two[0][i], one[0][0]) and torch.equal(two[1][:, i], one[1][:, 0]) for i in range(3))
    back = fq.kv_cache_read(w.cache, i32(np.repeat(w.pages, 3, 0)), i32([40] * 3), 60)
    assert torch.equal(back[:20], back[20:40]) and torch.equal(back[:20], back[40:])


def test_a_step_taken_back_is_overwritten():
    """Drafted tokens that were not accepted: the length goes back, the next tokens take their slots."""
    w = World(0, 64, 16, 2, 1, [30], rows=6, seed=21)
    w.fill()
    w.append()
    w.lens, w.T = [27], 2
    w.rows = ref.rows_of(1, 2, None)
    t, x = w.append()
    w.check_cache()
    w.attend(t, x)


def test_entry_points_refuse():
    c = fq.KvCache.allocate(4, 2, 64, 16)
    q = torch.zeros((2, 8 * 64), device="cuda").bfloat16()
    p, n = i32([[0, 1], [2, 3]]), i32([3, 4])
    for call in (lambda **k: fq.kv_cache_append(**{**dict(cache=c, qkv=q, pages=p, lens=n, n_heads=4), **k}),
                 lambda **k: fq.attention_cached(**{**dict(cache=c, qkv=q, pages=p, lens=n, n_heads=4), **k})):
        call()
        for bad in (dict(qkv=q[:, :64].contiguous()), dict(qkv=q.cpu()), dict(qkv=q[0]), dict(qkv=q.t()), dict(pages=p.long()),
                    dict(pages=p[0]), dict(pages=p.t()), dict(lens=n.long()), dict(lens=n[:1]), dict(lens=[3, 4]),
                    dict(row_start=n), dict(row_start=i32([0, 1, 2]).long()), dict(n_heads=3), dict(qkv=q.half()), dict(pages=None)):
            with pytest.raises((ValueError, TypeError)):
                call(**bad)
        with pytest.raises(fq.Fp8qError):
            call(qkv=torch.zeros((3, 8 * 64), device="cuda").bfloat16())  # 3 rows of 2 sequences
    with pytest.raises(TypeError):
        fq.attention_cached(c, q.float(), p, n, 4)
    with pytest.raises(TypeError):
        fq.kv_cache_read(c, p, n, 2, dtype=torch.float16)
    with pytest.raises(ValueError):
        fq.kv_cache_read(c, p, n, 2, kv=torch.empty((2, 64), device="cuda"))
    with pytest.raises(ValueError):
        fq.attention_cached(c, q, p, n, 4, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        fq.attention_cached(c, q, p, n, 4, att=torch.empty((2, 64), device="cuda").bfloat16())
    with pytest.raises(fq.Fp8qError):
        fq.kv_cache_read(c, p, n, 0)
    for bad in (dict(k=c.k[:, :, :8]), dict(k_scale=c.k_scale.int()), dict(v=c.v[:2]), dict(v=c.v.cpu()), dict(fmt=3)):
        with pytest.raises((ValueError, TypeError)):
            fq.KvCache(**{**dict(k=c.k, v=c.v, k_scale=c.k_scale, v_scale=c.v_scale), **bad})


def test_copies_of_a_cache_are_their_own():
    w = World(0, 64, 16, 2, 1, [20], rows=1, seed=15)
    w.fill()
    t, x = w.append()
    want = fq.attention_cached(w.cache, t, *w.args(), 2)
    other = copy.deepcopy(w.cache)
    w.cache.k.zero_()
    for c in (other, pickle.loads(pickle.dumps(other))):
        got = fq.attention_cached(c, t, *w.args(), 2)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_calls_on_another_stream_and_in_graphs():
    """stream=; a captured step replayed with new lengths; two graphs with workspaces of their own at once."""
    w = World(0, 128, 64, 8, 2, [130, 64, 1], rows=1, seed=16, extra=4)
    w.fill()
    t, x = w.append()
    args = w.args()
    want = w.attend(t, x)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = fq.attention_cached(w.cache, t, *args, 8, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graphs, outs = [], []
    with torch.cuda.stream(side):
        fq.kv_cache_append(w.cache, t, *args, 8)
    side.synchronize()
    for _ in range(2):
        ws = torch.empty(fq.attention_cached_workspace_size(w.cache, 3, 3, 8), dtype=torch.uint8, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(fq.attention_cached(w.cache, t, *args, 8, ws=ws) + (fq.kv_cache_read(w.cache, *args, 3), ws))
        graphs.append(g)
    for lens in ([130, 64, 1], [100, 3, 0]):
        args[1].copy_(i32(lens))
        torch.cuda.synchronize()
        for g in graphs:
            with torch.cuda.stream(torch.cuda.Stream()):
                g.replay()
        torch.cuda.synchronize()
        eager = fq.attention_cached(w.cache, t, *args, 8) + (fq.kv_cache_read(w.cache, *args, 3),)
        for o in outs:
            assert all(torch.equal(a, b) for a, b in zip(o, eager))


def test_a_sequence_run_token_by_token():
    """rope, append and attention as a program uses them: a prompt through attention_fwd and into the cache, then tokens one
    at a time; each against attention over the values that the cache holds.  The prompt's last token is also attended to over the cache: it
    differs from attention_fwd's by the codes' rounding.  V's is at most 2^-4 of each value, and as independent from value to value as
    they are, so it moves the sum by at most 2^-4 of itself; K's moves a score by at most 2^-4 of its own spread (about 0.7^2), and the sum
    by that much: together below 2 2^-4."""
    S, hq, hkv, steps = 256, 8, 2, 20
    g = torch.Generator(device="cuda").manual_seed(3)
    rope = fq.Rope.make()
    w = World(0, 128, 64, hq, hkv, [S + steps] * 2, rows=1, seed=17)
    qkv = (0.7 * torch.randn((2 * S, (hq + 2 * hkv) * 128), generator=g, device="cuda")).bfloat16()
    pos = torch.arange(S, device="cuda").repeat(2).int()
    qkv = fq.rope_fwd(qkv, pos, rope, hq, hkv, out=qkv)
    att, _ = fq.attention_fwd(qkv, S, hq, hkv)
    w.lens, w.T = [S, S], 2 * S
    w.rows = ref.rows_of(2, 2 * S, None)
    fq.kv_cache_append(w.cache, qkv, *w.args(), hq)
    host = qkv.double().cpu().numpy().reshape(2 * S, -1, 128)
    ref.append(w.ref, 0, 64, w.pages, w.lens, w.rows, host[:, hq:].reshape(-1, 2, hkv, 128))
    w.check_cache()
    last = qkv[[S - 1, 2 * S - 1]].contiguous()
    cached, _ = fq.attention_cached(w.cache, last, *w.args(), hq)
    off = (cached.float() - att[[S - 1, 2 * S - 1]].float()).norm() / att[[S - 1, 2 * S - 1]].float().norm()
    assert float(off) < 2 * 2.0 ** -4
    lens = i32([S, S])
    for i in range(steps):
        lens += 1
        w.lens, w.T = [S + i + 1] * 2, 2
        w.rows = ref.rows_of(2, 2, None)
        t = (0.7 * torch.randn((2, (hq + 2 * hkv) * 128), generator=g, device="cuda")).bfloat16()
        t = fq.rope_fwd(t, lens - 1, rope, hq, hkv)
        x = t.double().cpu().numpy().reshape(2, -1, 128)
        fq.kv_cache_append(w.cache, t, i32(w.pages), lens, hq)
        ref.append(w.ref, 0, 64, w.pages, w.lens, w.rows, x[:, hq:].reshape(-1, 2, hkv, 128))
        got = fq.attention_cached(w.cache, t, i32(w.pages), lens, hq)
        w.check_attention(*got, x[:, :hq])
    w.check_cache()


@pytest.mark.parametrize("lens,rows", [([900, 300], 100), ([2000] * 40, 40)])
def test_waits_that_run_out_end_the_call_and_nothing_else(lens, rows):
    """Every wait of the kernel for many rows gives up at once: the status says so, the call returns, and the next call is right."""
    w = World(0, 128, 64, 4, 2, lens, rows=rows, seed=40)
    w.fill()
    t, x = w.append()
    want = fq.attention_cached(w.cache, t, *w.args(), 4)
    torch.cuda.synchronize()
    fq.get_status(clear=True)
    for _ in range(3):
        fq.selftest_attention_cached_wait_limit(w.cache, t, *w.args(), 4, 1e-9)
        torch.cuda.synchronize()
        assert fq.get_status(clear=True) == fq.STATUS_TIMEOUT
    got = fq.attention_cached(w.cache, t, *w.args(), 4)
    torch.cuda.synchronize()
    assert fq.get_status() == 0 and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("lens,rows", [([900, 300], 100), ([128], 100), ([250] * 5, 60)])
def test_waits_that_run_out_after_the_last_copy_leave_none_in_flight(lens, rows):
    """A CTA of one or two blocks has asked for all of its copies when the roles that wait for them give up.  It stays until they have
    landed, so the kernels that follow at once have its shared memory to themselves and are right."""
    w = World(0, 128, 64, 4, 2, lens, rows=rows, seed=45)
    w.fill()
    t, x = w.append()
    want = fq.attention_cached(w.cache, t, *w.args(), 4)
    args = w.args()
    torch.cuda.synchronize()
    fq.get_status(clear=True)
    outs = []
    for _ in range(20):
        fq.selftest_attention_cached_wait_limit(w.cache, t, *args, 4, 1e-9)
        outs.append(fq.attention_cached(w.cache, t, *args, 4))
    torch.cuda.synchronize()
    assert fq.get_status(clear=True) == fq.STATUS_TIMEOUT
    assert all(torch.equal(a, b) for o in outs for a, b in zip(o, want))


def _on_a_stream():
    w = World(0, 128, 64, 8, 2, [130, 64, 1], rows=1, seed=41)
    w.fill()
    t, _ = w.append()
    m = World(0, 64, 32, 4, 1, [300, 90], rows=60, seed=42)
    m.fill()
    s, _ = m.append()
    args, margs = w.args(), m.args()
    return {"attention_cached": (lambda **k: fq.attention_cached(w.cache, t, *args, 8, **k), fq.attention_cached_workspace_size(w.cache, 3, 3, 8)),
            "attention_cached_many": (lambda **k: fq.attention_cached(m.cache, s, *margs, 4, **k), fq.attention_cached_workspace_size(m.cache, 120, 2, 4)),
            "kv_cache_read": (lambda **k: (fq.kv_cache_read(m.cache, *margs, 120, **k),), 0)}


@pytest.mark.parametrize("name", ["attention_cached", "attention_cached_many", "kv_cache_read"])
def test_memory_of_calls_on_another_stream(name):
    """What a call allocates on a busy stream is that stream's: neither its workspace nor its outputs are handed out meanwhile."""
    call, ws = _on_a_stream()[name]
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
    out = call(stream=s)
    junk = [torch.full((max(ws, 1),), 0xA5, dtype=torch.uint8, device="cuda") for _ in range(3)]
    torch.cuda.synchronize()
    assert all(bool((j == 0xA5).all()) for j in junk) and all(torch.equal(a, b) for a, b in zip(out, want))
    torch.cuda.current_stream().wait_stream(s)
    out = call(stream=s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(20_000_000)
    copies, sizes = [t.clone() for t in out], [t.nbytes for t in out]
    del out
    with torch.cuda.stream(s):
        junk = [torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda") for n in sizes]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(copies, want)) and len(junk) == len(want)


def test_appends_on_another_stream_and_captured():
    """kv_cache_append with stream=, and replayed from a graph over a length that the program moves on."""
    w = World(0, 64, 16, 2, 1, [20, 33], rows=1, seed=43)
    w.fill()
    lens = i32([19, 32])
    t = torch.zeros((2, 4 * 64), device="cuda").bfloat16()
    pages = i32(w.pages)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        lens += 1
        fq.kv_cache_append(w.cache, t, pages, lens, 2)
    w.lens = [20, 33]
    v, x = w.qkv()
    t.copy_(v)
    lens.copy_(i32([19, 32]))
    torch.cuda.synchronize()
    graph.replay()
    ref.append(w.ref, 0, 16, w.pages, w.lens, w.rows, x[:, 2:].reshape(-1, 2, 1, 64))
    w.check_cache()
    v, x = w.qkv()  # the same tokens again, larger: the scales grow
    v *= 64
    torch.cuda.synchronize()
    fq.kv_cache_append(w.cache, v, pages, i32(w.lens), 2, stream=side)
    side.synchronize()
    ref.append(w.ref, 0, 16, w.pages, w.lens, w.rows, 64 * x[:, 2:].reshape(-1, 2, 1, 64))
    w.check_cache()


def test_launches_are_traced_and_counted():
    import ctypes
    w = World(0, 64, 16, 2, 1, [20], rows=1, seed=44)
    w.fill()
    t, _ = w.qkv()
    assert fq.lib.fp8q_trace_start(16) == 0
    counts = []
    for call in (lambda: fq.kv_cache_append(w.cache, t, *w.args(), 2), lambda: fq.kv_cache_read(w.cache, *w.args(), 1),
                 lambda: fq.attention_cached(w.cache, t, *w.args(), 2)):
        call()
        counts.append(fq.last_launch_count())
    fq.lib.fp8q_trace_stop()
    torch.cuda.synchronize()
    ms, kinds = (ctypes.c_float * 16)(), (ctypes.c_int * 16)()
    n = fq.lib.fp8q_trace_read(ms, kinds, 16)
    assert [fq.lib.fp8q_kernel_name(kinds[k]).decode() for k in range(n)] == ["kv_append", "kv_read", "attn_cached"]
    assert counts == [1, 1, 2] and all(ms[k] > 0 for k in range(n))
