"""Cases of the 8-bit key/value cache that are timed and compared: writing tokens into it with a scale
for each page and head, reading them back, and attention over it.

``run`` computes an operator in its plain form (elementary torch operations in 32 bits) where ``own`` is
false, and calls the framework's entry points where it is true.  Both return the same outputs of the same
inputs.  Sizes are those of this repository's workloads (40 query and 8 key heads of 128, 28 and 4, 12 and 12
heads of 64, 4096 to 16384 tokens), or generic.

The cache: pages of a few tokens; codes [pages, heads, tokens of a page, head_dim] in E4M3 or E5M2 for K and for
V, and for each page and head the code X + 127 of a scale 2^X: the smallest with which no value of the page is
clipped.  A page that gets a larger token later has its codes shifted to the new scale.
"""

import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
_FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
_EMAX = {"e4m3": 8, "e5m2": 15}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
# n sequences of up to len tokens; rows: the tokens of each in this call (0: all of them); ragged: rows differ from
# sequence to sequence, up to that; idle: a fifth of the sequences are empty slots of a padded batch.
def listed():
    return [
        # one new token for each of 16 running sequences of the 32B class: latency
        {"name": "append_token", "op": "append", "n": 16, "len": 4096, "rows": 1, "ragged": False, "idle": False,
         "hq": 40, "hkv": 8, "dh": 128, "page": 64, "fmt": "e4m3", "dtype": "bf16"},
        # a few drafted tokens for each of many sequences, small pages, an fp32 projection
        {"name": "append_drafts", "op": "append", "n": 61, "len": 2000, "rows": 7, "ragged": True, "idle": False,
         "hq": 12, "hkv": 12, "dh": 64, "page": 16, "fmt": "e5m2", "dtype": "f32"},
        # the prompts of four new sequences, 16384 tokens at most
        {"name": "append_prompts", "op": "append", "n": 4, "len": 4096, "rows": 0, "ragged": True, "idle": False,
         "hq": 40, "hkv": 8, "dh": 128, "page": 64, "fmt": "e4m3", "dtype": "bf16"},
        # one short sequence moved to another machine
        {"name": "read_one", "op": "read", "n": 1, "len": 333, "rows": 0, "ragged": True, "idle": False,
         "hq": 0, "hkv": 4, "dh": 128, "page": 32, "fmt": "e4m3", "dtype": "bf16"},
        # the shared beginnings of long sequences as fp32 rows
        {"name": "read_prefixes", "op": "read", "n": 9, "len": 8191, "rows": 0, "ragged": True, "idle": False,
         "hq": 0, "hkv": 8, "dh": 96, "page": 64, "fmt": "e5m2", "dtype": "f32"},
        # one sequence's next token, a short chat: latency
        {"name": "attend_short", "op": "attend", "n": 1, "len": 301, "rows": 1, "ragged": False, "idle": False,
         "hq": 28, "hkv": 4, "dh": 128, "page": 64, "fmt": "e4m3", "dtype": "bf16"},
        # a running batch of the 32B class, lengths of all kinds, some slots empty
        {"name": "attend_batch", "op": "attend", "n": 64, "len": 8192, "rows": 1, "ragged": False, "idle": True,
         "hq": 40, "hkv": 8, "dh": 128, "page": 64, "fmt": "e4m3", "dtype": "bf16"},
        # one very long document
        {"name": "attend_document", "op": "attend", "n": 1, "len": 250007, "rows": 1, "ragged": False, "idle": False,
         "hq": 28, "hkv": 4, "dh": 128, "page": 128, "fmt": "e4m3", "dtype": "bf16"},
        # drafted tokens checked at once, a narrow model with a key head for each query head
        {"name": "attend_drafts", "op": "attend", "n": 24, "len": 3000, "rows": 6, "ragged": True, "idle": False,
         "hq": 12, "hkv": 12, "dh": 64, "page": 16, "fmt": "e5m2", "dtype": "bf16"},
        # long prompts taken in pieces, each against all that came before
        {"name": "attend_chunk", "op": "attend", "n": 2, "len": 8192, "rows": 512, "ragged": False, "idle": False,
         "hq": 40, "hkv": 8, "dh": 128, "page": 64, "fmt": "e4m3", "dtype": "bf16"},
        # many long sequences: the cache is most of what the card reads
        {"name": "attend_long", "op": "attend", "n": 48, "len": 32768, "rows": 1, "ragged": False, "idle": False,
         "hq": 40, "hkv": 8, "dh": 128, "page": 64, "fmt": "e4m3", "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


_HEADS = [(40, 8), (28, 4), (12, 12), (8, 1), (16, 2), (6, 6), (5, 1)]
_LARGEST = 48 * 32768 * 8 * 128  # elements of K (or V) that a call has in its cache
_MOST = 4 * 2 * 512 * 8192 * 40 * 128  # operations of one call


def draw(rng: random.Random):
    op = rng.choice(["append", "read", "attend", "attend", "attend"])
    hq, hkv = rng.choice(_HEADS)
    c = {"op": op, "hq": hq, "hkv": hkv, "dh": rng.choice([64, 96, 128, 128]), "page": rng.choice([16, 32, 64, 128]),
         "fmt": rng.choice(["e4m3", "e4m3", "e5m2"]), "dtype": rng.choice(["bf16", "bf16", "f32"])}
    if op == "attend":
        c["dtype"] = "bf16"
    if op == "read":
        c["hq"] = 0
    while True:
        n, length = _log(rng, 1, 200), _log(rng, 1, 100000)
        if op == "read" or (op == "append" and rng.random() < 0.5):
            if n * length > 40000:
                continue
            c.update(n=n, len=length, rows=0, ragged=True, idle=False)
            return c
        rows = min(length, rng.choice([1, 1, 1, _log(rng, 2, 8), _log(rng, 8, 512)]))
        ragged = rows > 1 and rng.random() < 0.6
        c.update(n=n, len=length, rows=rows, ragged=ragged, idle=not ragged and rng.random() < 0.3)
        if n * length * hkv * c["dh"] > (_LARGEST if op == "attend" else _LARGEST // 16) or n * rows > 16384:
            continue
        if op == "attend" and 4 * n * rows * length * hq * c["dh"] > _MOST:
            continue
        return c


def _shape(case):
    """Each sequence's length and its tokens in this call: the case's own, whatever the seed."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    lens, rows = [], []
    for i in range(case["n"]):
        longest = max(1, case["len"] if i == 0 else _log(rng, max(1, case["len"] / 8), case["len"]))
        k = case["rows"] or longest
        r = min(longest, k if i == 0 or not case["ragged"] or not case["rows"] else rng.randint(1, k))
        if not case["ragged"]:
            r, longest = k, max(longest, k)
        if case["idle"] and i % 5 == 2:
            longest = 0
        lens.append(longest)
        rows.append(r)
    return lens, rows


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _normal(shape, g, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std


def _exponent(amax, fmt):
    """The smallest X with amax <= fmax 2^X; fmax is 1.75 2^EMAX."""
    mant, exp = torch.frexp(amax)
    x = exp - 1 - _EMAX[fmt] + (2.0 * mant > 1.75).to(torch.int32)
    return torch.where(amax > 0, x.clamp(-127, 127), torch.full_like(x, -127))


def _times2(x, X):
    """x 2^X for whole X from -126 to 127."""
    return x * ((X + 127).clamp(1, 254).to(torch.int32) << 23).view(torch.float32)


def _pool(case, n_pages, g, channels):
    """Pages as a running program has them, every slot written once (recycled pages hold what was there before):
    values of unit size with a few wide channels, pages of a size of their own."""
    hkv, P, dh = case["hkv"], case["page"], case["dh"]
    codes = torch.empty((n_pages, hkv, P, dh), dtype=torch.uint8, device="cuda")
    scale = torch.empty((n_pages, hkv), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // (hkv * P * dh))
    for i in range(0, n_pages, step):
        m = min(step, n_pages - i)
        x = _normal((m, hkv, P, dh), g) * channels
        x *= 0.5 + torch.rand((m, hkv, 1, 1), generator=g, device="cuda")
        X = _exponent(x.abs().amax(dim=(2, 3)), case["fmt"])
        x = _times2(x, -X[:, :, None, None]).to(_F8[case["fmt"]])
        codes[i:i + m] = x.view(torch.uint8)
        scale[i:i + m] = (X + 127).to(torch.uint8)
    return codes, scale


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 6271 + 29)
    lens, rows = _shape(case)
    hq, hkv, dh, P, n = case["hq"], case["hkv"], case["dh"], case["page"], case["n"]
    T = sum(rows)
    need = [-(-length // P) for length in lens]
    width = max(1, max(need))
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    # the table: each sequence's pages in the order of its tokens, -1 behind them
    at = torch.arange(width, device="cuda")[None]
    need_t = torch.tensor(need, device="cuda")[:, None]
    first = torch.cumsum(need_t, dim=0) - need_t
    pages = torch.where(at < need_t, order[(first + at).clamp(max=n_pages - 1)], torch.full_like(order[:1], -1)).contiguous()
    wide = torch.where(torch.rand((dh,), generator=g, device="cuda") < 0.03, 4.0, 1.0)
    flat = torch.ones((dh,), device="cuda")
    k, k_scale = _pool(case, n_pages, g, wide)
    v, v_scale = _pool(case, n_pages, g, flat)
    s = {"case": case, "k": k, "v": v, "k_scale": k_scale, "v_scale": v_scale, "pages": pages, "T": T, "most": max(rows),
         "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"), "row_start": None}
    if case["ragged"]:
        start = [0]
        for r in rows:
            start.append(start[-1] + r)
        s["row_start"] = torch.tensor(start, dtype=torch.int32, device="cuda")
    if case["op"] != "read":
        # the QKV projection's rows (rotated already)
        qkv = _normal((T, hq + 2 * hkv, dh), g)
        qkv[:, hq:hq + hkv] *= wide
        qkv *= 0.5 + torch.rand((T, 1, 1), generator=g, device="cuda")
        s["qkv"] = qkv.view(T, -1).to(_DT[case["dtype"]])
    if own:
        import fp8_absmax_reduce_gb300 as fq
        s["cache"] = fq.KvCache(k, v, k_scale, v_scale, fmt=fq.E4M3 if case["fmt"] == "e4m3" else fq.E5M2)
        if case["op"] == "attend":
            need = fq.attention_cached_workspace_size(s["cache"], T, n, hq)
            s["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def _rows(s):
    """Each row's sequence, its position there, and each sequence's first row and number of rows."""
    case, T = s["case"], s["T"]
    if s["row_start"] is None:
        count = torch.full((case["n"],), T // case["n"], dtype=torch.int64, device="cuda")
        start = torch.arange(case["n"], device="cuda") * (T // case["n"])
    else:
        start = s["row_start"][:-1].long()
        count = s["row_start"][1:].long() - start
    seq = torch.repeat_interleave(torch.arange(case["n"], device="cuda"), count, output_size=T)
    pos = s["lens"].long()[seq] - count[seq] + torch.arange(T, device="cuda") - start[seq]
    return seq, pos, start, count


def _plain_write(s, codes, scale, x, page, slot):
    """x [rows, heads, dh] in 32 bits into slots `slot` of pages `page`."""
    case = s["case"]
    f8, n_pages, hkv = _F8[case["fmt"]], codes.shape[0], case["hkv"]
    amax = torch.zeros((n_pages, hkv), device="cuda").scatter_reduce(0, page[:, None].expand(-1, hkv), x.abs().amax(dim=2), "amax")
    first = torch.full((n_pages,), case["page"], dtype=torch.int64, device="cuda").scatter_reduce(0, page, slot, "amin")
    touched = torch.nonzero(first < case["page"])[:, 0]
    first = first[touched]
    before = scale[touched].to(torch.int32) - 127
    X = _exponent(amax[touched], case["fmt"])
    X = torch.where((first > 0)[:, None], torch.maximum(X, before), X)
    # tokens of these pages that were there before: to the new scale
    old = codes[touched]
    moved = _times2(old.view(f8).float(), (before - X)[:, :, None, None]).to(f8).view(torch.uint8)
    keep = (torch.arange(case["page"], device="cuda")[None] < first[:, None])[:, None, :, None]
    codes[touched] = torch.where(keep, moved, old)
    scale[touched] = (X + 127).to(torch.uint8)
    y = _times2(x, 127 - scale[page].to(torch.int32)[:, :, None])
    y = y.clamp(-_FMAX[case["fmt"]], _FMAX[case["fmt"]]).to(f8).view(torch.uint8)
    codes[page, :, slot] = y


def _plain_append(s):
    case, qkv = s["case"], s["qkv"]
    hq, hkv, dh, P = case["hq"], case["hkv"], case["dh"], case["page"]
    seq, pos, _, _ = _rows(s)
    row = torch.nonzero(pos >= 0)[:, 0]
    seq, pos = seq[row], pos[row]
    page, slot = s["pages"][seq, pos // P].long(), pos % P
    x = qkv.view(-1, hq + 2 * hkv, dh)[row, hq:].float()
    _plain_write(s, s["k"], s["k_scale"], x[:, :hkv], page, slot)
    _plain_write(s, s["v"], s["v_scale"], x[:, hkv:], page, slot)
    return _cache_out(s)


def _cache_out(s):
    f8 = _F8[s["case"]["fmt"]]
    return s["k"].view(f8), s["v"].view(f8), s["k_scale"], s["v_scale"]


def _plain_read(s):
    case = s["case"]
    P, f8 = case["page"], _F8[case["fmt"]]
    seq, pos, _, _ = _rows(s)
    page, slot = s["pages"][seq, pos // P].long(), pos % P
    both = [_times2(c[page, :, slot].view(f8).float(), x[page].to(torch.int32)[:, :, None] - 127)
            for c, x in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"]))]
    return torch.cat(both, dim=1).view(s["T"], -1).to(_DT[case["dtype"]])


def _plain_attend(s):
    case, T, most = s["case"], s["T"], s["most"]
    hq, hkv, dh, n, f8 = case["hq"], case["hkv"], case["dh"], case["n"], _F8[case["fmt"]]
    group = hq // hkv
    seq, pos, start, count = _rows(s)
    pages = s["pages"].clamp(min=0).long()
    K, V = (_times2(c[pages].view(f8).float(), x[pages].to(torch.int32)[..., None, None] - 127)
            .transpose(1, 2).reshape(n, hkv, -1, dh) for c, x in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])))
    j = torch.arange(most, device="cuda")[None]
    row = (start[:, None] + j).clamp(max=T - 1)
    q = s["qkv"].view(T, -1, dh)[row, :hq].float().view(n, most, hkv, group, dh)
    q = q.permute(0, 2, 1, 3, 4).reshape(n, hkv, most * group, dh)
    z = (q @ K.transpose(2, 3)) * (1.0 / math.sqrt(dh))
    last = s["lens"].long()[:, None] - count[:, None] + j  # the last key that a row sees
    hidden = torch.arange(K.shape[2], device="cuda") > last.repeat_interleave(group, dim=1)[:, None, :, None]
    z = z.masked_fill_(hidden, -math.inf)
    m = z.amax(dim=3, keepdim=True).clamp(min=-1e30)
    p = torch.exp(z - m)
    total = p.sum(dim=3, keepdim=True)
    out = (p @ V) / total.clamp(min=1e-30)
    lse = (m + torch.log(total))[..., 0]
    k = torch.arange(T, device="cuda") - start[seq]
    out = out.view(n, hkv, most, group, dh)[seq, :, k].reshape(T, hq * dh)
    lse = lse.view(n, hkv, most, group)[seq, :, k].reshape(T, hq).t().contiguous()
    return out.to(torch.bfloat16), lse


def run(state):
    s = state
    op, hq = s["case"]["op"], s["case"]["hq"]
    if own:
        import fp8_absmax_reduce_gb300 as fq
        if op == "append":
            fq.kv_cache_append(s["cache"], s["qkv"], s["pages"], s["lens"], hq, row_start=s["row_start"])
            return _cache_out(s)
        if op == "read":
            return fq.kv_cache_read(s["cache"], s["pages"], s["lens"], s["T"], row_start=s["row_start"],
                                    dtype=_DT[s["case"]["dtype"]])
        return fq.attention_cached(s["cache"], s["qkv"], s["pages"], s["lens"], hq, row_start=s["row_start"], ws=s["ws"])
    if op == "append":
        return _plain_append(s)
    if op == "read":
        return _plain_read(s)
    return _plain_attend(s)


def work(case):
    lens, rows = _shape(case)
    hkv, dh, P = case["hkv"], case["dh"], case["page"]
    e = 2 if case["dtype"] == "bf16" else 4
    T = sum(r for r, length in zip(rows, lens) if length)
    table = 4 * sum(-(-length // P) for length in lens) + 8 * case["n"]
    if case["op"] == "append":  # K and V of the rows in; codes out; the scales of the pages that they touch
        touched = sum((length - 1) // P - (length - r) // P + 1 for r, length in zip(rows, lens) if length)
        return {"bytes": 2 * T * hkv * dh * (e + 1) + 4 * touched * hkv + 4 * touched + 8 * case["n"], "flops": 3 * 2 * T * hkv * dh}
    if case["op"] == "read":  # codes and scales in; rows out
        return {"bytes": 2 * T * hkv * dh * (1 + e) + table // 4 * 2 * hkv + table, "flops": 2 * T * hkv * dh}
    # codes, scales and q in; att and lse out; the two products over the keys that each row sees
    hq = case["hq"]
    keys = sum(r * length - r * (r - 1) // 2 for r, length in zip(rows, lens) if length)
    return {"bytes": 2 * sum(lens) * hkv * dh + table // 4 * 2 * hkv + table + 4 * sum(rows) * hq * dh + 4 * sum(rows) * hq,
            "flops": 4 * keys * hq * dh}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _values(fmt):
    """What each of the 256 codes stands for."""
    man = 3 if fmt == "e4m3" else 2
    bias = 7 if fmt == "e4m3" else 15
    v = []
    for code in range(256):
        e, m = (code & 127) >> man, code & ((1 << man) - 1)
        x = math.ldexp(m, 1 - bias - man) if e == 0 else math.ldexp((1 << man) + m, e - bias - man)
        if fmt == "e5m2" and e == 31:
            x = math.nan if m else math.inf
        if fmt == "e4m3" and (code & 127) == 127:
            x = math.nan
        v.append(-x if code & 128 else x)
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def exact(case, seed):
    s = prepare(case, seed)
    lens, rows = _shape(case)
    hq, hkv, dh, P = case["hq"], case["hkv"], case["dh"], case["page"]
    value = _values(case["fmt"])

    def held(i, codes, scale, upto):
        """Tokens 0 .. upto - 1 of sequence i, [heads, upto, dh]."""
        p = s["pages"][i, :-(-upto // P)].long()
        x = value[codes[p].int()] * torch.exp2(scale[p].double() - 127.0)[:, :, None, None]
        return x.transpose(0, 1).reshape(hkv, -1, dh)[:, :upto]

    if case["op"] == "read":
        out = [torch.cat([held(i, s["k"], s["k_scale"], n), held(i, s["v"], s["v_scale"], n)]).transpose(0, 1).reshape(n, -1)
               for i, n in enumerate(lens)]
        return torch.cat(out)
    qkv = s["qkv"].double().view(-1, hq + 2 * hkv, dh)
    first = 0
    if case["op"] == "append":
        # values over the page's new scale, not rounded to a code
        got = []
        for name, h0 in (("k", hq), ("v", hq + hkv)):
            out = value[s[name].int()]
            new_scale = s[name + "_scale"].clone()
            first = 0
            for i, (r, n) in enumerate(zip(rows, lens)):
                at = n - r
                while n and at < n:
                    page, slot = int(s["pages"][i, at // P]), at % P
                    m = min(P - slot, n - at)
                    x = qkv[first + at - (n - r):first + at - (n - r) + m, h0:h0 + hkv].transpose(0, 1)
                    amax = x.abs().amax(dim=(1, 2))
                    X = torch.ceil(torch.log2(amax / _FMAX[case["fmt"]]))
                    X = torch.where(amax > _FMAX[case["fmt"]] * torch.exp2(X), X + 1, X)
                    X = torch.where(amax <= _FMAX[case["fmt"]] * torch.exp2(X - 1), X - 1, X)
                    was = s[name + "_scale"][page].double() - 127.0
                    if slot:
                        X = torch.maximum(X, was)
                        out[page, :, :slot] *= torch.exp2(was - X)[:, None, None]
                    out[page, :, slot:slot + m] = x * torch.exp2(-X)[:, None, None]
                    new_scale[page] = (X + 127).to(torch.uint8)
                    at += m
                first += r
            got.append((out, new_scale))
        return got[0][0], got[1][0], got[0][1], got[1][1]
    att = torch.zeros((s["T"], hq, dh), dtype=torch.float64, device="cuda")
    lse = torch.full((hq, s["T"]), -math.inf, dtype=torch.float64, device="cuda")
    for i, (r, n) in enumerate(zip(rows, lens)):
        if n:
            K, V = held(i, s["k"], s["k_scale"], n), held(i, s["v"], s["v_scale"], n)
            late = torch.arange(n, device="cuda")[None] > torch.arange(n - r, n, device="cuda")[:, None]
            for h in range(hq):
                z = torch.einsum("jd,kd->jk", qkv[first:first + r, h], K[h // (hq // hkv)]) / math.sqrt(dh)
                z = z.masked_fill(late, -math.inf)
                lse[h, first:first + r] = torch.logsumexp(z, dim=1)
                att[first:first + r, h] = torch.softmax(z, dim=1) @ V[h // (hq // hkv)]
        first += r
    return att.view(s["T"], -1), lse
