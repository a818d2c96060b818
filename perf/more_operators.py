"""Rotary positions and the int8 KV cache's operators as measured workloads.

Operators: ``rope`` (rotary positions of query and key rows, with an optional RMS
norm per head, and its gradient), ``rows`` (K/V rows quantised into int8 cells
and read back as the values the cache stands for), ``write`` (a step's rows:
queries rotated, keys rotated and quantised, values quantised; then read back)
and ``decode`` (attention of one new token per sequence over int8 cells that
block tables name).  ``run`` computes them with elementary torch operations, or,
where ``own`` is true, with the library's calls.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one decode step of a serving batch: queries and keys of 48 requests (latency)
        dict(name="rope step 48", op="rope", rows=48, pad=16, hq=32, hkv=8, d=128, rot=128, layout="half", type="bf16",
             scaling="plain", norm=False, inverse=False, max_pos=32768, spread=1),
        # a long prompt chunk, the first half of each head rotated, positions divided for a longer context
        dict(name="rope chunk 20001", op="rope", rows=20001, pad=0, hq=32, hkv=8, d=128, rot=64, layout="interleaved",
             type="f16", scaling="linear", norm=False, inverse=False, max_pos=131072, spread=2),
        # the gradient of the rotation at far positions, in 32 bits
        dict(name="rope gradient 5000 f32", op="rope", rows=5000, pad=0, hq=32, hkv=8, d=128, rot=128, layout="half",
             type="f32", scaling="pairs", norm=False, inverse=True, max_pos=1000000, spread=3),
        # one decode step's rows of 40 requests into the cache, heads normed first (latency)
        dict(name="write step 40", op="write", rows=40, pad=24, hq=32, hkv=8, d=128, dv=128, rot=128, layout="half",
             type="bf16", scaling="plain", norm=True, page=16, max_pos=32768, spread=4),
        # the rows of long prompt chunks into the cache
        dict(name="write chunk 16001", op="write", rows=16001, pad=0, hq=32, hkv=8, d=128, dv=128, rot=128,
             layout="half", type="f16", scaling="rotations", norm=False, page=64, max_pos=131072, spread=5),
        # a few rows without positions (values that were rotated before, or need none)
        dict(name="rows 64 bf16", op="rows", rows=64, hkv=8, d=128, dv=128, page=16, type="bf16"),
        # a long prompt's rows
        dict(name="rows 20001 f16", op="rows", rows=20001, hkv=8, d=128, dv=128, page=64, type="f16"),
        # one short conversation: latency
        dict(name="decode 1x700", op="decode", n_seq=1, max_len=700, min_len=700, hq=32, hkv=8, d=128, dv=128,
             page=16, type="bf16", spread=6),
        # one long context, 8 KV and 32 query heads
        dict(name="decode 1x32768", op="decode", n_seq=1, max_len=32768, min_len=32768, hq=32, hkv=8, d=128, dv=128,
             page=64, type="f16", spread=7),
        # a serving batch of ragged contexts
        dict(name="decode 40 ragged", op="decode", n_seq=40, max_len=32768, min_len=3, hq=32, hkv=8, d=128, dv=128,
             page=32, type="bf16", spread=8),
        # short contexts of many requests, small heads, eight query heads a KV head
        dict(name="decode 100 small heads", op="decode", n_seq=100, max_len=2100, min_len=1, hq=32, hkv=4, d=64, dv=64,
             page=16, type="f16", spread=9),
        # very long contexts over single scattered cells, the largest read
        dict(name="decode 6x140000 cells", op="decode", n_seq=6, max_len=140000, min_len=90000, hq=32, hkv=8, d=128,
             dv=128, page=1, type="bf16", spread=10),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "rows", "write", "write", "decode", "decode", "decode"])
    hkv, spread = rng.choice([1, 2, 4, 8]), rng.randrange(1 << 20)
    if op == "decode":
        d, dv = rng.choice([(64, 64), (80, 80), (128, 128), (128, 128), (192, 128), (256, 256)])
        n = _log(rng, 1, 100)
        return dict(op=op, n_seq=n, max_len=_log(rng, 1, min(140000, 700000 // n)), min_len=1,
                    hq=hkv * rng.choice([1, 2, 3, 4, 7, 8, 16]), hkv=hkv, d=d, dv=dv,
                    page=rng.choice([1, 16, 32, 64, 256]), type=rng.choice(["f16", "bf16"]), spread=spread)
    if op == "rows":
        return dict(op=op, rows=_log(rng, 1, 20000), hkv=hkv, d=rng.choice([64, 80, 128, 256]),
                    dv=rng.choice([64, 96, 128]), page=rng.choice([1, 16, 64]), type=rng.choice(["f32", "f16", "bf16"]))
    d = rng.choice([64, 80, 96, 128, 128, 256])
    case = dict(op=op, rows=_log(rng, 1, 12000), pad=rng.choice([0, 0, 5, 37]), hq=hkv * rng.choice([1, 2, 4, 7]),
                hkv=hkv, d=d, rot=rng.choice([d, d, d // 2, d // 4]), layout=rng.choice(["half", "interleaved"]),
                scaling=rng.choice(["plain", "linear", "base", "rotations", "pairs"]), norm=rng.random() < 0.4,
                max_pos=_log(rng, 10, 1000000), spread=spread)
    if op == "rope":
        inverse = not case["norm"] and rng.random() < 0.4
        return dict(case, inverse=inverse, type=rng.choice(["f32", "f16", "bf16"]))
    return dict(case, dv=rng.choice([64, 128]), page=rng.choice([1, 16, 64]), type=rng.choice(["f16", "bf16"]))


def _lens(case):
    """Lengths of the sequences: the first has the most, the others are spread over the range."""
    r = random.Random(case["spread"])
    lo = min(case["min_len"], case["max_len"])
    return [case["max_len"] if i == 0 else r.randint(lo, case["max_len"]) for i in range(case["n_seq"])]


# base of the frequencies, and (factor, original length, rotations of the fast and of the slow end) of the scalings
BASE, FACTOR, ORIGINAL, FAST, SLOW = 500000.0, 8.0, 8192.0, 32.0, 1.0


def _frequencies(case):
    """Radians per position of each pair, and the factor on the rotated values."""
    rot, kind = case["rot"], case["scaling"]
    base = BASE * FACTOR ** (rot / (rot - 2)) if kind == "base" else BASE
    f = [base ** (-2.0 * j / rot) for j in range(rot // 2)]
    if kind == "linear":
        f = [x / FACTOR for x in f]
    if kind == "rotations":                       # by how often a pair turns within the original length
        part = [min(1.0, max(0.0, (ORIGINAL * x / (2 * math.pi) - SLOW) / (FAST - SLOW))) for x in f]
        f = [x * p + x / FACTOR * (1 - p) for x, p in zip(f, part)]
    if kind == "pairs":                           # by the pair's number between those that turn so often
        at = [rot * math.log(ORIGINAL / (2 * math.pi * b)) / (2 * math.log(BASE)) for b in (FAST, SLOW)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        hi = hi + 0.001 if hi == lo else hi
        slow = [min(1.0, max(0.0, (j - lo) / (hi - lo))) for j in range(rot // 2)]
        f = [x / FACTOR * s + x * (1 - s) for x, s in zip(f, slow)]
    return f, (0.1 * math.log(FACTOR) + 1.0 if kind == "pairs" else 1.0)


# ---------------------------------------------------------------- inputs

def _activations(g, n, h, d):
    """Rows like a projection's: N(0, 1), with a few channels of each head eight times as large, and an offset."""
    x = torch.randn((n, h, d), generator=g, device="cuda")
    big = torch.randint(0, d, (h, max(1, d // 32)), generator=g, device="cuda")
    gain = torch.ones((h, d), device="cuda").scatter_(1, big, 8.0)
    return x * gain + 0.2 * torch.randn((h, d), generator=g, device="cuda")


def _quantise(x):
    """int8 codes and 16-bit scales of rows: scale = max |x| / 127, code = round(x / scale)."""
    s = (x.abs().amax(-1, keepdim=True) / 127).half().float()
    c = torch.where(s > 0, torch.round(x / torch.where(s > 0, s, torch.ones_like(s))).clamp(-127, 127),
                    torch.zeros_like(x))
    return c.to(torch.int8), s[..., 0].half()


def _pool(g, n_cells, h, d):
    """Cells filled with quantised rows."""
    rows = torch.empty((n_cells, h, d), dtype=torch.int8, device="cuda")
    scales = torch.empty((n_cells, h), dtype=torch.float16, device="cuda")
    step = max(1, (1 << 27) // (h * d))
    for i in range(0, n_cells, step):
        n = min(step, n_cells - i)
        rows[i:i + n], scales[i:i + n] = _quantise(_activations(g, n, h, d))
    return rows, scales


def _positions(g, case):
    """Positions of a step's rows: runs of several prompt chunks, or single tokens; -1 in the rows behind them."""
    n, r = case["rows"], random.Random(case["spread"])
    chunks = n if n <= 64 else 5
    cuts = sorted(r.randint(0, n) for _ in range(chunks - 1)) if chunks < n else list(range(1, n))
    pos, at = [], 0
    for end in cuts + [n]:
        first = r.randint(0, max(0, case["max_pos"] - (end - at)))
        pos.append(torch.arange(first, first + end - at))
        at = end
    pos.append(torch.full((case["pad"],), -1))
    return torch.cat(pos).to(torch.int32).cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, st = case["op"], {"case": case}
    if op == "decode":
        lens, page, hkv = _lens(case), case["page"], case["hkv"]
        need = [-(-n // page) for n in lens]
        pool = sum(need) + 3
        perm = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
        st["table"] = torch.zeros((len(lens), max(need)), dtype=torch.int32, device="cuda")
        at = 0
        for i, n in enumerate(need):
            st["table"][i, :n] = perm[at:at + n]
            at += n
        st["len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        st["k_rows"], st["k_scales"] = _pool(g, pool * page, hkv, case["d"])
        st["v_rows"], st["v_scales"] = _pool(g, pool * page, hkv, case["dv"])
        st["q"] = _activations(g, len(lens), case["hq"], case["d"]).to(DT[case["type"]])
        st["scale"] = 1.0 / math.sqrt(case["d"])
        if own:
            import quantized_kv_cache_tq_gb300 as tq
            st["k"] = tq.Int8Cache.from_planes(st["k_rows"], st["k_scales"])
            st["v"] = tq.Int8Cache.from_planes(st["v_rows"], st["v_scales"])
            st["out"] = torch.empty((len(lens), case["hq"], case["dv"]), dtype=st["q"].dtype, device="cuda")
            st["ws"] = tq.workspace(tq.int8_decode_workspace(st["k"], st["v"], case["hq"], len(lens)))
        return st
    n, typ, hkv = case["rows"] + case.get("pad", 0), DT[case["type"]], case["hkv"]
    heads = [("k", hkv, case["d"])]
    if op != "rope":
        heads.append(("v", hkv, case["dv"]))
        page = case["page"]
        cells = torch.randperm(-(-n // page) + 2, generator=g, device="cuda")
        slots = (cells[:, None] * page + torch.arange(page, device="cuda")).reshape(-1)
        st["slots"] = torch.cat([slots[:case["rows"]],
                                 torch.full((n - case["rows"],), -1, dtype=torch.int64, device="cuda")])
        for x, h, d in heads:
            st[x + "_rows"] = torch.zeros((len(slots), h, d), dtype=torch.int8, device="cuda")
            st[x + "_scales"] = torch.zeros((len(slots), h), dtype=torch.float16, device="cuda")
    if op != "rows":
        heads.append(("q", case["hq"], case["d"]))
        st["pos"] = _positions(g, case)
        f, st["gain"] = _frequencies(case)
        st["freq"] = torch.tensor(f, dtype=torch.float64, device="cuda")
        for x in ("q", "k"):
            st[x + "_norm"] = (1 + 0.1 * torch.randn((case["d"],), generator=g, device="cuda")) if case["norm"] else None
    for x, h, d in heads:
        st[x + "_src"] = _activations(g, n, h, d).to(typ)
        st[x + "_out"] = torch.zeros((n, h, d), dtype=typ, device="cuda")
    if own:
        import quantized_kv_cache_tq_gb300 as tq
        if op != "rows":
            st["rope"] = tq.Rope(case["rot"], BASE, layout=case["layout"], scaling=case["scaling"], factor=FACTOR,
                                 original_len=ORIGINAL, beta_fast=FAST, beta_slow=SLOW)
        if op != "rope":
            st["k"] = tq.Int8Cache.from_planes(st["k_rows"], st["k_scales"])
            st["v"] = tq.Int8Cache.from_planes(st["v_rows"], st["v_scales"])
    return st


# ---------------------------------------------------------------- the plain forms

def _turned(st, x):
    """Rows of st[x + "_src"], normed and rotated, in 32 bits (the angles in 64)."""
    case, y = st["case"], st[x + "_src"].float()
    if st[x + "_norm"] is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * st[x + "_norm"]
    angle = st["pos"].double()[:, None] * st["freq"]
    c, s = (torch.cos(angle) * st["gain"]).float()[:, None], (torch.sin(angle) * st["gain"]).float()[:, None]
    if case.get("inverse"):
        s = -s
    rot = case["rot"]
    if case["layout"] == "half":
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat([a * c - b * s, a * s + b * c], -1)
    else:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    return torch.cat([turned, y[..., rot:]], -1)


def _kept(st, x, y, live):
    """Rows that the call writes, rounded; the others as they were."""
    return torch.where(live[:, None, None], y.to(st[x + "_out"].dtype), st[x + "_out"])


def _stored(st, x, y, live):
    """Rows y into the cells, and back as the values that these stand for."""
    at = st["slots"][live]
    codes, scales = _quantise(y[live])
    st[x + "_rows"][at], st[x + "_scales"][at] = codes, scales
    at = torch.where(live, st["slots"], torch.zeros_like(st["slots"]))
    back = st[x + "_rows"][at].float() * st[x + "_scales"][at].float()[..., None]
    return _kept(st, x, back, live)


def _rows_plain(st):
    op = st["case"]["op"]
    if op == "rows":
        live = st["slots"] >= 0
        return [_stored(st, x, st[x + "_src"].float(), live) for x in ("k", "v")]
    live = st["pos"] >= 0
    q = _kept(st, "q", _turned(st, "q"), live)
    if op == "rope":
        return [q, _kept(st, "k", _turned(st, "k"), live)]
    return [q, _stored(st, "k", _turned(st, "k"), live), _stored(st, "v", st["v_src"].float(), live)]


def _decode_plain(st):
    case, q, page = st["case"], st["q"].float(), st["case"]["page"]
    n, hq, d = q.shape
    cells = (st["table"].long()[:, :, None] * page + torch.arange(page, device=q.device)).flatten(1)
    live = torch.arange(cells.shape[1], device=q.device) < st["len"].long()[:, None]
    qg = q.reshape(n, case["hkv"], hq // case["hkv"], d)
    k = st["k_rows"][cells].float() * st["k_scales"][cells].float()[..., None]           # [n, L, KV heads, d]
    s = torch.matmul(qg, k.permute(0, 2, 3, 1)) * st["scale"]
    del k
    s = torch.where(live[:, None, None], s, torch.full_like(s, -math.inf))
    p = torch.exp(s - s.amax(-1, keepdim=True))
    v = st["v_rows"][cells].float() * st["v_scales"][cells].float()[..., None]
    o = torch.matmul(p / p.sum(-1, keepdim=True), v.transpose(1, 2))
    return o.flatten(1, 2).to(st["q"].dtype)


# ---------------------------------------------------------------- one pass

def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        return _decode_plain(st) if op == "decode" else _rows_plain(st)
    import quantized_kv_cache_tq_gb300 as tq
    if op == "decode":
        return tq.int8_decode(st["k"], st["v"], st["table"], st["len"], st["q"], st["scale"], page_size=case["page"],
                              out=st["out"], ws=st["ws"])
    if op == "rope":
        return tq.rope_rows(st["rope"], st["pos"], st["q_src"], st["k_src"], q_norm=st["q_norm"], k_norm=st["k_norm"],
                            eps=EPS, inverse=case["inverse"], q_out=st["q_out"], k_out=st["k_out"])
    if op == "rows":
        tq.int8_set_rows(st["k"], st["v"], st["k_src"], st["v_src"], st["slots"])
        return tq.int8_get_rows(st["k"], st["v"], st["slots"], k_out=st["k_out"], v_out=st["v_out"])
    q = tq.int8_rope_set_rows(st["k"], st["v"], st["rope"], st["pos"], st["q_src"], st["k_src"], st["v_src"],
                              st["slots"], q_norm=st["q_norm"], k_norm=st["k_norm"], eps=EPS, q_out=st["q_out"])
    return (q, *tq.int8_get_rows(st["k"], st["v"], st["slots"], k_out=st["k_out"], v_out=st["v_out"]))


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op, hkv, size = case["op"], case["hkv"], torch.finfo(DT[case["type"]]).bits // 8
    if op == "decode":
        lens = _lens(case)
        cells, wide = sum(lens), case["d"] + case["dv"]
        return {"bytes": cells * hkv * (wide + 4) + len(lens) * (case["hq"] * size * wide + 4)
                + 4 * sum(-(-n // case["page"]) for n in lens), "flops": 2 * cells * case["hq"] * wide}
    rows = case["rows"]
    if op == "rope":
        n = rows * (case["hq"] + hkv) * case["d"]
        return {"bytes": 2 * size * n + 4 * rows, "flops": (8 if case["norm"] else 4) * n}
    # a source row is read, its cell written, the cell read, its values written
    n = rows * hkv
    got = {"bytes": n * sum(2 * size * d + 2 * (d + 2) for d in (case["d"], case["dv"])) + 16 * rows,
           "flops": 6 * n * (case["d"] + case["dv"])}
    if op == "write":
        q = rows * case["hq"] * case["d"]
        got["bytes"] += 2 * size * q + 4 * rows
        got["flops"] += (8 if case["norm"] else 4) * (q + n * case["d"])
    return got


# ---------------------------------------------------------------- the definition, in 64 bits

def _exact_turned(case, x, pos, norm):
    y = x.double()
    if norm is not None:
        y = y / torch.sqrt((y ** 2).sum(-1, keepdim=True) / y.shape[-1] + EPS) * norm.double()
    f, gain = _frequencies(case)
    out, half = y.clone(), case["rot"] // 2
    for j in range(half):
        a, b = (j, j + half) if case["layout"] == "half" else (2 * j, 2 * j + 1)
        t = pos.double() * (-f[j] if case.get("inverse") else f[j])
        z = torch.complex(y[..., a], y[..., b]) * torch.polar(torch.full_like(t, gain), t)[:, None]
        out[..., a], out[..., b] = z.real, z.imag
    return out


def _exact_values(y):
    step = (y.abs().max(-1, keepdim=True).values / 127).to(torch.float16).double()
    return (y / step).nan_to_num(0.0).round().clamp(-127, 127) * step


def exact(case, seed):
    op = case["op"]
    st = prepare(case, seed)
    if op == "decode":
        g, page = case["hq"] // case["hkv"], case["page"]
        out = torch.zeros((case["n_seq"], case["hq"], case["dv"]), dtype=torch.float64, device="cuda")
        for s, n in enumerate(_lens(case)):
            t = torch.arange(n, device="cuda")
            cell = st["table"][s].long()[t // page] * page + t % page
            for h in range(case["hkv"]):
                k = st["k_rows"][cell, h].double() * st["k_scales"][cell, h].double()[:, None]
                v = st["v_rows"][cell, h].double() * st["v_scales"][cell, h].double()[:, None]
                x = st["q"][s, h * g:(h + 1) * g].double() @ k.T * st["scale"]
                out[s, h * g:(h + 1) * g] = torch.softmax(x, -1) @ v
        return out
    live = (st["slots"] if op == "rows" else st["pos"]) >= 0
    gone = lambda y: torch.where(live[:, None, None], y, torch.zeros_like(y))  # noqa: E731
    if op == "rows":
        return [gone(_exact_values(st[x + "_src"].double())) for x in ("k", "v")]
    q, k = (_exact_turned(case, st[x + "_src"], st["pos"], st[x + "_norm"]) for x in ("q", "k"))
    if op == "rope":
        return [gone(q), gone(k)]
    return [gone(q), gone(_exact_values(k)), gone(_exact_values(st["v_src"].double()))]
