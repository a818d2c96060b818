"""The paged 4-bit KV cache's operators as measured workloads.

Operators: ``plan`` (block tables and slot maps from request lengths), ``rows``
(K/V rows quantised into 4-bit pages and read back as the values the cache
stands for), ``decode`` and ``prefill`` (attention of one or many query rows per
sequence over the pages), ``diff_decode`` and ``diff_prefill`` (the same with
the difference of two softmax maps).  ``run`` computes them with elementary
torch operations, or, where ``own`` is true, with the library's calls.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # a decode step of a small serving batch: the planner before every step (latency)
        dict(name="plan step 48", op="plan", n_seq=48, max_new=1, max_len=8000, page=16, spread=1),
        # admission of many prompts at once, with finished requests returning their pages
        dict(name="plan admit 700", op="plan", n_seq=700, max_new=3000, max_len=6000, page=32, spread=2),
        # one decode step's rows of 32 requests (latency)
        dict(name="rows 32 bf16", op="rows", rows=32, hkv=8, dk=128, dv=128, page=16, type="bf16"),
        # the rows of a long prompt chunk
        dict(name="rows 20001 f16", op="rows", rows=20001, hkv=8, dk=128, dv=128, page=64, type="f16"),
        # one short conversation: latency
        dict(name="decode 1x900", op="decode", n_seq=1, max_len=900, min_len=900, hq=32, hkv=8, dk=128, dv=128,
             page=16, type="bf16", spread=3),
        # one long context, 8 KV and 32 query heads
        dict(name="decode 1x32768", op="decode", n_seq=1, max_len=32768, min_len=32768, hq=32, hkv=8, dk=128, dv=128,
             page=64, type="f16", spread=4),
        # a serving batch of ragged contexts, the largest read
        dict(name="decode 40 ragged", op="decode", n_seq=40, max_len=32768, min_len=3, hq=32, hkv=8, dk=128, dv=128,
             page=32, type="bf16", spread=5),
        # prompt chunks of several short requests together
        dict(name="prefill 5x300", op="prefill", n_seq=5, max_rows=300, max_len=1500, hq=32, hkv=8, dk=128, dv=128,
             page=16, type="bf16", spread=6),
        # a 2048-row chunk at the end of a long context, the most arithmetic
        dict(name="prefill 2048 at 32768", op="prefill", n_seq=1, max_rows=2048, max_len=32768, hq=32, hkv=8, dk=128,
             dv=128, page=64, type="f16", spread=7),
        # differential attention, single token: K heads of 64 in pairs, V heads of 128
        dict(name="diff decode 12", op="diff_decode", n_seq=12, max_len=9000, min_len=100, hq=16, hkv=8, dk=64,
             dv=128, page=32, type="bf16", norm=True, spread=8),
        dict(name="diff decode 1x2000", op="diff_decode", n_seq=1, max_len=2000, min_len=2000, hq=8, hkv=8, dk=128,
             dv=128, page=16, type="f16", norm=False, spread=9),
        # differential attention over prompt chunks
        dict(name="diff prefill 3x700", op="diff_prefill", n_seq=3, max_rows=700, max_len=4000, hq=16, hkv=8, dk=64,
             dv=128, page=32, type="bf16", norm=True, spread=10),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "rows", "decode", "decode", "prefill", "prefill", "diff_decode", "diff_prefill"])
    page, typ, spread = rng.choice([16, 32, 64, 128]), rng.choice(["f16", "bf16"]), rng.randrange(1 << 20)
    if op == "plan":
        return dict(op=op, n_seq=_log(rng, 1, 1500), max_new=rng.choice([1, 1, _log(rng, 2, 1200)]),
                    max_len=_log(rng, 20, 6000), page=page, spread=spread)
    hkv = rng.choice([1, 2, 4, 8])
    if op == "rows":
        return dict(op=op, rows=_log(rng, 1, 20000), hkv=hkv, dk=rng.choice([64, 80, 128]),
                    dv=rng.choice([64, 96, 128]), page=page, type=typ)
    diff = op.startswith("diff")
    dk, dv = rng.choice([(64, 64), (64, 128), (128, 128)] if diff else [(64, 64), (80, 80), (128, 128), (128, 128)])
    hq = hkv * rng.choice([1, 2, 4] if diff else [1, 2, 3, 4, 7, 8])
    case = dict(op=op, hq=hq, hkv=hkv, dk=dk, dv=dv, page=page, type=typ, spread=spread)
    if diff:
        case["norm"] = rng.random() < 0.7
    if op.endswith("decode"):
        n = _log(rng, 1, 48)
        return dict(case, n_seq=n, max_len=_log(rng, 1, min(32768, 400000 // n)), min_len=1)
    n = rng.choice([1, 1, 2, 3, 6])
    rows = _log(rng, 1, 2000 // n)
    return dict(case, n_seq=n, max_rows=rows, max_len=max(rows, _log(rng, 16, 24000 // n)))


def _lens(case):
    """Lengths of the sequences: the first has the most, the others are spread over the range."""
    r = random.Random(case["spread"])
    lo = case.get("min_len", 1)
    return [case["max_len"] if i == 0 else r.randint(lo, case["max_len"]) for i in range(case["n_seq"])]


def _rows(case):
    """(query rows, context lengths) of a prompt batch's sequences."""
    r = random.Random(case["spread"])
    nq = [case["max_rows"] if i == 0 else r.randint(0, case["max_rows"]) for i in range(case["n_seq"])]
    return nq, [case["max_len"] if i == 0 else r.randint(n, case["max_len"]) for i, n in enumerate(nq)]


def _requests(case):
    """(cells held, new tokens) of a planner's requests; -cells: the request ends and returns its pages."""
    r = random.Random(case["spread"])
    old, new = [], []
    for _ in range(case["n_seq"]):
        have = r.choice([0, r.randint(0, case["max_len"])]) if case["max_new"] > 1 else r.randint(1, case["max_len"])
        u = r.random()
        old.append(have)
        new.append(-have if u < 0.05 else 0 if u < 0.1 else r.randint(1, case["max_new"]))
    return old, new


def _up(x, a):
    return -(-x // a) * a


def _width(d):
    return 64 if d <= 64 else 128 if d <= 128 else 256


def _pages(n, page):
    return -(-n // page)


# ---------------------------------------------------------------- inputs

def _activations(g, n, h, d):
    """Rows like a projection's: N(0, 1), with a few channels of each head eight times as large, and an offset."""
    x = torch.randn((n, h, d), generator=g, device="cuda")
    big = torch.randint(0, d, (h, max(1, d // 32)), generator=g, device="cuda")
    gain = torch.ones((h, d), device="cuda").scatter_(1, big, 8.0)
    return x * gain + 0.2 * torch.randn((h, d), generator=g, device="cuda")


def _quantise(x):
    """Codes (0..15) and (scale, offset) of rows: offset = min, scale = (max - min) / 15, both in 16 bits."""
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    m = lo.half().float()
    s = ((hi - lo) / 15).half().float()
    c = torch.where(s > 0, torch.round((x - m) / torch.where(s > 0, s, torch.ones_like(s))).clamp(0, 15),
                    torch.zeros_like(x))
    return c.to(torch.uint8), torch.cat([s, m], -1).half()


def _pack(c, width):
    """Two codes a byte, the even element in the low four bits; rows filled up with zero codes to their stored width."""
    c = torch.nn.functional.pad(c, (0, width - c.shape[-1]))
    return c[..., 0::2] | (c[..., 1::2] << 4)


def _pool(g, n_pages, h, page, d):
    """A pool of pages filled with quantised rows."""
    codes = torch.empty((n_pages, h, page, _width(d) // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((n_pages, h, page, 2), dtype=torch.float16, device="cuda")
    step = max(1, (1 << 26) // (h * page * d))
    for i in range(0, n_pages, step):
        n = min(step, n_pages - i)
        c, s = _quantise(_activations(g, n * page, h, d))
        codes[i:i + n] = _pack(c, _width(d)).reshape(n, page, h, -1).transpose(1, 2)
        scales[i:i + n] = s.reshape(n, page, h, 2).transpose(1, 2)
    return codes, scales


def _tables(g, lens, page, extra=3):
    """Block tables over a pool in random page order: (table, pages in the pool, ids that nobody holds)."""
    need = [_pages(n, page) for n in lens]
    pool = sum(need) + extra
    perm = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((len(lens), max(max(need), 1)), dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = perm[at:at + n]
        at += n
    return table, pool, perm[at:].contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, page = case["op"], case["page"]
    st = {"case": case}
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    if op == "plan":
        old, new = _requests(case)
        after = [a + b for a, b in zip(old, new)]
        table, pool, _ = _tables(g, old, page, extra=0)
        wide = max(_pages(n, page) for n in after + old) + 1
        st["table"] = torch.zeros((case["n_seq"], wide), dtype=torch.int32, device="cuda")
        st["table"][:, :table.shape[1]] = table
        grow = sum(max(0, _pages(b, page) - _pages(a, page)) for a, b in zip(old, after)) + 40
        held = sum(_pages(n, page) for n in old)
        st["free"] = torch.cat([torch.randperm(grow, generator=g, device="cuda").to(torch.int32) + held,
                                torch.full((held,), -1, dtype=torch.int32, device="cuda")])
        st["free_count"], st["len"], st["new"] = i32([grow]), i32(old), i32(new)
        st["n_rows"] = _up(sum(max(0, n) for n in new) + 1, 64)
        if own:
            import quantized_kv_cache_tq_gb300 as tq
            st["plan"] = tq.PagePlan(case["n_seq"], st["n_rows"])
        return st
    if op == "rows":
        n, hkv = case["rows"], case["hkv"]
        pool = _pages(n, page) + 2
        cells = torch.randperm(pool, generator=g, device="cuda")[:_pages(n, page)]
        st["slots"] = (cells[:, None] * page + torch.arange(page, device="cuda")).reshape(-1)[:n].contiguous()
        for x, d in (("k", case["dk"]), ("v", case["dv"])):
            st[x + "_src"] = _activations(g, n, hkv, d).to(DT[case["type"]])
            st[x + "_codes"] = torch.zeros((pool, hkv, page, _width(d) // 2), dtype=torch.uint8, device="cuda")
            st[x + "_scales"] = torch.zeros((pool, hkv, page, 2), dtype=torch.float16, device="cuda")
    else:
        diff, hkv = op.startswith("diff"), case["hkv"]
        if op.endswith("prefill"):
            nq, lens = _rows(case)
            st["q_start"] = i32([sum(nq[:i]) for i in range(len(nq) + 1)])
            n_rows = sum(nq)
        else:
            lens = _lens(case)
            n_rows = len(lens)
        st["table"], pool, _ = _tables(g, lens, page)
        st["len"] = i32(lens)
        maps = 2 if diff else 1
        st["k_codes"], st["k_scales"] = _pool(g, pool, maps * hkv, page, case["dk"])
        st["v_codes"], st["v_scales"] = _pool(g, pool, hkv, page, case["dv"])
        st["q"] = _activations(g, n_rows, maps * case["hq"], case["dk"]).to(DT[case["type"]])
        st["scale"] = 1.0 / math.sqrt(case["dk"])
        if diff:
            st["lam"] = 0.2 + 0.6 * torch.rand((case["hq"],), generator=g, device="cuda")
            st["norm"] = (1 + 0.1 * torch.randn((case["dv"],), generator=g, device="cuda")) if case["norm"] else None
    if own:
        import quantized_kv_cache_tq_gb300 as tq
        for x, d in (("k", case["dk"]), ("v", case["dv"])):
            st[x] = tq.Paged4Cache.from_planes(st[x + "_codes"], st[x + "_scales"], d)
        if op != "rows":
            dt, dev = st["q"].dtype, st["q"].device
            st["out"] = torch.empty((st["q"].shape[0], case["hq"], case["dv"]), dtype=dt, device=dev)
            if op.endswith("decode"):
                st["ws"] = tq.workspace(tq.paged4_decode_workspace(st["k"], st["v"], case["hq"], case["n_seq"]))
            else:
                st["ws"] = tq.workspace(tq.paged4_prefill_workspace(
                    st["k"], st["v"], case["hq"], case["n_seq"], st["q"].shape[0],
                    max_len=st["table"].shape[1] * page))
        else:
            st["k_out"], st["v_out"] = torch.empty_like(st["k_src"]), torch.empty_like(st["v_src"])
    return st


# ---------------------------------------------------------------- the plain forms

def _plan_plain(st):
    page = st["case"]["page"]
    table, free = st["table"].clone(), st["free"].clone()
    old, new = st["len"].long(), st["new"].long()
    after = old + new
    have, need = (old + page - 1) // page, (after + page - 1) // page
    back, more = (have - need).clamp(min=0), (need - have).clamp(min=0)
    back_at, more_at = back.cumsum(0) - back, more.cumsum(0) - more
    count = st["free_count"].long()
    j = torch.arange(table.shape[1], device=table.device)[None]
    # pages given back go on the free list's end, in the order of the sequences
    given = (j >= need[:, None]) & (j < have[:, None])
    free[(count + back_at[:, None] + j - need[:, None])[given]] = table[given]
    top = count + back.sum()
    taken = (j >= have[:, None]) & (j < need[:, None])
    table[taken] = free[(top - 1 - (more_at[:, None] + j - have[:, None]))[taken]]
    rows = new.clamp(min=0)
    q_start = torch.cat([rows.new_zeros(1), rows.cumsum(0)])
    r = torch.arange(st["n_rows"], device=table.device)
    seq = (torch.searchsorted(q_start, r, right=True) - 1).clamp(max=len(old) - 1)
    pos = old[seq] + r - q_start[seq]
    live = r < q_start[-1]
    pos = torch.where(live, pos, torch.zeros_like(pos))
    slot = table[seq, pos // page].long() * page + pos % page
    minus = torch.full_like(slot, -1)
    return (table, free, (top - more.sum()).int(), after.int(), q_start.int(), torch.where(live, slot, minus),
            torch.where(live, pos, minus).int())


def _values(codes, scales, d):
    """What the stored rows stand for, in 32 bits: scale * code + offset."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)[..., :d].float()
    s = scales.float()
    return s[..., :1] * c + s[..., 1:]


def _rows_plain(st):
    case, out = st["case"], []
    page, slot = st["slots"] // case["page"], st["slots"] % case["page"]
    for x, d in (("k", case["dk"]), ("v", case["dv"])):
        c, s = _quantise(st[x + "_src"].float())
        st[x + "_codes"][page, :, slot] = _pack(c, _width(d))
        st[x + "_scales"][page, :, slot] = s
        out.append(_values(st[x + "_codes"][page, :, slot], st[x + "_scales"][page, :, slot], d)
                   .to(st[x + "_src"].dtype))
    return out


def _gathered(st, x, d):
    """[sequence, head, position, dim] values of the cells that the block tables name."""
    t = st["table"].long()
    v = _values(st[x + "_codes"][t], st[x + "_scales"][t], d)          # [n, P, H, page, d]
    return v.transpose(1, 2).flatten(2, 3)


def _weights(s, live):
    """softmax over the live positions; a row without any gets zeros."""
    s = torch.where(live, s, torch.full_like(s, -math.inf))
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    return p / p.sum(-1, keepdim=True).clamp(min=1e-30)


def _attend(q, k, v, live, scale):
    """q [n, rows, heads, d], k and v [n, KV heads, L, d]; live [n, rows, L]."""
    n, r, h, d = q.shape
    g = h // k.shape[1]
    qg = q.reshape(n, r, k.shape[1], g, d).permute(0, 2, 3, 1, 4).flatten(2, 3)         # [n, KV heads, g * rows, d]
    s = torch.matmul(qg, k.transpose(2, 3)) * scale
    p = _weights(s.unflatten(2, (g, r)), live[:, None, None]).flatten(2, 3)
    o = torch.matmul(p, v)                                                              # [n, KV heads, g * rows, dv]
    return o.unflatten(2, (g, r)).permute(0, 3, 1, 2, 4).flatten(2, 3)


def _attention_plain(st):
    case = st["case"]
    op, q = case["op"], st["q"].float()
    diff = op.startswith("diff")
    k, v = _gathered(st, "k", case["dk"]), _gathered(st, "v", case["dv"])
    pos = torch.arange(k.shape[2], device=q.device)
    length = st["len"].long()
    if op.endswith("prefill"):
        start = st["q_start"].long()
        nq = start[1:] - start[:-1]
        i = torch.arange(case["max_rows"], device=q.device)
        there = i[None] < nq[:, None]
        at = torch.where(there, start[:-1, None] + i, torch.zeros_like(i)[None])
        q = q[at]                                                                       # [n, rows, heads, d]
        last = (length - nq)[:, None] + i                                               # the position of each row
        live = (pos <= last[..., None]) & there[..., None]
    else:
        q = q[:, None]
        live = (pos < length[:, None])[:, None]
    if diff:
        o = _attend(q[:, :, 0::2], k[:, 0::2], v, live, st["scale"])
        o = o - st["lam"][:, None] * _attend(q[:, :, 1::2], k[:, 1::2], v, live, st["scale"])
        if st["norm"] is not None:
            o = o * torch.rsqrt((o * o).mean(-1, keepdim=True) + 1e-5) * st["norm"] * 0.8
    else:
        o = _attend(q, k, v, live, st["scale"])
    return (o[there] if op.endswith("prefill") else o[:, 0]).to(st["q"].dtype)


# ---------------------------------------------------------------- one pass

def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        return _plan_plain(st) if op == "plan" else _rows_plain(st) if op == "rows" else _attention_plain(st)
    import quantized_kv_cache_tq_gb300 as tq
    if op == "plan":
        p = tq.page_plan(st["len"], st["new"], case["page"], st["table"], st["free"], st["free_count"], plan=st["plan"])
        return (st["table"], st["free"], p.free_count, p.seq_len, p.q_start, p.slots, p.positions)
    if op == "rows":
        tq.paged4_set_rows(st["k"], st["v"], st["k_src"], st["v_src"], st["slots"])
        return tq.paged4_get_rows(st["k"], st["v"], st["slots"], k_out=st["k_out"], v_out=st["v_out"])
    if op == "decode":
        return tq.paged4_decode(st["k"], st["v"], st["table"], st["len"], st["q"], st["scale"], out=st["out"],
                                ws=st["ws"])
    if op == "prefill":
        return tq.paged4_prefill(st["k"], st["v"], st["table"], st["len"], st["q"], st["q_start"], st["scale"],
                                 out=st["out"], ws=st["ws"])
    after = dict(norm_weight=st["norm"], eps=1e-5, out_scale=1.0 if st["norm"] is None else 0.8, out=st["out"],
                 ws=st["ws"])
    if op == "diff_decode":
        return tq.paged4_diff_decode(st["k"], st["v"], st["table"], st["len"], st["q"], st["lam"], st["scale"], **after)
    return tq.paged4_diff_prefill(st["k"], st["v"], st["table"], st["len"], st["q"], st["q_start"], st["lam"],
                                  st["scale"], **after)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "plan":
        old, new = _requests(case)
        page, rows = case["page"], _up(sum(max(0, n) for n in new) + 1, 64)
        grow = sum(abs(_pages(a + b, page) - _pages(a, page)) for a, b in zip(old, new))
        # lengths in and out, prefix sums, moved page ids read and written, slots and positions
        held = sum(_pages(a + b, page) for a, b in zip(old, new) if b > 0) - grow
        return {"bytes": 4 * (4 * case["n_seq"] + 3) + 8 * grow + 4 * max(0, min(held, rows)) + 12 * rows, "flops": 0}
    hkv = case["hkv"]
    stored = [_width(d) // 2 + 4 for d in (case["dk"], case["dv"])]
    if op == "rows":
        size = torch.finfo(DT[case["type"]]).bits // 8
        n = case["rows"] * hkv
        return {"bytes": n * sum(2 * size * d + 2 * w for d, w in zip((case["dk"], case["dv"]), stored))
                + 16 * case["rows"], "flops": 8 * n * (case["dk"] + case["dv"])}
    maps = 2 if op.startswith("diff") else 1
    if op.endswith("prefill"):
        nq, lens = _rows(case)
        pairs = sum(n * (c - n) + n * (n + 1) // 2 for n, c in zip(nq, lens))
        cells, rows = sum(c for n, c in zip(nq, lens) if n), sum(nq)
    else:
        lens = _lens(case)
        pairs = cells = sum(lens)
        rows = len(lens)
    size = 2
    return {"bytes": cells * hkv * (maps * stored[0] + stored[1]) + rows * case["hq"] * size * (maps * case["dk"] + case["dv"])
            + 4 * sum(_pages(n, case["page"]) + 1 for n in lens),
            "flops": 2 * pairs * case["hq"] * maps * (case["dk"] + case["dv"])}


# ---------------------------------------------------------------- the definition, in 64 bits

def _exact_rows(codes, scales, ids, head, d):
    """Rows of one head in the pages `ids`, as 64-bit values."""
    b = codes[ids, head].reshape(-1, codes.shape[-1]).to(torch.int64)
    c = torch.empty((b.shape[0], 2 * b.shape[1]), dtype=torch.float64, device=b.device)
    c[:, 0::2] = (b % 16).double()
    c[:, 1::2] = (b // 16).double()
    s = scales[ids, head].reshape(-1, 2).double()
    return c[:, :d] * s[:, :1] + s[:, 1:]


def _exact_map(q, k, v, end, scale):
    """softmax(scale q k^T) v over the first end[i] keys of row i."""
    x = q @ k.T * scale
    x.masked_fill_(torch.arange(k.shape[0], device=q.device)[None] >= end[:, None], -math.inf)
    x = x.sub_(x.max(1, keepdim=True).values).exp_()
    return (x @ v) / x.sum(1, keepdim=True)


def exact(case, seed):
    op = case["op"]
    if op == "plan":
        return None                                            # whole numbers
    st = prepare(case, seed)
    if op == "rows":
        got = []
        for x in ("k", "v"):
            y = st[x + "_src"].double()
            lo = y.min(-1, keepdim=True).values
            step = ((y.max(-1, keepdim=True).values - lo) / 15).to(torch.float16).double()
            lo = lo.to(torch.float16).double()
            code = ((y - lo) / step).nan_to_num(0.0).round().clamp(0, 15)
            got.append(code * step + lo)
        return got
    diff, g = op.startswith("diff"), case["hq"] // case["hkv"]
    maps = 2 if diff else 1
    if op.endswith("prefill"):
        nq, lens = _rows(case)
    else:
        lens = _lens(case)
        nq = [1] * len(lens)
    q = st["q"].double()
    out = torch.zeros((q.shape[0], case["hq"], case["dv"]), dtype=torch.float64, device=q.device)
    at = 0
    for s, (n, length) in enumerate(zip(nq, lens)):
        if n:
            ids = st["table"][s, :_pages(length, case["page"])].long()
            end = torch.arange(length - n + 1, length + 1, device=q.device)
            for h in range(case["hkv"]):
                v = _exact_rows(st["v_codes"], st["v_scales"], ids, h, case["dv"])[:length]
                ks = [_exact_rows(st["k_codes"], st["k_scales"], ids, maps * h + m, case["dk"])[:length]
                      for m in range(maps)]
                for j in range(h * g, (h + 1) * g):
                    o = [_exact_map(q[at:at + n, maps * j + m], ks[m], v, end, st["scale"]) for m in range(maps)]
                    if diff:
                        y = o[0] - st["lam"][j].double() * o[1]
                        if st["norm"] is not None:
                            y = y / torch.sqrt((y * y).mean(1, keepdim=True) + 1e-5) * st["norm"].double() * 0.8
                        o = [y]
                    out[at:at + n, j] = o[0]
        at += n
    return out
