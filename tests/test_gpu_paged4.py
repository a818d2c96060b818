"""The paged 4-bit cache on the GPU against the plain formulas of oracle/paged4.py.

Codes, scales, plans and read-back rows are compared exactly.  Attention outputs
are held to half a step of the output type (2^-8 bfloat16, 2^-11 binary16,
relative) plus the bound that oracle.paged4.softmax_map derives from binary16
weights and fp32 sums."""
import numpy as np
import pytest

from oracle import paged4 as P

pytestmark = pytest.mark.gpu


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _rows(rng, n, h, d):
    """N(0, 1) with an offset per channel and a few channels eight times as large."""
    x = rng.standard_normal((n, h, d)) + 0.3 * rng.standard_normal((h, d))
    x[:, :, rng.permutation(d)[:max(1, d // 32)]] *= 8
    return x.astype(np.float32)


def _upload(c: P.Cache):
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    return tq.Paged4Cache.from_planes(torch.from_numpy(c.codes.copy()).cuda(), torch.from_numpy(c.scales.copy()).cuda(),
                                      c.head_dim)


def _tables(rng, lens, page, spare=2, junk=None):
    """Block tables over a pool in random page order; entries that no cell needs hold `junk`."""
    need = [-(-n // page) for n in lens]
    pool = sum(need) + spare
    perm = rng.permutation(pool)
    t = np.full((len(lens), max(need + [1]) + 1), 0x7ffffff0 if junk is None else junk, np.int32)
    at = 0
    for s, n in enumerate(need):
        t[s, :n] = perm[at:at + n]
        at += n
    return t, pool


class Batch:
    """Caches filled for sequences of `lens` cells (other cells hold NaN scales and random codes)."""

    def __init__(self, seed, lens, hkv, dk, dv, page, maps=1, scale_rows=1.0):
        import torch
        rng = np.random.default_rng(seed)
        self.rng, self.lens = rng, list(lens)
        self.table, pool = _tables(rng, lens, page)
        self.k, self.v = P.Cache(maps * hkv, dk, page, pool), P.Cache(hkv, dv, page, pool)
        for c in (self.k, self.v):
            c.codes[:] = rng.integers(0, 256, c.codes.shape, dtype=np.uint8)
            c.scales[:] = np.nan
            for s, n in enumerate(lens):
                slots = self.table[s][np.arange(n) // page].astype(np.int64) * page + np.arange(n) % page
                x = _rows(rng, n, c.n_kv_heads, c.head_dim)
                c.set_rows(x * (scale_rows if c is self.v else 1.0), slots)
        self.gk, self.gv = _upload(self.k), _upload(self.v)
        self.gt = torch.from_numpy(self.table).cuda()
        self.gl = torch.tensor(self.lens, dtype=torch.int32, device="cuda")

    def query(self, n, heads, dtype, gain=1.0):
        import torch
        q = torch.from_numpy(gain * _rows(self.rng, n, heads, self.k.head_dim)).to(getattr(torch, dtype)).cuda()
        return q


def _check(out, ref, bound, dtype):
    got = _np(out)
    assert got.shape == ref.shape and np.all(np.isfinite(got))
    half = 2.0 ** -8 if dtype == "bfloat16" else 2.0 ** -11
    tiny = 2.0 ** -25 if dtype == "float16" else 0.0
    tol = half * (np.abs(ref) + bound) + bound + tiny + 1e-30
    worst = float(np.max(np.abs(got - ref) / tol, initial=0.0))
    assert worst <= 1.0, f"{worst:.2f} times the tolerance"


# ---------------------------------------------------------------- rows

@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("dk,dv,page", [(64, 64, 16), (80, 96, 32), (128, 128, 16), (192, 128, 64), (256, 256, 128), (8, 40, 16)])
def test_set_and_get_rows(dtype, dk, dv, page):
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    rng = np.random.default_rng(dk + dv)
    n, hk, hv, pool = 77, 3, 2, 6 * 128 // page + 2
    dt = getattr(torch, dtype)
    # rows are slices of one wide buffer, as of a fused projection
    wide = torch.from_numpy(_rows(rng, n, 1, hk * dk + hv * dv + 16)[:, 0]).to(dt).cuda()
    xk = wide[:, 8:8 + hk * dk].unflatten(1, (hk, dk))
    xv = wide[:, 8 + hk * dk:8 + hk * dk + hv * dv].unflatten(1, (hv, dv))
    xk[3], xv[4] = 2.5, 0.0                                  # constant rows
    slots = rng.permutation(pool * page)[:n].astype(np.int64)
    slots[5], slots[9] = -1, -1
    kc, vc = P.Cache(hk, dk, page, pool), P.Cache(hv, dv, page, pool)
    kc.set_rows(xk.float().cpu().numpy(), slots)
    vc.set_rows(xv.float().cpu().numpy(), slots)
    gk, gv = tq.Paged4Cache(hk, dk, page, pool), tq.Paged4Cache(hv, dv, page, pool)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    gs = torch.from_numpy(slots).cuda()
    tq.paged4_set_rows(gk, gv, xk, xv, gs, dev_status=st)
    for g, c in ((gk, kc), (gv, vc)):
        assert np.array_equal(g.codes.cpu().numpy(), c.codes)
        assert np.array_equal(g.scales.cpu().numpy().view(np.int16), c.scales.view(np.int16))
    assert int(st) == 0
    # back: fp32 scale * code + offset, rounded once; skipped rows keep what they had
    ko = torch.full((n, hk, dk), 7.0, dtype=dt, device="cuda")
    vo = torch.full((n, hv, dv), 7.0, dtype=dt, device="cuda")
    tq.paged4_get_rows(gk, gv, gs, k_out=ko, v_out=vo, dev_status=st)
    for o, c, d in ((ko, kc, dk), (vo, vc, dv)):
        ref = np.full(o.shape, 7.0)
        live = slots >= 0
        page_, at = slots[live] // page, slots[live] % page
        ref[live] = P.values(P.unpack(c.codes[page_, :, at], d), c.scales[page_, :, at, 0], c.scales[page_, :, at, 1])
        assert torch.equal(o.cpu(), torch.from_numpy(ref).float().to(dt))
    assert int(st) == 0


def test_rows_out_of_range_and_special_values():
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    x = torch.randn((4, 1, 64), device="cuda")
    x[0, 0, 3], x[1, 0, 0], x[1, 0, 1], x[2] = float("nan"), float("inf"), float("-inf"), 1e30
    slots = torch.tensor([1, 2, 3, 16 * 4], device="cuda")
    g = tq.Paged4Cache(1, 64, 16, 4)
    g2 = tq.Paged4Cache(1, 64, 16, 4)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tq.paged4_set_rows(g, g2, x, x, slots, dev_status=st)
    c = P.Cache(1, 64, 16, 4)
    c.set_rows(x.cpu().numpy(), [1, 2, 3, -1])
    assert np.array_equal(g.codes.cpu().numpy(), c.codes) and torch.equal(g2.codes, g.codes)
    assert np.array_equal(g.scales.cpu().numpy(), c.scales) and np.all(np.isfinite(c.scales))
    assert int(st) == tq._lib.TQ_ERR_DEVICE_CHECK
    out, _ = tq.paged4_get_rows(g, g2, torch.tensor([-2, 1 << 40], device="cuda"), dtype=torch.float32)
    assert not out.any()


def test_rows_past_32_bit_offsets():
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    n_pages = 70000                                           # 70000 x 8 x 128 x 64 B = 4.6 GB of codes
    g = tq.Paged4Cache(8, 128, 128, n_pages)
    v = tq.Paged4Cache(8, 128, 128, n_pages)
    assert g.codes.numel() > 1 << 32
    rng = np.random.default_rng(3)
    x = torch.from_numpy(_rows(rng, 40, 8, 128)).half().cuda()
    pages = torch.tensor([n_pages - 1], device="cuda")
    slots = pages * 128 + torch.arange(40, device="cuda")
    tq.paged4_set_rows(g, v, x, x, slots)
    got, _ = tq.paged4_get_rows(g, v, slots, dtype=torch.float32)
    c, s, m = P.quantise(x.float().cpu().numpy())
    assert np.array_equal(got.cpu().numpy(), P.values(c, s, m).astype(np.float32))
    q = torch.from_numpy(_rows(rng, 1, 16, 128)).half().cuda()
    out = tq.paged4_decode(g, v, pages[:, None].int(), torch.tensor([40], dtype=torch.int32, device="cuda"), q)
    small = P.Cache(8, 128, 128, 1)
    small.set_rows(x.float().cpu().numpy(), range(40))
    ref, b = P.attention(small, small, [[0]], [40], _np(q), [0, 1], 16, 128 ** -0.5)
    _check(out, ref, b, "float16")


# ---------------------------------------------------------------- plan

def _plan_case(rng, n, page, width, max_new):
    old = [int(rng.integers(0, page * width // 2)) if rng.random() < 0.8 else 0 for _ in range(n)]
    new = []
    for o in old:
        u = rng.random()
        new.append(-o if u < 0.1 else -int(rng.integers(0, o + 1)) if u < 0.2 else 0 if u < 0.3
                   else int(rng.integers(0, min(max_new, page * width - o) + 1)))
    need = [-(-o // page) for o in old]
    perm = rng.permutation(sum(need) + n * width + 8).astype(np.int32)
    table = np.full((n, width), -7, np.int32)
    at = 0
    for s, k in enumerate(need):
        table[s, :k] = perm[at:at + k]
        at += k
    rows = sum(max(0, x) for x in new)
    free = np.concatenate([perm[at:], np.full(sum(need), -9, np.int32)])
    return np.array(old, np.int32), np.array(new, np.int32), table, free, len(perm) - at, rows


def _run_plan(tq, torch, old, new, page, table, free, count, n_rows, in_place=False):
    g = lambda x: torch.from_numpy(np.array(x, np.int32).copy()).cuda()  # noqa: E731
    go, gn, gt, gf, gc = g(old), g(new), g(table), g(free), g([count])
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    p = tq.page_plan(go, gn, page, gt, gf, gc, n_rows=n_rows, in_place=in_place, dev_status=st)
    return (gt, gf, gc if in_place else p.free_count, go if in_place else p.seq_len, p.q_start, p.page_start, p.slots,
            p.positions), int(st)


@pytest.mark.parametrize("n,page,width,max_new,extra", [
    (1, 16, 4, 1, 0), (7, 16, 6, 1, 1), (33, 32, 9, 200, 0), (300, 16, 20, 40, 5), (1500, 64, 5, 300, 64),
    (2100, 16, 6, 1, 3), (5, 1, 30, 20, 2), (64, 128, 3, 1, 0)])
@pytest.mark.parametrize("in_place", [False, True])
def test_page_plan(n, page, width, max_new, extra, in_place):
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    case = _plan_case(np.random.default_rng(n + page), n, page, width, max_new)
    old, new, table, free, count, rows = case
    ref = P.page_plan(old, new, page, table, free, count, rows + extra)
    assert ref[0]
    got, st = _run_plan(tq, torch, old, new, page, table, free, count, rows + extra, in_place)
    assert st == 0
    for name, a, b in zip(("table", "free", "count", "len", "q_start", "page_start", "slots", "positions"), got, ref[1:]):
        assert np.array_equal(a.cpu().numpy().reshape(-1), np.asarray(b).reshape(-1)), name


@pytest.mark.parametrize("why", ["pages", "rows", "table", "negative", "below", "capacity", "count"])
def test_page_plan_that_cannot_be_carried_out_changes_nothing(why):
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    old, new = [20, 40, 0], [13, -40, 30]
    table, free, count, rows = [[0, 1, 9], [2, 3, 4], [9, 9, 9]], [5, 6, 7, 0, 0, 0], 3, 50
    if why == "pages":
        new, free, count = [13, 0, 30], [5, 6, 0, 0, 0, 0], 2
    if why == "rows":
        rows = 42
    if why == "table":
        new = [13, -40, 49]
    if why == "negative":
        old = [20, -1, 0]
    if why == "below":
        new = [-21, 0, 1]
    if why == "capacity":
        free = [5, 6, 7, 0, 0]
    if why == "count":
        count = -1
    ref = P.page_plan(old, new, 16, table, free, count, rows)
    assert not ref[0]
    for in_place in (False, True):
        got, st = _run_plan(tq, torch, old, new, 16, table, free, count, rows, in_place)
        assert st == tq._lib.TQ_ERR_DEVICE_CHECK
        for a, b in zip(got, ref[1:]):
            assert np.array_equal(a.cpu().numpy().reshape(-1), np.asarray(b).reshape(-1))


def test_page_plan_without_sequences_or_rows():
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    got, st = _run_plan(tq, torch, np.zeros(0), np.zeros(0), 16, np.zeros((0, 3)), [4, 5], 2, 5)
    assert st == 0 and int(got[2]) == 2 and got[6].tolist() == [-1] * 5
    got, st = _run_plan(tq, torch, [16], [-16], 16, [[3]], [4, 0], 1, 0)
    assert st == 0 and got[1].tolist() == [4, 3] and got[3].tolist() == [0]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n", [1024, 1025, 1500, 2100])
def test_page_plan_of_many_sequences_that_only_shrink(n, in_place):
    # no row to fill (n_rows 0), on both sides of what one chunk of sequences holds
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    rng = np.random.default_rng(n)
    old, new, table, free, count, _ = _plan_case(rng, n, 16, 5, 1)
    new = np.array([-int(rng.integers(0, o + 1)) if rng.random() < 0.7 else 0 for o in old], np.int32)
    ref = P.page_plan(old, new, 16, table, free, count, 0)
    assert ref[0] and ref[3] > count
    got, st = _run_plan(tq, torch, old, new, 16, table, free, count, 0, in_place)
    assert st == 0
    for name, a, b in zip(("table", "free", "count", "len", "q_start", "page_start", "slots", "positions"), got, ref[1:]):
        assert np.array_equal(a.cpu().numpy().reshape(-1), np.asarray(b).reshape(-1)), name


# ---------------------------------------------------------------- decode

@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (80, 80), (128, 128), (192, 128), (256, 256), (40, 8), (200, 256)])
@pytest.mark.parametrize("hkv,group,page", [(1, 1, 16), (2, 4, 32), (3, 8, 16), (2, 11, 128)])
def test_decode(dtype, dk, dv, hkv, group, page):
    import quantized_kv_cache_tq_gb300 as tq
    b = Batch(dk + group, [1, 0, 17, 63, 64, 65, 130, 700], hkv, dk, dv, page)
    q = b.query(8, hkv * group, dtype)
    out = tq.paged4_decode(b.gk, b.gv, b.gt, b.gl, q)
    ref, bound = P.attention(b.k, b.v, b.table, b.lens, _np(q), range(9), hkv * group, dk ** -0.5)
    ref[1], bound[1] = 0.0, 0.0
    _check(out, ref, bound, dtype)


@pytest.mark.parametrize("n_seq,length", [(1, 5000), (1, 1), (400, 40), (5, 2048), (1000, 1)])
def test_decode_splits(n_seq, length):
    # one sequence over all CTAs, many per CTA, more sequences than threads of a CTA
    import quantized_kv_cache_tq_gb300 as tq
    rng = np.random.default_rng(length)
    lens = [length] + [int(rng.integers(0, length + 1)) for _ in range(n_seq - 1)]
    b = Batch(7, lens, 2, 64, 64, 16)
    q = b.query(n_seq, 4, "float16")
    out = tq.paged4_decode(b.gk, b.gv, b.gt, b.gl, q, 0.2)
    ref, bound = P.attention(b.k, b.v, b.table, b.lens, _np(q), range(n_seq + 1), 4, 0.2)
    ref[np.array(lens) == 0] = 0.0
    _check(out, ref, bound, "float16")


@pytest.mark.parametrize("v_gain", [1e-4, 1.0, 500.0])
@pytest.mark.parametrize("q_gain,scale", [(1.0, 1.0), (100.0, 0.01), (1e-4, 300.0), (3.0, -0.3)])
def test_decode_ranges(v_gain, q_gain, scale):
    # peaked softmax, tiny and large values and queries, a negative scale
    import quantized_kv_cache_tq_gb300 as tq
    b = Batch(11, [300, 37], 2, 128, 128, 16, scale_rows=v_gain)
    for dtype in ("float16", "bfloat16"):
        q = b.query(2, 8, dtype, q_gain)
        out = tq.paged4_decode(b.gk, b.gv, b.gt, b.gl, q, scale)
        ref, bound = P.attention(b.k, b.v, b.table, b.lens, _np(q), [0, 1, 2], 8, scale)
        _check(out, ref, bound, dtype)


def test_decode_scales_far_apart():
    # value rows whose scales span 2^28: the heaviest key has the smallest one, and the other way round
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    b = Batch(13, [200, 200], 1, 64, 64, 16)
    for s in range(2):
        for t in range(200):
            page, at = b.table[s][t // 16], t % 16
            e = -14 - 10 * (t == 150) if s == 0 else (10 if t == 150 else -10)
            b.v.scales[page, 0, at] = (2.0 ** e, 2.0 ** e * 3)
            b.k.scales[page, 0, at, 1] = 5.0 if t == 150 else -1.0
            b.k.scales[page, 0, at, 0] = 0.01
    gk, gv = _upload(b.k), _upload(b.v)
    q = torch.full((2, 2, 64), 0.25, dtype=torch.float16, device="cuda")
    q[1, 1] = -0.25
    out = tq.paged4_decode(gk, gv, b.gt, b.gl, q, 0.2)
    ref, _ = P.attention(b.k, b.v, b.table, b.lens, _np(q), [0, 1, 2], 2, 0.2)
    # relative 2^-11 of weights and of the output (subnormal binary16 outputs: steps of 2^-24)
    assert np.all(np.abs(_np(out) - ref) <= 2.0 ** -9 * np.abs(ref) + 2.0 ** -25)


def test_decode_strided_queries_and_given_out():
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    b = Batch(17, [50, 90], 2, 128, 128, 16)
    wide = torch.randn((2, 3, 8 * 128 + 64), device="cuda").bfloat16()
    q = wide[:, 1, 32:32 + 8 * 128].unflatten(1, (8, 128))
    assert not q.is_contiguous()
    out = torch.full((2, 8, 128), 9.0, device="cuda", dtype=torch.bfloat16)
    ws = tq.workspace(tq.paged4_decode_workspace(b.gk, b.gv, 8, 2))
    assert tq.paged4_decode(b.gk, b.gv, b.gt, b.gl, q, 0.1, out=out, ws=ws) is out
    ref, bound = P.attention(b.k, b.v, b.table, b.lens, _np(q), [0, 1, 2], 8, 0.1)
    _check(out, ref, bound, "bfloat16")
    assert tq._lib.tq_workspace_status(ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream) == 0


def test_one_row_has_any_stride():
    # the distance to a second row that is not there
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    b = Batch(89, [130], 2, 128, 128, 16)
    q = b.query(1, 8, "float16")
    odd = torch.zeros(4096, device="cuda", dtype=q.dtype).as_strided((1, 8, 128), (1027, 128, 1)).copy_(q)
    assert torch.equal(tq.paged4_decode(b.gk, b.gv, b.gt, b.gl, odd), tq.paged4_decode(b.gk, b.gv, b.gt, b.gl, q))
    slots = torch.tensor([3], device="cuda")
    x = q[:, :2]
    odd = odd[:, :2]
    c = [tq.Paged4Cache(2, 128, 16, 1) for _ in range(4)]
    tq.paged4_set_rows(c[0], c[1], odd, odd, slots)
    tq.paged4_set_rows(c[2], c[3], x.contiguous(), x.contiguous(), slots)
    assert torch.equal(c[0].codes, c[2].codes) and torch.equal(c[1].scales, c[3].scales) and bool(c[0].codes.any())


def test_decode_bad_pages_and_lengths_are_reported():
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    b = Batch(19, [100, 40, 30], 2, 128, 128, 16)
    b.table[0, 2], b.table[1, 0] = -5, b.k.n_pages
    ws = tq.workspace(tq.paged4_decode_workspace(b.gk, b.gv, 4, 3))
    status = lambda: tq._lib.tq_workspace_status(ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)  # noqa: E731
    q = b.query(3, 4, "float16")
    out = tq.paged4_decode(b.gk, b.gv, torch.from_numpy(b.table).cuda(), b.gl, q, 0.1, ws=ws)
    ref, bound = P.attention(b.k, b.v, b.table, b.lens, _np(q), range(4), 4, 0.1)
    _check(out, ref, bound, "float16")
    assert status() == tq._lib.TQ_ERR_DEVICE_CHECK and status() == 0
    # a length beyond the table is cut to it, one below 0 to 0
    wide = b.table.shape[1] * 16
    lens = torch.tensor([100, -3, wide + 1], dtype=torch.int32, device="cuda")
    table = torch.from_numpy(np.where((b.table < 0) | (b.table >= b.k.n_pages), 0, b.table)).cuda()
    out = tq.paged4_decode(b.gk, b.gv, table, lens, q, 0.1, ws=ws)
    assert status() == tq._lib.TQ_ERR_DEVICE_CHECK
    assert not out[1].any()


def test_decode_graph_follows_lengths_and_shares_a_workspace():
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    b = Batch(23, [500, 300, 0, 64], 2, 128, 128, 16)
    d = Batch(24, [90, 1000], 3, 64, 128, 32, maps=2)
    q, dq = b.query(4, 8, "bfloat16"), d.query(2, 12, "float16")
    lam = torch.full((6,), 0.35, device="cuda")
    ws = tq.workspace(max(tq.paged4_decode_workspace(b.gk, b.gv, 8, 4), tq.paged4_decode_workspace(d.gk, d.gv, 6, 2)))
    out, dout = torch.zeros((4, 8, 128), device="cuda").bfloat16(), torch.zeros((2, 6, 128), device="cuda").half()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        tq.paged4_decode(b.gk, b.gv, b.gt, b.gl, q, 0.1, out=out, ws=ws)
        tq.paged4_diff_decode(d.gk, d.gv, d.gt, d.gl, dq, lam, 0.1, out=dout, ws=ws)
        side.synchronize()
        g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(g1, stream=side):
            tq.paged4_decode(b.gk, b.gv, b.gt, b.gl, q, 0.1, out=out, ws=ws)
        with torch.cuda.graph(g2, stream=side):
            tq.paged4_diff_decode(d.gk, d.gv, d.gt, d.gl, dq, lam, 0.1, out=dout, ws=ws)
        for lens in ([500, 300, 0, 64], [1, 0, 0, 33], [17, 299, 0, 2]):
            b.gl.copy_(torch.tensor(lens, dtype=torch.int32))
            out.fill_(5.0)
            for g in (g1, g2, g1, g2):
                g.replay()
            side.synchronize()
            ref, bound = P.attention(b.k, b.v, b.table, lens, _np(q), range(5), 8, 0.1)
            ref[np.array(lens) == 0] = 0.0
            _check(out, ref, bound, "bfloat16")
            ref, bound = P.attention(d.k, d.v, d.table, d.lens, _np(dq), range(3), 6, 0.1, lam=[0.35] * 6)
            _check(dout, ref, bound, "float16")


def test_a_workspace_is_zero_in_its_head_only():
    # NaN everywhere else before the first use; all four calls, in both ways of cutting a prompt's work
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    b = Batch(101, [1500, 300, 0, 64], 2, 128, 128, 16)
    d = Batch(103, [1500, 300, 0, 64], 2, 64, 128, 16, maps=2)
    gs = torch.tensor([0, 140, 150, 150, 170], dtype=torch.int32, device="cuda")
    q, dq, lam = b.query(170, 8, "float16"), d.query(170, 8, "float16"), torch.full((4,), 0.3, device="cuda")

    def calls(ws):
        for max_len in (1500, 1 << 18):
            yield tq.paged4_prefill(b.gk, b.gv, b.gt, b.gl, q, gs, max_len=max_len, ws=ws())
            yield tq.paged4_diff_prefill(d.gk, d.gv, d.gt, d.gl, dq, gs, lam, max_len=max_len, ws=ws())
        yield tq.paged4_decode(b.gk, b.gv, b.gt, b.gl, q[:4], ws=ws())
        yield tq.paged4_diff_decode(d.gk, d.gv, d.gt, d.gl, dq[:4], lam, ws=ws())

    def dirty():
        ws = torch.full((128 << 20,), 0xff, dtype=torch.uint8, device="cuda")
        ws[:tq._lib.PAGED4_WORKSPACE_HEAD] = 0
        return ws
    for got, want in zip(calls(dirty), calls(lambda: tq.workspace(128 << 20))):
        assert bool(torch.isfinite(got).all()) and torch.equal(got, want)


@pytest.mark.parametrize("maps", [1, 2])
def test_the_largest_steps_workspace_serves_smaller_steps(maps):
    # sized once for the most rows; steps of fewer rows take other ways of cutting the work, with other room for partials
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    lens = [1100, 900, 640, 700]
    b = Batch(107, lens, 8, 64, 128 if maps == 2 else 64, 16, maps=maps)
    heads, lam = 32, torch.full((32,), 0.3, device="cuda")
    ws = tq.workspace(tq.paged4_prefill_workspace(b.gk, b.gv, heads, 4, 2048 // maps, 4096))
    for nq, max_len in (([600 // maps, 700 // maps, 640 // maps, 108 // maps], 1100), ([700, 0, 0, 0], 4096),
                        ([512, 0, 0, 0], 4096), ([128, 5, 1, 60], 4096), ([64, 0, 0, 0], 1100), ([9, 1, 1, 1], 0),
                        ([1, 0, 1, 1], 1100)):
        start = np.cumsum([0] + nq)
        q = b.query(int(start[-1]), maps * heads, "bfloat16")
        gs = torch.tensor(start, dtype=torch.int32, device="cuda")
        if maps == 2:
            out = tq.paged4_diff_prefill(b.gk, b.gv, b.gt, b.gl, q, gs, lam, max_len=max_len or None, ws=ws)
        else:
            out = tq.paged4_prefill(b.gk, b.gv, b.gt, b.gl, q, gs, max_len=max_len or None, ws=ws)
        pick = np.sort(b.rng.permutation(int(start[-1]))[:40])
        for s in range(4):                                         # some rows of each sequence, one by one
            for r in pick[(pick >= start[s]) & (pick < start[s + 1])]:
                n = lens[s] - int(start[s + 1] - 1 - r)
                ref, bound = P.attention(b.k, b.v, b.table[s:s + 1], [n], _np(q[r:r + 1]), [0, 1], heads, 64 ** -0.5,
                                         lam=[0.3] * heads if maps == 2 else None)
                _check(out[r:r + 1], ref, bound, "bfloat16")


def test_decode_repeats_bit_for_bit():
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    b = Batch(29, [3000, 10, 777], 2, 128, 128, 16)
    q = b.query(3, 8, "bfloat16")
    outs = [tq.paged4_decode(b.gk, b.gv, b.gt, b.gl, q) for _ in range(5)]
    assert all(torch.equal(o, outs[0]) for o in outs)


@pytest.mark.parametrize("gain", [0.5, 1.0])
def test_decode_error_in_binary16_is_the_outputs_own(gain):
    # the weights' second parts and centred codes leave errors of some 2^-20, against 2^-12 of rounding the output:
    # together at most 3% above the error of the exact result rounded (rms over 4 x 8 x 128 values)
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    b = Batch(97, [3000], 1, 128, 128, 16)
    d = Batch(98, [3000], 1, 128, 128, 16, maps=2)
    got, exact = [], []
    for _ in range(4):
        q = b.query(1, 8, "float16", gain)
        got.append(_np(tq.paged4_decode(b.gk, b.gv, b.gt, b.gl, q)))
        exact.append(P.attention(b.k, b.v, b.table, b.lens, _np(q), range(2), 8, 128 ** -0.5)[0])
        q = d.query(1, 16, "float16", gain)
        got.append(_np(tq.paged4_diff_decode(d.gk, d.gv, d.gt, d.gl, q, torch.zeros(8, device="cuda"))))
        exact.append(P.attention(d.k, d.v, d.table, d.lens, _np(q), range(2), 8, 128 ** -0.5, lam=[0.0] * 8)[0])
    got, exact = np.array(got), np.array(exact)
    rms = lambda x: float(np.sqrt(np.mean(x * x)))  # noqa: E731
    assert rms(got - exact) <= 1.03 * rms(exact.astype(np.float16) - exact)


# ---------------------------------------------------------------- prefill

PRE = [  # dk, dv, kv heads, group, page, query rows, lens
    (128, 128, 2, 4, 16, [40, 0, 3, 64], [40, 90, 200, 333]),
    (128, 128, 1, 1, 32, [300, 129], [300, 700]),
    (128, 128, 2, 7, 16, [130, 1], [1000, 1]),
    (64, 64, 2, 4, 64, [65, 128, 1], [65, 500, 1025]),
    (80, 80, 3, 3, 16, [50], [77]),
    (64, 64, 1, 16, 16, [33], [64]),
    (192, 128, 2, 2, 16, [31, 2], [100, 300]),
    (256, 256, 1, 2, 32, [70], [130]),
    (128, 128, 8, 4, 16, [5, 5, 5], [600, 30, 5]),
    (128, 128, 1, 8, 16, [513], [2000]),
    (64, 64, 2, 1, 32, [1, 200, 0, 0, 17, 300, 129, 128, 5], [1, 900, 10, 0, 17, 300, 200, 1025, 2]),
]


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("causal,max_len", [(True, None), (False, None), (True, 1 << 20)])
@pytest.mark.parametrize("dk,dv,hkv,group,page,nq,lens", PRE)
def test_prefill(dk, dv, hkv, group, page, nq, lens, causal, max_len, dtype):
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    b = Batch(31 + dk, lens, hkv, dk, dv, page)
    start = np.cumsum([0] + nq)
    rows = int(start[-1]) + 5                                  # rows behind the last sequence stay as they were
    q = b.query(rows, hkv * group, dtype)
    q[start[-1]:] = float("nan")
    out = torch.full((rows, hkv * group, dv), 3.0, device="cuda", dtype=q.dtype)
    gs = torch.tensor(start, dtype=torch.int32, device="cuda")
    # (a long max_len has the work cut as one line over the SMs, a short one as CTAs per row tile)
    tq.paged4_prefill(b.gk, b.gv, b.gt, b.gl, q, gs, causal=causal, max_len=max_len, out=out)
    ref, bound = P.attention(b.k, b.v, b.table, lens, _np(q), start, hkv * group, dk ** -0.5, causal)
    ref[start[-1]:], bound[start[-1]:] = 3.0, 0.0
    _check(out, ref, bound, dtype)


@pytest.mark.parametrize("max_rows,max_len", [(0, None), (4, 1500), (1, 64), (5000, 1 << 20)])
def test_prefill_hints_only_choose_the_kernel(max_rows, max_len):
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    nq, lens = [3, 200, 0, 1], [1500, 200, 40, 64]
    b = Batch(37, lens, 2, 128, 128, 16)
    start = np.cumsum([0] + nq)
    q = b.query(int(start[-1]), 8, "float16")
    gs = torch.tensor(start, dtype=torch.int32, device="cuda")
    out = tq.paged4_prefill(b.gk, b.gv, b.gt, b.gl, q, gs, max_rows=max_rows, max_len=max_len)
    ref, bound = P.attention(b.k, b.v, b.table, lens, _np(q), start, 8, 128 ** -0.5)
    _check(out, ref, bound, "float16")


def test_prefill_rows_that_see_nothing_and_bad_row_ranges():
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    # more rows than cells: the first rows see nothing; no cells: zeros; rows outside q: none
    nq, lens = [50, 20, 40], [30, 0, 40]
    b = Batch(41, lens, 2, 128, 128, 16)
    start = np.cumsum([0] + nq)
    q = b.query(110, 4, "float16")
    ws = tq.workspace(tq.paged4_prefill_workspace(b.gk, b.gv, 4, 3, 110, 64))
    stream = torch.cuda.current_stream().cuda_stream
    gs = torch.tensor(start, dtype=torch.int32, device="cuda")
    for max_rows in (0, 1):
        out = tq.paged4_prefill(b.gk, b.gv, b.gt, b.gl, q, gs, max_rows=max_rows, max_len=64, ws=ws)
        ref, bound = P.attention(b.k, b.v, b.table, lens, _np(q), start, 4, 128 ** -0.5)
        ref = np.nan_to_num(ref)
        assert not ref[:20].any() and not ref[50:70].any()
        _check(out, ref, bound, "float16")
        assert tq._lib.tq_workspace_status(ws.data_ptr(), ws.numel(), stream) == 0
        bad = torch.tensor([0, 50, 111, 110], dtype=torch.int32, device="cuda")
        o2 = torch.full_like(out, 8.0)
        tq.paged4_prefill(b.gk, b.gv, b.gt, b.gl, q, bad, max_rows=max_rows, max_len=64, out=o2, ws=ws)
        assert torch.equal(o2[:50], out[:50]) and bool((o2[50:] == 8.0).all())
        assert tq._lib.tq_workspace_status(ws.data_ptr(), ws.numel(), stream) == tq._lib.TQ_ERR_DEVICE_CHECK


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("causal,max_len", [(True, 1500), (True, 1 << 20), (False, 1500)])
@pytest.mark.parametrize("dk,dv,maps", [(128, 128, 1), (64, 64, 1), (64, 128, 2), (128, 128, 2)])
def test_prefill_error_is_that_of_its_roundings(dk, dv, maps, causal, max_len, dtype):
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    n, rows, heads = 1500, 150, 2
    b = Batch(127 + dk, [n], 1, dk, dv, 16, maps=maps)
    gs = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    q = b.query(rows, maps * heads, dtype)
    args = (b.gk, b.gv, b.gt, b.gl, q, gs)
    if maps == 2:
        lam = torch.tensor([0.25, 0.75], device="cuda")
        out = tq.paged4_diff_prefill(*args, lam, causal=causal, max_len=max_len)
    else:
        out = tq.paged4_prefill(*args, causal=causal, max_len=max_len)
    exact, limit = P.rms_limit(b.k, b.v, b.table[0], n, _np(q), heads, dk ** -0.5, dtype, causal,
                               lam=[0.25, 0.75] if maps == 2 else None)
    err = _np(out) - exact
    assert float(np.sqrt(np.mean(err * err))) <= limit


@pytest.mark.parametrize("max_len", [9000, 1 << 20])
def test_prefill_long_context_few_tiles(max_len):
    # one tile of rows over a long context: its keys are shared by several CTAs
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    b = Batch(43, [9000], 1, 128, 128, 64)
    q = b.query(100, 2, "bfloat16")
    gs = torch.tensor([0, 100], dtype=torch.int32, device="cuda")
    out = tq.paged4_prefill(b.gk, b.gv, b.gt, b.gl, q, gs, max_len=max_len)
    ref, bound = P.attention(b.k, b.v, b.table, [9000], _np(q), [0, 100], 2, 128 ** -0.5)
    _check(out, ref, bound, "bfloat16")
    again = tq.paged4_prefill(b.gk, b.gv, b.gt, b.gl, q, gs, max_len=max_len)
    assert torch.equal(out, again)


def test_prefill_bad_pages_are_reported():
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    lens = [400]
    b = Batch(47, lens, 2, 128, 128, 16)
    b.table[0, 3], b.table[0, 20] = -1, b.k.n_pages + 7
    q = b.query(150, 4, "float16")
    gs = torch.tensor([0, 150], dtype=torch.int32, device="cuda")
    ws = tq.workspace(tq.paged4_prefill_workspace(b.gk, b.gv, 4, 1, 150, 1 << 16))
    out = tq.paged4_prefill(b.gk, b.gv, torch.from_numpy(b.table).cuda(), b.gl, q, gs, max_len=1 << 16, ws=ws)
    ref, bound = P.attention(b.k, b.v, b.table, lens, _np(q), [0, 150], 4, 128 ** -0.5)
    _check(out, ref, bound, "float16")
    assert (tq._lib.tq_workspace_status(ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
            == tq._lib.TQ_ERR_DEVICE_CHECK)


@pytest.mark.parametrize("v_gain,q_gain,scale", [(1e-4, 30.0, 1.0), (500.0, 1e-4, 300.0), (1.0, 3.0, -0.3)])
def test_prefill_ranges(v_gain, q_gain, scale):
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    b = Batch(53, [300], 2, 128, 128, 16, scale_rows=v_gain)
    gs = torch.tensor([0, 140], dtype=torch.int32, device="cuda")
    for dtype in ("float16", "bfloat16"):
        q = b.query(140, 4, dtype, q_gain)
        out = tq.paged4_prefill(b.gk, b.gv, b.gt, b.gl, q, gs, scale)
        ref, bound = P.attention(b.k, b.v, b.table, [300], _np(q), [0, 140], 4, scale)
        _check(out, ref, bound, dtype)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("s,m", [(0.5, -4.0), (2.0 ** -10, 1000.0), (2.0 ** -10, 1024.0), (2.0 ** -12, -600.0),
                                 (2.0 ** -3, 65504.0), (2.0 ** -14, 500.0), (2.0 ** -24, 0.25)])
def test_scores_of_key_rows_that_are_nearly_constant(s, m, dtype):
    # offsets of up to 2^23 steps, and queries whose entries add up to 0: only the codes tell the keys apart
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    b = Batch(139, [400], 1, 64, 64, 16)
    b.k.scales[:] = np.nan
    for t in range(400):
        b.k.scales[b.table[0][t // 16], 0, t % 16] = (s, m)
    gk, gs = _upload(b.k), torch.tensor([0, 150], dtype=torch.int32, device="cuda")
    q = np.ones((150, 2, 64))
    for row in q.reshape(-1, 64):
        row[b.rng.permutation(64)[:32]] = -1
    q = torch.from_numpy(q).to(getattr(torch, dtype)).cuda()
    scale = 2 / (37 * s)                                           # scores of some +-2: sums of +-codes have 37 rms
    for max_len in (400, 1 << 20):
        out = tq.paged4_prefill(gk, b.gv, b.gt, b.gl, q, gs, scale, max_len=max_len)
        exact, limit = P.rms_limit(b.k, b.v, b.table[0], 400, _np(q), 2, scale, dtype)
        err = _np(out) - exact
        assert float(np.sqrt(np.mean(err * err))) <= limit
    one = tq.paged4_decode(gk, b.gv, b.gt, b.gl, q[-1:], scale)
    assert float(np.sqrt(np.mean((_np(one) - exact[-1:]) ** 2))) <= limit


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("max_len", [96, 1 << 20])
@pytest.mark.parametrize("where", ["future", "light", "bad page"])
def test_prefill_small_values_beside_large_ones(dtype, max_len, where):
    # one key has all the weight and small values; among its neighbours stands a row of values up to 2^35 times as large,
    # which no row sees before it (causal), or which has no weight; or rows of zeros (a page outside the cache)
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    b = Batch(109, [96], 1, 128, 128, 16)
    q = torch.full((40, 2, 128), 0.125, dtype=getattr(torch, dtype), device="cuda")
    gs = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    low, half = (-10, 2.0 ** -11) if dtype == "float16" else (-24, 2.0 ** -8)
    at = lambda t: (b.table[0][t // 16], 0, t % 16)  # noqa: E731
    for far in (0, 5, 6, 7, 8, 11, 14, 17, 21) + (() if dtype == "float16" else (24, 30, 35)):
        for t in range(96):
            b.k.scales[at(t)] = (2.0 ** -7, 8.0 if t == 50 else -8.0)
            b.v.scales[at(t)] = (2.0 ** low, 2.0 ** low)           # values 2^low (1 .. 16)
        big = 60 if where == "future" else 40
        b.v.scales[at(big)] = (2.0 ** (low + far), 2.0 ** (low + far))
        table = b.gt.clone()
        if where == "bad page":
            table[0, 2] = -1                                       # keys 32 .. 47, the large row's among them
        out = tq.paged4_prefill(_upload(b.k), _upload(b.v), table, b.gl, q, gs, 1.0, max_len=max_len)
        heavy = P.values(P.unpack(b.v.codes[at(50)], 128), b.v.scales[at(50)][0], b.v.scales[at(50)][1])
        # (rows of a zero page have the score 0, 2^-178 of the weight); the weight's, the value's and the output's rounding
        tol = (2 * 2.0 ** -11 + half) * (1 + 2.0 ** -6) * heavy
        assert np.all(np.abs(_np(out) - heavy) <= tol), (far, float(np.max(np.abs(_np(out) - heavy) / heavy)))


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("causal,max_len,maps", [(True, 300, 1), (False, 1 << 20, 1), (True, 1 << 20, 2)])
def test_prefill_value_scales_far_apart(dtype, causal, max_len, maps):
    # value rows of scales spread over 2^20 within every 32 keys, weights over e^16: all values positive, so that the
    # result carries no more than its terms' relative errors
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    n, rows, low, half = 300, 140, *((-12, 2.0 ** -11) if dtype == "float16" else (-24, 2.0 ** -8))
    b = Batch(113, [n], 1, 64, 128 if maps == 2 else 64, 16, maps=maps)
    at = lambda t: (b.table[0][t // 16], slice(None), t % 16)  # noqa: E731
    for t in range(n):
        e = low + (0 if t % 32 == 5 else 20 if t % 32 == 21 else int(b.rng.integers(0, 21)))
        b.v.scales[at(t)] = (2.0 ** e, 2.0 ** e)                   # values 2^e (1 .. 16)
        b.k.scales[at(t)] = np.stack([np.zeros(maps), b.rng.uniform(-1, 1, maps)], -1)
    q = torch.full((rows, 2 * maps, 64), 0.125, dtype=getattr(torch, dtype), device="cuda")
    gs, gk, gv = torch.tensor([0, rows], dtype=torch.int32, device="cuda"), _upload(b.k), _upload(b.v)
    if maps == 2:
        # without a second map's share the result is the first map's
        lam = torch.zeros(2, device="cuda")
        out = tq.paged4_diff_prefill(gk, gv, b.gt, b.gl, q, gs, lam, 1.0, causal=causal, max_len=max_len)
    else:
        out = tq.paged4_prefill(gk, gv, b.gt, b.gl, q, gs, 1.0, causal=causal, max_len=max_len)
    v, k = b.v.rows(b.table[0], n, 0)[0], b.k.rows(b.table[0], n, 0)[0]
    x = k @ np.full(64, 0.125)
    assert np.ptp(x) > 14
    top = np.exp2(np.floor(np.log2(v.max(-1))))
    got = _np(out)
    for i in range(rows):
        m = n - rows + i + 1 if causal else n
        p = np.exp(x[:m] - x[:m].max())
        p /= p.sum()
        ref = p @ v[:m]
        # weight, value and output, fp32 scores and sums; weights below 2^-14 of the largest term's in steps of 2^-24
        tol = ref * (2 * 2.0 ** -11 + half) * (1 + 2.0 ** -6) + ref * 2.0 ** -16 + m * 2.0 ** -24 * (p * top[:m]).max()
        assert np.all(np.abs(got[i] - ref) <= tol), (i, float(np.max(np.abs(got[i] - ref) / tol)))


@pytest.mark.parametrize("n_seq,group,hkv,max_len", [(32, 4, 2, 600), (33, 5, 8, 4096), (40, 4, 2, 600), (40, 4, 8, 4096),
                                                     (1600, 4, 1, 400), (1600, 4, 1, 16384)])
def test_prefill_many_sequences(n_seq, group, hkv, max_len):
    # up to 32 sequences a warp finds the work alone, beyond the CTA, beyond 768 in several steps; long max_len: one line
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    rng = np.random.default_rng(n_seq)
    nq = [int(x) for x in rng.integers(0, 4 if n_seq > 100 else 90, n_seq)]
    nq[-1] = 60
    lens = [n + int(rng.integers(0, 40 if n_seq > 100 else 300)) for n in nq]
    b = Batch(61, lens, hkv, 64, 64, 16)
    start = np.cumsum([0] + nq)
    q = b.query(int(start[-1]), hkv * group, "float16")
    gs = torch.tensor(start, dtype=torch.int32, device="cuda")
    out = tq.paged4_prefill(b.gk, b.gv, b.gt, b.gl, q, gs, max_len=max_len)
    ref, bound = P.attention(b.k, b.v, b.table, lens, _np(q), start, hkv * group, 64 ** -0.5)
    _check(out, ref, bound, "float16")


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("up", [4, 12, 15])
def test_scores_up_to_2_24(up, dtype):
    # keys whose scores are 2^(up + 2) and more apart, the largest 2^(up + 8.6): all weight is on the best key
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    b = Batch(137, [100], 1, 64, 64, 16)
    order = b.rng.permutation(100)
    for t in range(100):
        b.k.scales[b.table[0][t // 16], 0, t % 16] = (0.0, 0.5 * float(order[t]) - 2.0)
    q = torch.full((100, 1, 64), 8.0, dtype=getattr(torch, dtype), device="cuda")
    scale = 2.0 ** up / 64
    gk, gs = _upload(b.k), torch.tensor([0, 100], dtype=torch.int32, device="cuda")
    best = [int(np.argmax(order[:t + 1])) for t in range(100)]
    v = b.v.rows(b.table[0], 100, 0)[0][best][:, None]
    # a weight, a value and the output rounded (the other keys' weights are below e^-64)
    tol = (2 * 2.0 ** -11 + (2.0 ** -11 if dtype == "float16" else 2.0 ** -8)) * (1 + 2.0 ** -6) * np.abs(v) + 2.0 ** -20
    for max_len in (100, 1 << 20):
        out = tq.paged4_prefill(gk, b.gv, b.gt, b.gl, q, gs, scale, max_len=max_len)
        assert np.all(np.abs(_np(out) - v) <= tol)
    one = tq.paged4_decode(gk, b.gv, b.gt, b.gl, q[:1], scale)
    assert np.all(np.abs(_np(one)[0] - v[-1]) <= tol[-1])


@pytest.mark.parametrize("up", [118, -90])
def test_scaled_queries_with_the_inverse_scale(up):
    # a power of two moved from the queries to the scale changes nothing, near the ends of bfloat16's range too
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    b = Batch(59, [300, 90], 2, 128, 128, 16)
    gs = torch.tensor([0, 140, 190], dtype=torch.int32, device="cuda")
    q = b.query(190, 4, "bfloat16").clamp(-16, 16)
    q = torch.where(q.abs() < 2.0 ** -16, torch.zeros_like(q), q)
    big = q.double().mul(2.0 ** up).bfloat16()
    assert torch.equal(big.double().mul(2.0 ** -up), q.double())
    one = tq.paged4_prefill(b.gk, b.gv, b.gt, b.gl, q, gs, 0.125)
    two = tq.paged4_prefill(b.gk, b.gv, b.gt, b.gl, big, gs, 0.125 * 2.0 ** -up)
    assert torch.isfinite(one).all() and torch.equal(one, two)
    one = tq.paged4_decode(b.gk, b.gv, b.gt, b.gl, q[:2], 0.125)
    two = tq.paged4_decode(b.gk, b.gv, b.gt, b.gl, big[:2], 0.125 * 2.0 ** -up)
    assert torch.isfinite(one).all() and torch.equal(one, two)


def test_sequences_that_share_pages():
    # a common prefix: its pages stand in several block tables; pages of 1024 cells
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    for page, lens in ((16, [200, 200, 131]), (1024, [2100, 2100, 1500])):
        b = Batch(67, lens, 2, 128, 128, page)
        shared = 128 // page if page < 128 else 1
        b.table[1, :shared] = b.table[2, :shared] = b.table[0, :shared]
        gt = torch.from_numpy(b.table).cuda()
        q = b.query(3, 8, "bfloat16")
        out = tq.paged4_decode(b.gk, b.gv, gt, b.gl, q)
        ref, bound = P.attention(b.k, b.v, b.table, lens, _np(q), range(4), 8, 128 ** -0.5)
        _check(out, ref, bound, "bfloat16")
        start = [0, 33, 60, 80]
        q = b.query(80, 8, "bfloat16")
        out = tq.paged4_prefill(b.gk, b.gv, gt, b.gl, q, torch.tensor(start, dtype=torch.int32, device="cuda"))
        ref, bound = P.attention(b.k, b.v, b.table, lens, _np(q), start, 8, 128 ** -0.5)
        _check(out, ref, bound, "bfloat16")


def test_prefill_lengths_beyond_the_table_are_cut():
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    b = Batch(71, [160, 160], 2, 128, 128, 16)
    b.table = b.table[:, :10].copy()
    gs = torch.tensor([0, 40, 70], dtype=torch.int32, device="cuda")
    q = b.query(70, 4, "float16")
    gl = torch.tensor([5000, -3], dtype=torch.int32, device="cuda")
    ws = tq.workspace(tq.paged4_prefill_workspace(b.gk, b.gv, 4, 2, 70, 160))
    out = tq.paged4_prefill(b.gk, b.gv, torch.from_numpy(b.table).cuda(), gl, q, gs, ws=ws)
    ref, bound = P.attention(b.k, b.v, b.table, [160, 0], _np(q), [0, 40, 70], 4, 128 ** -0.5)
    ref[40:], bound[40:] = 0.0, 0.0
    _check(out, ref, bound, "float16")
    assert (tq._lib.tq_workspace_status(ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
            == tq._lib.TQ_ERR_DEVICE_CHECK)


def test_calls_on_two_streams_at_once():
    # each with a workspace of its own
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    b = Batch(73, [3000, 700, 90], 4, 128, 128, 16)
    q, dq = b.query(400, 8, "bfloat16"), b.query(3, 8, "bfloat16")
    gs = torch.tensor([0, 350, 380, 400], dtype=torch.int32, device="cuda")
    want = tq.paged4_prefill(b.gk, b.gv, b.gt, b.gl, q, gs), tq.paged4_decode(b.gk, b.gv, b.gt, b.gl, dq)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = [[] for _ in streams]
    wss = [tq.workspace(tq.paged4_prefill_workspace(b.gk, b.gv, 8, 3, 400, 3000)) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                if i % 2:
                    got[i].append(tq.paged4_decode(b.gk, b.gv, b.gt, b.gl, dq, ws=wss[i]))
                else:
                    got[i].append(tq.paged4_prefill(b.gk, b.gv, b.gt, b.gl, q, gs, max_len=3000, ws=wss[i]))
    torch.cuda.synchronize()
    for i in range(len(streams)):
        assert all(torch.equal(o, got[i % 2][0]) for o in got[i])
    assert torch.equal(got[1][0], want[1])
    assert all(tq._lib.tq_workspace_status(w.data_ptr(), w.numel(), 0) == 0 for w in wss)


@pytest.mark.parametrize("max_len", [700, 1 << 20])
def test_prefill_graphs_share_a_workspace_with_decode(max_len):
    # lengths and row ranges move between the replays; both forms of cutting the work
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    b = Batch(79, [600, 300], 2, 128, 128, 16)
    d = Batch(83, [400, 257], 2, 64, 128, 32, maps=2)
    q, dq, one = b.query(160, 8, "bfloat16"), d.query(160, 8, "float16"), b.query(2, 8, "bfloat16")
    lam = torch.full((4,), 0.4, device="cuda")
    gs = torch.tensor([0, 100, 160], dtype=torch.int32, device="cuda")
    ws = tq.workspace(max(tq.paged4_prefill_workspace(b.gk, b.gv, 8, 2, 160, max_len),
                          tq.paged4_prefill_workspace(d.gk, d.gv, 4, 2, 160, max_len),
                          tq.paged4_decode_workspace(b.gk, b.gv, 8, 2)))
    out, o1 = torch.zeros((160, 8, 128), device="cuda").bfloat16(), torch.zeros((2, 8, 128), device="cuda").bfloat16()
    dout = torch.zeros((160, 4, 128), device="cuda").half()
    calls = (lambda: tq.paged4_prefill(b.gk, b.gv, b.gt, b.gl, q, gs, max_len=max_len, out=out, ws=ws),
             lambda: tq.paged4_diff_prefill(d.gk, d.gv, d.gt, d.gl, dq, gs, lam, max_len=max_len, out=dout, ws=ws),
             lambda: tq.paged4_decode(b.gk, b.gv, b.gt, b.gl, one, out=o1, ws=ws))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for c in calls:
            c()
        side.synchronize()
        graphs = [torch.cuda.CUDAGraph() for _ in calls]
        for g, c in zip(graphs, calls):
            with torch.cuda.graph(g, stream=side):
                c()
        for lens, dlens, start in (([600, 300], [400, 257], [0, 100, 160]), ([90, 17], [33, 257], [0, 90, 107]),
                                   ([600, 0], [1, 100], [0, 1, 1])):
            b.gl.copy_(torch.tensor(lens, dtype=torch.int32))
            d.gl.copy_(torch.tensor(dlens, dtype=torch.int32))
            gs.copy_(torch.tensor(start, dtype=torch.int32))
            out.fill_(5.0)
            dout.fill_(5.0)
            for g in graphs + graphs[::-1]:
                g.replay()
            side.synchronize()
            n = start[-1]
            ref, bound = P.attention(b.k, b.v, b.table, lens, _np(q), start, 8, 128 ** -0.5)
            _check(out[:n], np.nan_to_num(ref[:n]), bound[:n], "bfloat16")
            ref, bound = P.attention(d.k, d.v, d.table, dlens, _np(dq), start, 4, 64 ** -0.5, lam=[0.4] * 4)
            _check(dout[:n], np.nan_to_num(ref[:n]), bound[:n], "float16")
            assert bool((out[n:] == 5.0).all()) and bool((dout[n:] == 5.0).all())
            ref, bound = P.attention(b.k, b.v, b.table, lens, _np(one), range(3), 8, 128 ** -0.5)
            ref[np.array(lens) == 0] = 0.0
            _check(o1, ref, bound, "bfloat16")
        assert tq._lib.tq_workspace_status(ws.data_ptr(), ws.numel(), side.cuda_stream) == 0


# ---------------------------------------------------------------- differential

DIFF = [(64, 64, 1, 1, 16), (64, 128, 2, 2, 32), (128, 128, 2, 4, 16), (128, 256, 1, 2, 16), (48, 96, 2, 3, 64),
        (64, 128, 1, 9, 16)]


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("dk,dv,hkv,group,page", DIFF)
def test_diff_decode(dk, dv, hkv, group, page, norm):
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    lens = [1, 0, 40, 64, 65, 900]
    b = Batch(59 + dk, lens, hkv, dk, dv, page, maps=2)
    heads = hkv * group
    lam = torch.linspace(-0.2, 0.9, heads, device="cuda")
    w = torch.linspace(0.5, 1.5, dv, device="cuda") if norm else None
    for dtype in ("float16", "bfloat16"):
        q = b.query(6, 2 * heads, dtype)
        out = tq.paged4_diff_decode(b.gk, b.gv, b.gt, b.gl, q, lam, norm_weight=w, eps=1e-4, out_scale=0.8)
        ref, bound = P.attention(b.k, b.v, b.table, lens, _np(q), range(7), heads, dk ** -0.5, lam=_np(lam),
                                 norm_weight=_np(w) if norm else None, eps=1e-4, out_scale=0.8)
        ref[1], bound[1] = 0.0, 0.0
        _check(out, ref, bound, dtype)


@pytest.mark.parametrize("norm,causal,dtype,max_len", [
    (True, True, "bfloat16", None), (False, True, "float16", 1 << 20), (True, False, "float16", 64)])
@pytest.mark.parametrize("dk,dv,hkv,group,page", DIFF)
def test_diff_prefill(dk, dv, hkv, group, page, norm, causal, dtype, max_len):
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    nq, lens = [70, 0, 5, 150], [70, 20, 300, 400]
    b = Batch(61 + dk, lens, hkv, dk, dv, page, maps=2)
    heads, start = hkv * group, np.cumsum([0] + nq)
    lam = torch.linspace(-0.2, 0.9, heads, device="cuda")
    w = torch.linspace(0.5, 1.5, dv, device="cuda") if norm else None
    rows = int(start[-1]) + 3
    q = b.query(rows, 2 * heads, dtype)
    out = torch.full((rows, heads, dv), 3.0, device="cuda", dtype=q.dtype)
    gs = torch.tensor(start, dtype=torch.int32, device="cuda")
    tq.paged4_diff_prefill(b.gk, b.gv, b.gt, b.gl, q, gs, lam, norm_weight=w, eps=1e-4, out_scale=0.8, causal=causal,
                           max_len=max_len, out=out)
    ref, bound = P.attention(b.k, b.v, b.table, lens, _np(q), start, heads, dk ** -0.5, causal, lam=_np(lam),
                             norm_weight=_np(w) if norm else None, eps=1e-4, out_scale=0.8)
    ref[start[-1]:], bound[start[-1]:] = 3.0, 0.0
    _check(out, ref, bound, dtype)


@pytest.mark.parametrize("max_rows,max_len", [(0, 64), (1, 64), (0, 1 << 20)])
def test_diff_rows_without_values_are_zeros_without_eps(max_rows, max_len):
    # rows that see no cell, sequences without cells, and value rows of zeros, normalised with eps = 0
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    nq, lens = [50, 20, 40], [30, 0, 40]
    b = Batch(131, lens, 2, 64, 128, 16, maps=2)
    page = [b.table[2][t // 16] for t in range(40)]
    for t in range(40):
        b.v.scales[page[t], :, t % 16] = 0.0                       # the third sequence's values
    gv = _upload(b.v)
    start = np.cumsum([0] + nq)
    q, lam, w = b.query(110, 8, "float16"), torch.full((4,), 0.4, device="cuda"), torch.ones(128, device="cuda")
    gs = torch.tensor(start, dtype=torch.int32, device="cuda")
    out = tq.paged4_diff_prefill(b.gk, gv, b.gt, b.gl, q, gs, lam, norm_weight=w, eps=0.0, max_rows=max_rows, max_len=max_len)
    assert not out[:20].any() and not out[50:].any() and bool(torch.isfinite(out).all())
    ref, bound = P.attention(b.k, b.v, b.table[:1], [30], _np(q[20:50]), [0, 30], 4, 64 ** -0.5, lam=[0.4] * 4,
                             norm_weight=np.ones(128))
    _check(out[20:50], ref, bound, "float16")
    one = tq.paged4_diff_decode(b.gk, gv, b.gt, b.gl, q[:3], lam, norm_weight=w, eps=0.0)
    assert not one[1:].any() and bool(torch.isfinite(one).all()) and bool(one[0].any())


# ---------------------------------------------------------------- together, as a server uses them

def test_serving_steps_in_one_captured_graph():
    """Prompts admitted, then decode steps: plan, rows, attention from one captured graph whose inputs change."""
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    rng = np.random.default_rng(67)
    n, hkv, hq, d, page, pool, width, cap = 4, 2, 8, 128, 16, 60, 12, 96
    gk, gv = tq.Paged4Cache(hkv, d, page, pool), tq.Paged4Cache(hkv, d, page, pool)
    table = torch.zeros((n, width), dtype=torch.int32, device="cuda")
    free = torch.from_numpy(rng.permutation(pool).astype(np.int32)).cuda()
    count = torch.tensor([pool], dtype=torch.int32, device="cuda")
    lens, new = (torch.zeros(n, dtype=torch.int32, device="cuda") for _ in range(2))
    plan = tq.PagePlan(n, cap)
    qkv = torch.zeros((cap, (hq + 2 * hkv) * d), device="cuda", dtype=torch.bfloat16)
    q = qkv[:, :hq * d].unflatten(1, (hq, d))
    k = qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
    v = qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
    out = torch.zeros((cap, hq, d), device="cuda", dtype=torch.bfloat16)
    ws = tq.workspace(tq.paged4_prefill_workspace(gk, gv, hq, n, cap, width * page))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step():
        tq.page_plan(lens, new, page, table, free, count, plan=plan, in_place=True, dev_status=st)
        tq.paged4_set_rows(gk, gv, k, v, plan.slots, dev_status=st)
        tq.paged4_prefill(gk, gv, table, lens, q, plan.q_start, out=out, ws=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step()                                                # no new cells: changes nothing
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            step()
        kept = [np.zeros((0, hkv, d), np.float32) for _ in range(n)], [np.zeros((0, hkv, d), np.float32) for _ in range(n)]
        for news in ([40, 7, 0, 17], [1, 1, 0, 1], [1, 1, 30, 1], [-41, 1, 1, 1], [50, 1, 1, -3], [1, 1, 1, 1]):
            x = torch.from_numpy(_rows(rng, cap, 1, (hq + 2 * hkv) * d)[:, 0]).bfloat16()
            qkv.copy_(x)
            new.copy_(torch.tensor(news, dtype=torch.int32))
            if news[0] == -41:
                news[0] = -int(kept[0][0].shape[0])
                new[0] = news[0]
            graph.replay()
            side.synchronize()
            assert int(st) == 0
            start = np.cumsum([0] + [max(0, m) for m in news])
            assert plan.q_start.tolist() == start.tolist()
            xk, xv = k.float().cpu().numpy(), v.float().cpu().numpy()
            for s, m in enumerate(news):
                for which, src in ((0, xk), (1, xv)):
                    rows = kept[which][s]
                    kept[which][s] = rows[:len(rows) + m] if m < 0 else np.concatenate([rows, src[start[s]:start[s + 1]]])
            now = [len(r) for r in kept[0]]
            assert lens.tolist() == now
            pk, pv = P.Cache(hkv, d, page, n * width), P.Cache(hkv, d, page, n * width)
            tables = np.arange(n * width).reshape(n, width)
            for s in range(n):
                slots = s * width * page + np.arange(now[s])
                pk.set_rows(kept[0][s], slots)
                pv.set_rows(kept[1][s], slots)
            ref, bound = P.attention(pk, pv, tables, now, _np(q), start, hq, d ** -0.5)
            live = int(start[-1])
            _check(out[:live], ref[:live], bound[:live], "bfloat16")
    held = sum(-(-m // page) for m in now)
    assert int(count) == pool - held
    ids = sorted(free[:pool - held].tolist() + [int(p) for s in range(n) for p in table[s, :-(-now[s] // page)]])
    assert ids == list(range(pool))                           # no page lost or held twice


def test_plan_feeds_the_turbo_cache():
    """The slots are cell ids for tq_set_rows too (a page is a run of cells of a TqCache)."""
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    table = torch.zeros((2, 4), dtype=torch.int32, device="cuda")
    free = torch.tensor([3, 1, 0, 2], dtype=torch.int32, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    plan = tq.page_plan(i32([0, 0]), i32([70, 64]), 64, table, free, i32([4]), n_rows=134)
    cache, same = tq.TqCache(4, 1, 128, 256), tq.TqCache(4, 1, 128, 256)
    cb = tq.codebook(4, [1, 2, 3, 4])
    x = torch.randn((134, 1, 128), device="cuda")
    tq.set_rows(cache, cb, x, plan.slots)
    cells = torch.cat([128 + torch.arange(64), torch.arange(6), 64 + torch.arange(64)]).cuda()
    tq.set_rows(same, cb, x, cells)
    assert torch.equal(plan.slots, cells) and torch.equal(cache.qs, same.qs) and torch.equal(cache.norms, same.norms)
