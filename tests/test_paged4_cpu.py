"""The paged 4-bit cache without a GPU: its plain formulas against hand-made
cases, and every refusal of its C ABI and of its Python calls."""
import numpy as np
import pytest

from oracle import paged4 as P


def _lib():
    from quantized_kv_cache_tq_gb300 import _lib
    return _lib


# ---------------------------------------------------------------- the formulas

def test_quantise_by_hand():
    # min -1, max 2: scale 0.2 (binary16 0.19995...), codes by nearest
    c, s, m = P.quantise(np.array([[-1.0, -0.9, -0.8, 0.0, 2.0, 1.9, 0.5, -1.0]]))
    assert m[0] == -1 and s[0] == np.float16(3 / 15)
    assert list(c[0]) == [0, 1, 1, 5, 15, 15, 8, 0] or list(c[0]) == [0, 1, 1, 5, 15, 14, 8, 0]
    x = P.values(c, s, m)[0]
    assert np.all(np.abs(x - [-1.0, -0.9, -0.8, 0.0, 2.0, 1.9, 0.5, -1.0]) <= 0.5 * float(s[0]) + 15 * 2.0 ** -14)


def test_quantise_special_rows():
    c, s, m = P.quantise(np.array([[3.0] * 8, [np.nan, 0, 0, 0, 0, 0, 0, 15.0], [np.inf, -np.inf, 0, 0, 0, 0, 0, 0]]))
    assert s[0] == 0 and m[0] == 3 and not c[0].any()
    assert s[1] == 1 and list(c[1]) == [0, 0, 0, 0, 0, 0, 0, 15]
    assert m[2] == -65504 and c[2][0] == 15 and c[2][1] == 0


def test_error_is_at_most_half_a_step():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((200, 96)).astype(np.float32)
    c, s, m = P.quantise(x)
    # half a step, the offset's rounding, and the range's rounding up to 15 steps of relative 2^-11
    tol = 0.5 * s.astype(np.float64) + 2.0 ** -11 * np.abs(m.astype(np.float64)) + 15 * 2.0 ** -11 * s.astype(np.float64)
    assert np.all(np.abs(P.values(c, s, m) - x) <= tol[:, None] + 1e-6)


def test_pack_layout():
    p = P.pack(np.arange(80, dtype=np.uint8)[None] % 16)
    assert p.shape == (1, 64) and p[0, 0] == 0x10 and p[0, 7] == 0xfe and not p[0, 40:].any()
    assert np.array_equal(P.unpack(p, 80)[0], np.arange(80) % 16)


def test_attention_by_loops():
    rng = np.random.default_rng(1)
    kc, vc = P.Cache(1, 8, 16, 3), P.Cache(1, 8, 16, 3)
    xk, xv = rng.standard_normal((20, 1, 8)), rng.standard_normal((20, 1, 8))
    slots = [2 * 16 + i for i in range(16)] + [i for i in range(4)]          # pages 2, 0
    kc.set_rows(xk, slots)
    vc.set_rows(xv, slots)
    q = rng.standard_normal((3, 2, 8))
    out, _ = P.attention(kc, vc, [[2, 0]], [20], q, [0, 3], 2, 0.5)
    k, v = P.values(*P.quantise(xk)), P.values(*P.quantise(xv))
    for i in range(3):
        for h in range(2):
            e = [np.exp(0.5 * float(q[i, h] @ k[t, 0])) for t in range(18 + i)]
            ref = sum(w * v[t, 0] for t, w in enumerate(e)) / sum(e)
            assert np.allclose(out[i, h], ref, rtol=1e-12)


def test_differential_by_two_maps():
    rng = np.random.default_rng(2)
    kc, vc = P.Cache(2, 8, 16, 1), P.Cache(1, 16, 16, 1)
    kc.set_rows(rng.standard_normal((10, 2, 8)), range(10))
    vc.set_rows(rng.standard_normal((10, 1, 16)), range(10))
    q = rng.standard_normal((1, 2, 8))
    out, _ = P.attention(kc, vc, [[0]], [10], q, [0, 1], 1, 0.3, lam=[0.4])
    one = []
    for m in range(2):
        km = P.Cache(1, 8, 16, 1)
        km.codes, km.scales = kc.codes[:, m:m + 1], kc.scales[:, m:m + 1]
        one.append(P.attention(km, vc, [[0]], [10], q[:, m:m + 1], [0, 1], 1, 0.3)[0])
    assert np.allclose(out, one[0] - 0.4 * one[1], rtol=1e-12)
    w = rng.standard_normal(16)
    normed, _ = P.attention(kc, vc, [[0]], [10], q, [0, 1], 1, 0.3, lam=[0.4], norm_weight=w, eps=1e-3, out_scale=0.5)
    assert np.allclose(normed[0, 0], 0.5 * w * out[0, 0] / np.sqrt((out[0, 0] ** 2).mean() + 1e-3), rtol=1e-12)


@pytest.mark.parametrize("dtype,bits,within", [("float16", 11, True), ("bfloat16", 11, True), ("float16", 10, False),
                                               ("float16", 9, False), ("bfloat16", 7, False)])
def test_rms_limit_holds_for_binary16_operands_and_for_no_fewer_bits(dtype, bits, within):
    # the prompt kernel's roundings in numpy, with weights and values of `bits` significant bits
    rng = np.random.default_rng(4)
    n, rows = 800, 60
    kc, vc = P.Cache(1, 64, 16, 50), P.Cache(1, 64, 16, 50)
    kc.set_rows(rng.standard_normal((n, 1, 64)), range(n))
    vc.set_rows(rng.standard_normal((n, 1, 64)) + 0.3, range(n))
    q = rng.standard_normal((rows, 2, 64))
    exact, limit = P.rms_limit(kc, vc, np.arange(50), n, q, 2, 0.125, dtype)
    assert np.allclose(exact, P.attention(kc, vc, [np.arange(50)], [n], q, [0, rows], 2, 0.125)[0], rtol=1e-12)

    def cut(x):
        m, e = np.frexp(x)
        return np.ldexp(np.rint(m * 2.0 ** bits), e - bits)
    k, v = kc.rows(np.arange(50), n, 0)[0], cut(vc.rows(np.arange(50), n, 0)[0])
    got = np.zeros_like(exact)
    for i in range(rows):
        for h in range(2):
            p = np.exp(0.125 * (k[:n - rows + i + 1] @ q[i, h]))
            got[i, h] = cut(p) @ v[:len(p)] / p.sum()
    err = P.round_to(got, dtype) - exact
    assert (np.sqrt(np.mean(err * err)) <= limit) == within


def test_plan_by_hand():
    # pages of 4: s0 5 -> 9 cells (takes one page), s1 8 -> 0 (returns two), s2 0 -> 1 (takes one)
    table = [[10, 11, 0], [12, 13, 0], [0, 0, 0]]
    ok, t, f, n, after, qs, ps, slots, pos = P.page_plan([5, 8, 0], [4, -8, 1], 4, table, [7, 8, 0, 0, 0], 2, 6)
    assert ok and list(f) == [7, 8, 12, 13, 0] and n == 2
    assert t[0].tolist() == [10, 11, 13] and t[2].tolist() == [12, 0, 0]
    assert list(after) == [9, 0, 1] and list(qs) == [0, 4, 4, 5] and list(ps) == [0, 1, 1, 2]
    assert list(slots) == [45, 46, 47, 52, 48, -1] and list(pos) == [5, 6, 7, 8, 0, -1]
    assert not P.page_plan([5], [40], 4, [[10, 11, 0]], [7], 1, 50)[0]       # beyond the table
    assert not P.page_plan([5], [4], 4, [[10, 11, 0]], [7], 0, 50)[0]        # no free page
    assert not P.page_plan([5], [4], 4, [[10, 11, 0]], [7], 1, 3)[0]         # too few rows


# ---------------------------------------------------------------- the C ABI's refusals (nothing is launched)

def _cache(L, h=2, d=128, ps=16, n=8, codes=1 << 20, scales=1 << 24):
    return L.tq_paged4(h, d, ps, n, codes, scales)


def test_plane_bytes():
    L = _lib()
    assert L.tq_paged4_plane_bytes(8, 128, 16, 10) == (8 * 16 * 10 * 64, 8 * 16 * 10 * 4)
    assert L.tq_paged4_plane_bytes(1, 80, 32, 2) == (64 * 64, 64 * 4)
    assert L.tq_paged4_plane_bytes(1, 192, 16, 1)[0] == 16 * 128
    for bad in ((0, 128, 16, 1), (1, 0, 16, 1), (1, 100, 16, 1), (1, 264, 16, 1), (1, 128, 8, 1), (1, 128, 48, 1),
                (1, 128, 2048, 1), (1, 128, 16, 0)):
        with pytest.raises(L.TQError):
            L.tq_paged4_plane_bytes(*bad)


def test_row_calls_refuse():
    L = _lib()
    k, v = _cache(L), _cache(L)

    def call(k=k, v=v, ks=1 << 25, kst=256, vs=1 << 26, vst=256, t=L.TQ_F16, slots=1 << 27, n=4, status=None):
        got = {f(k, v, ks, kst, vs, vst, t, slots, n, status, None) for f in (L.tq_paged4_set_rows, L.tq_paged4_get_rows)}
        assert len(got) == 1
        return got.pop()

    bad = L.TQ_ERR_INVALID_ARG
    for c in (_cache(L, d=100), _cache(L, ps=24), _cache(L, n=0), _cache(L, codes=(1 << 20) + 8), _cache(L, scales=0),
              _cache(L, h=0), _cache(L, ps=32), _cache(L, n=9)):
        assert call(k=c) == bad and (call(v=c) == bad)
    assert call(t=9) == bad and call(n=-1) == bad and call(kst=248) == bad and call(vst=260) == bad
    assert call(ks=(1 << 25) + 2) == bad and call(vs=0) == bad and call(slots=(1 << 27) + 4) == bad
    assert call(status=(1 << 28) + 1) == bad
    assert call(n=0) == L.TQ_OK


def test_plan_refuses():
    L = _lib()

    def call(seq_len=1 << 20, n_new=1 << 21, n=3, ps=16, table=1 << 22, width=4, free=1 << 23, cap=10, count=1 << 24,
             new_len=1 << 25, new_count=1 << 26, qs=1 << 27, pst=1 << 28, slots=1 << 29, pos=1 << 30, rows=8, st=None):
        return L.tq_page_plan(seq_len, n_new, n, ps, table, width, free, cap, count, new_len, new_count, qs, pst, slots,
                              pos, rows, st, None)

    for kw in (dict(n=-1), dict(ps=0), dict(ps=24), dict(ps=1 << 17), dict(width=0), dict(cap=-1), dict(cap=1 << 31),
               dict(rows=-1), dict(rows=1 << 31), dict(ps=65536, width=1 << 16), dict(seq_len=0), dict(n_new=2),
               dict(table=0), dict(free=0), dict(count=0), dict(new_len=0), dict(new_count=1), dict(qs=0), dict(pst=0),
               dict(slots=(1 << 29) + 4), dict(pos=0), dict(st=2)):
        assert call(**kw) == L.TQ_ERR_INVALID_ARG, kw


def _attend(L, kind, **kw):
    a = dict(k=_cache(L, h=4 if "diff" in kind else 2), v=_cache(L), table=1 << 25, width=4, lens=1 << 26,
             qs=1 << 27, n=3, q=1 << 28, t=L.TQ_BF16, rows=9, heads=4, lam=1 << 29, nw=None, eps=1e-5, osc=1.0,
             scale=0.1, out=1 << 30, ws=1 << 31, ws_bytes=1 << 40, max_rows=0, max_len=0)
    a["stride"] = 4096
    a.update(kw)
    head = (a["k"], a["v"], a["table"], a["width"], a["lens"])
    tail = (a["out"], a["ws"], a["ws_bytes"], None)
    diff = (a["lam"], a["nw"], a["eps"], a["osc"])
    if kind == "decode":
        return L.tq_paged4_decode(*head, a["n"], a["q"], a["t"], a["stride"], a["heads"], a["scale"], *tail)
    if kind == "diff_decode":
        return L.tq_paged4_diff_decode(*head, a["n"], a["q"], a["t"], a["stride"], a["heads"], *diff, a["scale"], *tail)
    more = (a["qs"], a["n"], a["q"], a["t"], a["stride"], a["rows"], a["heads"], a["max_rows"], a["max_len"])
    if kind == "prefill":
        return L.tq_paged4_prefill(*head, *more, a["scale"], 1, *tail)
    return L.tq_paged4_diff_prefill(*head, *more, *diff, a["scale"], 1, *tail)


@pytest.mark.parametrize("kind", ["decode", "prefill", "diff_decode", "diff_prefill"])
def test_attention_calls_refuse(kind):
    L = _lib()
    bad, uns, wsp = L.TQ_ERR_INVALID_ARG, L.TQ_ERR_UNSUPPORTED, L.TQ_ERR_WORKSPACE
    diff, ragged = "diff" in kind, "prefill" in kind
    call = lambda **kw: _attend(L, kind, **kw)  # noqa: E731
    kh = 4 if diff else 2
    for kw in (dict(k=_cache(L, h=3)), dict(k=_cache(L, h=kh, ps=32)), dict(k=_cache(L, h=kh, n=9)), dict(v=_cache(L, d=12)),
               dict(heads=0), dict(heads=3), dict(t=9), dict(scale=float("nan")), dict(scale=float("inf")), dict(width=0),
               dict(n=-1), dict(stride=4096 + 4), dict(stride=8), dict(table=0), dict(table=(1 << 25) + 2), dict(lens=0),
               dict(q=(1 << 28) + 8), dict(q=0), dict(out=(1 << 30) + 8), dict(out=0), dict(width=1 << 28)):
        assert call(**kw) == bad, kw
    assert call(t=L.TQ_F32) == uns
    assert call(k=_cache(L, h=kh, d=64), v=_cache(L, d=256)) == uns
    assert call(k=_cache(L, h=kh, d=128), v=_cache(L, d=64)) == uns
    assert call(ws=0) == wsp and call(ws=(1 << 31) + 64) == wsp
    heads = 4
    need = (L.tq_paged4_prefill_workspace(_cache(L, h=kh), _cache(L), heads, 3, 9, 64) if ragged
            else L.tq_paged4_decode_workspace(_cache(L, h=kh), _cache(L), heads, 3))
    assert need > 256 and call(ws_bytes=need - 1, max_len=64) == wsp
    assert call(n=0) == L.TQ_OK
    if ragged:
        assert call(rows=0) == L.TQ_OK
        assert call(rows=-1) == bad and call(max_rows=-1) == bad and call(max_len=-1) == bad and call(qs=0) == bad
        assert call(rows=1 << 31) == bad
    if diff:
        for kw in (dict(lam=0), dict(lam=3), dict(nw=2), dict(eps=-1.0), dict(eps=float("nan")), dict(osc=float("inf"))):
            assert call(**kw) == bad, kw


def test_workspace_sizes_refuse():
    L = _lib()
    k, v = _cache(L), _cache(L)
    assert L.tq_paged4_decode_workspace(k, v, 4, 1) == L.tq_paged4_decode_workspace(k, v, 4, 1000) > 0
    assert L.tq_paged4_decode_workspace(k, v, 5, 1) == 0 and L.tq_paged4_decode_workspace(k, v, 4, -1) == 0
    assert L.tq_paged4_decode_workspace(_cache(L, h=3), v, 6, 1) == 0
    assert L.tq_paged4_prefill_workspace(k, v, 4, 2, 100, 1000) > 0
    assert L.tq_paged4_prefill_workspace(k, v, 4, 2, -1, 1000) == 0
    assert L.tq_paged4_prefill_workspace(k, v, 4, 2, 100, -1) == 0


@pytest.mark.parametrize("wk,wv,diff", [(64, 64, 0), (128, 128, 0), (256, 128, 0), (256, 256, 0), (64, 64, 1), (64, 128, 1),
                                        (128, 128, 1), (128, 256, 1)])
@pytest.mark.parametrize("columns", [8, 16])
def test_every_cta_of_a_launch_has_room_in_the_merge(wk, wv, diff, columns):
    # one item shared by the whole grid, on devices of any number of SMs
    import ctypes
    L = _lib()
    merge, smem = ctypes.c_int(), ctypes.c_int()
    for sms in (1, 2, 108, 152, 153, 200, 304, 511, 1000, 20000):
        ctas = L.lib.tq_testing_paged4_few_grid(wk, wv, columns, diff, sms, merge, smem)
        assert 0 < ctas <= 2 * sms and merge.value <= smem.value <= 227 * 1024
        assert sms > 152 or ctas in (sms, 2 * sms)               # every SM is used


def test_the_workspace_head_is_the_headers():
    import os
    import re
    import quantized_kv_cache_tq_gb300 as tq
    text = open(os.path.join(os.path.dirname(os.path.dirname(tq.__file__)), "include", "tq.h")).read()
    assert int(re.search(r"#define TQ_PAGED4_WORKSPACE_HEAD (\d+)", text).group(1)) == _lib().PAGED4_WORKSPACE_HEAD


def test_a_calls_own_workspace_is_cleared_no_further_than_it_has_to(monkeypatch):
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    head = _lib().PAGED4_WORKSPACE_HEAD
    names = tq._t()
    monkeypatch.setattr(names, "empty", lambda n, **kw: torch.full((n,), 7, **kw))
    ws = tq._paged4_ws(5 * head, "cpu")
    assert ws.numel() == 5 * head and not ws[:head].any() and bool((ws[head:] == 7).all())
    assert not tq._paged4_ws(0, "cpu").any()


@pytest.mark.parametrize("kind", ["prefill", "diff_prefill"])
@pytest.mark.parametrize("dk,dv,hkv,group", [(128, 128, 8, 4), (64, 64, 2, 1), (64, 128, 4, 2), (128, 128, 1, 16), (256, 256, 2, 2)])
def test_a_prefill_workspace_serves_every_smaller_call(kind, dk, dv, hkv, group):
    # (256, 256) and, in one map, (64, 128): forms that the call or the prompt kernel does not take
    L = _lib()
    maps = 2 if kind == "diff_prefill" else 1
    k, v, heads = _cache(L, h=maps * hkv, d=dk), _cache(L, h=hkv, d=dv), hkv * group
    size = lambda rows, n_seq, max_len: L.tq_paged4_prefill_workspace(k, v, heads, n_seq, rows, max_len)  # noqa: E731
    steps = [0, 1, 2, 3, 4, 5, 8, 16, 17, 30, 40, 64, 100, 128, 200, 300, 512, 700, 920, 1016, 1024, 1500, 2048]
    most = size(2048, 8, 32768)
    if (dk, dv, maps) in ((64, 128, 1), (256, 256, 2)):
        assert most == 0
        return
    last = 0
    for rows in steps:
        got = {size(rows, n_seq, max_len) for n_seq in (1, 3, 8) for max_len in (0, 64, 1000, 4096, 8192, 32768)}
        assert last <= min(got) and max(got) <= most, rows
        last = max(got)
    # what a call asks for is its own rows' size, whatever the hints (the few-row kernel's, if they choose that)
    for rows in (1, 9, 64, 920):
        need = size(rows, 3, 64)
        for max_rows in (0, 1, 40, 5000):
            for max_len in (0, 64, 4096, 100000):
                a = dict(k=k, v=v, rows=rows, heads=heads, stride=maps * heads * dk, max_rows=max_rows, max_len=max_len)
                few = L.tq_paged4_decode_workspace(k, v, heads, 3)
                assert _attend(L, kind, **a, ws_bytes=min(need, few) - 1) == L.TQ_ERR_WORKSPACE
                if max_rows == 0 or max_rows >= rows:
                    assert _attend(L, kind, **a, ws_bytes=need - 1) == L.TQ_ERR_WORKSPACE


def test_python_calls_refuse_before_the_library():
    # tensors on the CPU: every check that needs no device comes first
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    c = tq.Paged4Cache(2, 128, 16, 4, device="cpu")
    q = torch.zeros((1, 4, 128), dtype=torch.float16)
    table, lens = torch.zeros((1, 2), dtype=torch.int32), torch.zeros((1,), dtype=torch.int32)
    for bad in (dict(q=q.float()), dict(q=q[:, :, :64]), dict(q=q[0]), dict(table=table.long()), dict(table=table[0]),
                dict(lens=lens.long()), dict(lens=torch.zeros((2,), dtype=torch.int32)), dict(q=q.expand(2, 4, 128)),
                dict(out=torch.zeros((1, 4, 128))), dict()):
        a = dict(q=q, table=table, lens=lens, out=None)
        a.update(bad)
        with pytest.raises(ValueError):
            tq.paged4_decode(c, c, a["table"], a["lens"], a["q"], out=a["out"])
    with pytest.raises(ValueError):
        tq.paged4_set_rows(c, c, q[:, :2], q[:, :2].bfloat16(), torch.zeros((1,), dtype=torch.int64))
    with pytest.raises(ValueError):
        tq.paged4_set_rows(c, c, q[:, :2], q[:, ::2], torch.zeros((1,), dtype=torch.int64))
    with pytest.raises(ValueError):
        tq.Paged4Cache.from_planes(c.codes, c.scales[:, :1], 128)
    for ws in (torch.zeros(4096, dtype=torch.int32), torch.zeros(4096, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="ws: "):
            tq.paged4_decode(c, c, table, lens, q, ws=ws)
    with pytest.raises(tq.TQError):
        tq.Paged4Cache(2, 100, 16, 4, device="cpu")


@pytest.mark.parametrize("kind", ["decode", "prefill", "diff_decode", "diff_prefill"])
def test_attention_calls_refuse_tables_near_32_bits(kind):
    # lengths are rounded up to tiles of keys in 32 bits: tables end 2^16 cells before
    L = _lib()
    kh = 4 if "diff" in kind else 2
    k, v = _cache(L, h=kh, ps=1024), _cache(L, ps=1024)
    assert _attend(L, kind, k=k, v=v, width=(1 << 21) - 1) == L.TQ_ERR_INVALID_ARG
    assert _attend(L, kind, k=k, v=v, width=(1 << 21) - 63) == L.TQ_ERR_INVALID_ARG
    # (at the limit the checks go on, to a workspace of no bytes)
    assert _attend(L, kind, k=k, v=v, width=(1 << 21) - 64, ws_bytes=0) == L.TQ_ERR_WORKSPACE
