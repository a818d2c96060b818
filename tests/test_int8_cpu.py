"""Rotary positions and the int8 cache without a GPU: the plain formulas against
hand-made cases, frequencies and turns against them, and every refusal of the C
ABI and of the Python calls."""
import ctypes as C
import math

import numpy as np
import pytest

from oracle import int8 as I


def _lib():
    from quantized_kv_cache_tq_gb300 import _lib
    return _lib


# ---------------------------------------------------------------- the formulas

def test_quantise_by_hand():
    c, s = I.quantise(np.array([[-1.27, 0.635, 0.0, 0.01, 1.27, -0.004]]))
    assert s[0] == np.float16(0.01) and list(c[0]) == [-127, 63, 0, 1, 127, 0] or list(c[0]) == [-127, 64, 0, 1, 127, 0]
    c, s = I.quantise(np.array([[0.0] * 4, [np.nan, 0, 0, 127.0], [np.inf, 1, 0, -np.inf], [1e-9, 0, 0, 0]]))
    assert s[0] == 0 and not c[0].any()
    assert s[1] == 1 and list(c[1]) == [0, 0, 0, 127]
    assert s[2] == 65504 and list(c[2]) == [127, 0, 0, -127]
    assert s[3] == 0 and not c[3].any()


def test_error_is_at_most_half_a_step():
    x = np.random.default_rng(0).standard_normal((200, 96)).astype(np.float32)
    c, s = I.quantise(x)
    # half a step, and the scale's rounding: up to 127 steps of relative 2^-11
    tol = (0.5 + 127 * 2.0 ** -11) * s.astype(np.float64)
    assert np.all(np.abs(I.values(c, s) - x) <= tol[:, None] + 1e-6)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotation_by_hand(layout):
    x = np.arange(1.0, 9.0).reshape(1, 1, 8)
    f = [0.5, 0.25]
    y = I.turned(x, [3], f, layout)[0, 0]
    pairs = [(0, 2), (1, 3)] if layout == "half" else [(0, 1), (2, 3)]
    for j, (a, b) in enumerate(pairs):
        t = 3 * f[j]
        assert math.isclose(y[a], x[0, 0, a] * math.cos(t) - x[0, 0, b] * math.sin(t), rel_tol=1e-12)
        assert math.isclose(y[b], x[0, 0, a] * math.sin(t) + x[0, 0, b] * math.cos(t), rel_tol=1e-12)
    assert np.array_equal(y[4:], x[0, 0, 4:])
    assert np.allclose(I.turned(y[None, None], [3], f, layout, inverse=True), x, rtol=1e-12)
    w = np.linspace(0.5, 2, 8)
    n = I.turned(x, [0], f, layout, norm=w, eps=0.1)[0, 0]
    assert np.allclose(n, w * x[0, 0] / math.sqrt((x ** 2).mean() + 0.1), rtol=1e-12)


def test_attention_by_loops():
    rng = np.random.default_rng(1)
    kc, vc = I.Cache(1, 16, 40), I.Cache(1, 16, 40)
    xk, xv = rng.standard_normal((20, 1, 16)), rng.standard_normal((20, 1, 16))
    slots = [4 * 8 + i for i in range(8)] + [i for i in range(8)] + [16 + i for i in range(4)]
    kc.set_rows(xk, slots)
    vc.set_rows(xv, slots)
    q = rng.standard_normal((1, 2, 16))
    out, bound = I.attention(kc, vc, [[4, 0, 2]], [19], 8, q, 0.5, 11)
    k, v = I.values(*I.quantise(xk)), I.values(*I.quantise(xv))
    for h in range(2):
        e = [np.exp(0.5 * float(q[0, h] @ k[t, 0])) for t in range(19)]
        assert np.allclose(out[0, h], sum(w * v[t, 0] for t, w in enumerate(e)) / sum(e), rtol=1e-12)
    assert np.all(bound > 0) and np.all(bound < 2e-3)
    assert not I.attention(kc, vc, [[4, 0, 2]], [0], 8, q, 0.5, 11)[0].any()


# ---------------------------------------------------------------- frequencies and turns

SCALINGS = [("plain", {}), ("linear", dict(factor=4.0)), ("base", dict(factor=8.0)),
            ("rotations", dict(factor=8.0, original_len=8192.0, beta_fast=4.0, beta_slow=1.0)),
            ("pairs", dict(factor=16.0, original_len=4096.0, beta_fast=32.0, beta_slow=1.0)),
            ("pairs", dict(factor=0.5, original_len=4096.0, beta_fast=32.0, beta_slow=1.0)),
            ("pairs", dict(factor=4.0, original_len=3.0, beta_fast=32.0, beta_slow=1.0)),      # no pair turns once
            ("pairs", dict(factor=4.0, original_len=1e30, beta_fast=32.0, beta_slow=1.0))]     # all of them do


@pytest.mark.parametrize("rot", [2, 4, 20, 64, 128, 256])
@pytest.mark.parametrize("kind,more", SCALINGS)
def test_frequencies(kind, more, rot):
    import quantized_kv_cache_tq_gb300 as tq
    if kind == "base" and rot == 2:
        pytest.skip("a base cannot be raised for one pair")
    r = tq.Rope(rot, 500000.0, scaling=kind, device="cpu", **more)
    f, m = I.frequencies(rot, 500000.0, kind, **more)
    assert np.allclose(r.frequencies, f, rtol=1e-14) and math.isclose(r.magnitude, m, rel_tol=1e-6)
    assert r.turns.shape == (rot // 2,)
    assert tq.Rope(rot, frequencies=f, magnitude=0.5, device="cpu").magnitude == 0.5


def test_turns_are_frequencies_modulo_a_turn():
    L = _lib()
    f = [1.0, -1.0, 0.0, 2 * math.pi, 7.5, -7.5, 1e-9, 3e5, 1e-30, -1e-30]
    t = L.tq_rope_turns(f)
    assert t[1] == 2 ** 64 - t[0] and t[2] == 0 and t[8] == 0 and t[9] == 0 and t[5] == 2 ** 64 - t[4]
    for x, u in zip(f, t):
        want = x / (2 * math.pi)
        # the quotient's rounding in 64 bits, and the cut to 2^-64
        assert abs((u / 2 ** 64 - want + 0.5) % 1 - 0.5) <= abs(want) * 2.0 ** -52 + 2.0 ** -52
    # a position far away: the integer product modulo 2^64 is the angle
    p = 2 ** 31 - 1
    got = (p * t[0] % 2 ** 64) / 2 ** 64
    want = p / (2 * math.pi)
    assert abs((got - want + 0.5) % 1 - 0.5) <= want * 2.0 ** -51


def test_frequency_refusals():
    L = _lib()

    def ask(rot=64, base=10000.0, kind=0, factor=2.0, original=4096.0, fast=32.0, slow=1.0):
        f, m = (C.c_double * 128)(), C.c_float()
        s = L.tq_rope_scaling(kind, factor, original, fast, slow)
        return L.lib.tq_rope_frequencies(rot, base, C.byref(s), f, C.byref(m))

    assert ask() == L.TQ_OK and ask(kind=4) == L.TQ_OK
    nan, inf = float("nan"), float("inf")
    for bad in (dict(rot=0), dict(rot=3), dict(rot=258), dict(rot=-2), dict(base=0.0), dict(base=-1.0), dict(base=nan),
                dict(base=inf), dict(kind=5), dict(kind=-1), dict(kind=1, factor=0.0), dict(kind=1, factor=nan),
                dict(kind=2, rot=2), dict(kind=2, factor=1e300, base=1e300), dict(kind=3, original=0.0),
                dict(kind=3, fast=1.0), dict(kind=3, slow=0.0), dict(kind=3, fast=inf), dict(kind=4, base=1.0),
                dict(kind=4, base=0.5), dict(kind=4, original=inf)):
        assert ask(**bad) == L.TQ_ERR_INVALID_ARG, bad
    f, m = (C.c_double * 4)(), C.c_float()
    assert L.lib.tq_rope_frequencies(8, 100.0, None, f, C.byref(m)) == L.TQ_OK and m.value == 1.0
    assert L.lib.tq_rope_frequencies(8, 100.0, None, None, C.byref(m)) == L.TQ_ERR_INVALID_ARG
    with pytest.raises(L.TQError):
        L.tq_rope_turns([1.0, nan])


# ---------------------------------------------------------------- refusals of the C ABI (nothing reaches a device)

A = 1 << 24            # an address that is aligned and never read


def _heads(L, **kw):
    d = dict(src=A, src_stride=512, dst=A + 4096, dst_stride=512, norm_weight=None, n_heads=4)
    d.update(kw)
    return L.tq_head_rows(**d)


def _cache(L, **kw):
    d = dict(n_kv_heads=4, head_dim=128, n_cells=100, rows=A, scales=A)
    d.update(kw)
    return L.tq_int8(**d)


def _rope(L, **kw):
    d = dict(rot_dim=64, layout=0, magnitude=1.0, turns=A)
    d.update(kw)
    return L.tq_rope(**d)


def test_rope_rows_refusals():
    L = _lib()

    def call(rope=None, q=None, k=None, d=128, type=1, eps=1e-6, inverse=0, pos=A, n=3, st=None, none=False):
        return L.tq_rope_rows(rope or _rope(L), None if none else q or _heads(L), k, d, type, eps, inverse, pos, n, st,
                              None)

    assert call(n=0) == L.TQ_OK and call(n=0, pos=None) == L.TQ_OK
    bad = [dict(none=True), dict(d=0), dict(d=12), dict(d=264), dict(d=32), dict(type=3), dict(n=-1), dict(n=1 << 31),
           dict(rope=_rope(L, rot_dim=63)), dict(rope=_rope(L, rot_dim=0)), dict(rope=_rope(L, layout=2)),
           dict(rope=_rope(L, magnitude=float("inf"))), dict(q=_heads(L, n_heads=0)), dict(q=_heads(L, n_heads=65537)),
           dict(q=_heads(L, src_stride=504)), dict(q=_heads(L, src_stride=516)), dict(q=_heads(L, dst_stride=8)),
           dict(q=_heads(L, dst=A, dst_stride=1024)), dict(k=_heads(L, n_heads=5)),
           dict(q=_heads(L, norm_weight=A), inverse=1), dict(q=_heads(L, norm_weight=A), eps=float("nan")),
           dict(q=_heads(L, norm_weight=A), eps=-1.0)]
    for kw in bad:
        assert call(**kw) == L.TQ_ERR_INVALID_ARG, kw
        assert call(**{**kw, "n": kw.get("n", 0)}) == L.TQ_ERR_INVALID_ARG, kw      # with no rows, too
    for kw in (dict(q=_heads(L, src=A + 8)), dict(q=_heads(L, src=None)), dict(q=_heads(L, dst=None)),
               dict(q=_heads(L, norm_weight=A + 4)), dict(pos=A + 2), dict(pos=None), dict(st=A + 1),
               dict(rope=_rope(L, turns=A + 8)), dict(rope=_rope(L, turns=None)), dict(k=_heads(L, dst=A + 8))):
        assert call(**kw) == L.TQ_ERR_INVALID_ARG, kw
    assert L.lib.tq_rope_rows(None, _heads(L), None, 128, 1, 0.0, 0, A, 1, None, None) == L.TQ_ERR_INVALID_ARG


def test_int8_row_refusals():
    L = _lib()

    def rows(fn, k=None, v=None, kp=A, ks=512, vp=A, vs=512, type=1, slots=A, n=3, st=None):
        return getattr(L, fn)(k or _cache(L), v or _cache(L), kp, ks, vp, vs, type, slots, n, st, None)

    for fn in ("tq_int8_set_rows", "tq_int8_get_rows"):
        assert rows(fn, n=0) == L.TQ_OK
        for kw in (dict(k=_cache(L, n_kv_heads=0)), dict(k=_cache(L, n_kv_heads=65537)), dict(v=_cache(L, head_dim=120)),
                   dict(v=_cache(L, head_dim=272)), dict(v=_cache(L, head_dim=0)), dict(v=_cache(L, n_cells=0)),
                   dict(k=_cache(L, n_cells=1 << 30), v=_cache(L, n_cells=1 << 30)), dict(v=_cache(L, n_cells=99)),
                   dict(v=_cache(L, rows=A + 8)), dict(k=_cache(L, scales=None)), dict(type=3), dict(n=-1),
                   dict(n=1 << 31), dict(ks=504), dict(vs=513)):
            assert rows(fn, **{"n": 0, **kw}) == L.TQ_ERR_INVALID_ARG, kw
            assert rows(fn, **kw) == L.TQ_ERR_INVALID_ARG, kw
        for kw in (dict(kp=A + 8), dict(vp=None), dict(slots=A + 4), dict(st=A + 2)):
            assert rows(fn, **kw) == L.TQ_ERR_INVALID_ARG, kw


def test_int8_rope_set_rows_refusals():
    L = _lib()
    keys = lambda **kw: _heads(L, **{"dst": None, **kw})  # noqa: E731

    def call(k=None, v=None, rope=None, q=0, kr=None, vp=A, vs=512, type=1, eps=1e-6, pos=A, slots=A, n=3, st=None):
        return L.tq_int8_rope_set_rows(k or _cache(L), v or _cache(L), rope or _rope(L), _heads(L) if q == 0 else q,
                                       kr or keys(), vp, vs, type, eps, pos, slots, n, st, None)

    assert call(n=0) == L.TQ_OK and call(n=0, q=None) == L.TQ_OK
    for kw in (dict(rope=_rope(L, rot_dim=130)), dict(rope=_rope(L, layout=-1)), dict(kr=keys(n_heads=3)),
               dict(kr=keys(src_stride=256)), dict(q=_heads(L, dst_stride=256)), dict(q=_heads(L, n_heads=-1)),
               dict(v=_cache(L, n_cells=7)), dict(type=9), dict(vs=504), dict(n=-1),
               dict(kr=keys(norm_weight=A), eps=float("inf"))):
        assert call(**{"n": 0, **kw}) == L.TQ_ERR_INVALID_ARG, kw
        assert call(**kw) == L.TQ_ERR_INVALID_ARG, kw
    for kw in (dict(kr=keys(dst=A)), dict(kr=keys(src=None)), dict(q=_heads(L, dst=None)), dict(vp=A + 4),
               dict(pos=None), dict(slots=None), dict(st=A + 3), dict(rope=_rope(L, turns=A + 4)),
               dict(kr=keys(norm_weight=A + 8))):
        assert call(**kw) == L.TQ_ERR_INVALID_ARG, kw
    assert L.lib.tq_int8_rope_set_rows(_cache(L), _cache(L), _rope(L), None, None, A, 512, 1, 0.0, A, A, 1, None,
                                       None) == L.TQ_ERR_INVALID_ARG


def test_int8_decode_refusals_and_workspace():
    L = _lib()
    need = L.tq_int8_decode_workspace(_cache(L), _cache(L), 8, 3)
    assert need > 4096 and need == L.tq_int8_decode_workspace(_cache(L), _cache(L), 64, 5000)
    assert L.tq_int8_decode_workspace(_cache(L, head_dim=64), _cache(L), 8, 3) == 0           # widths
    assert L.tq_int8_decode_workspace(_cache(L, head_dim=192), _cache(L), 8, 3) == need
    assert L.tq_int8_decode_workspace(_cache(L), _cache(L), 9, 3) == 0
    # one workspace serves the paged 4-bit decode, too
    for d in (64, 128, 256):
        p = L.tq_paged4(4, d, 16, 10, A, A)
        assert 0 < L.lib.tq_paged4_decode_workspace(C.byref(p), C.byref(p), 8, 3) <= need

    def call(k=None, v=None, page=16, table=A, width=10, lens=A, n=3, q=A, type=1, stride=1024, heads=8, scale=0.1,
             out=A, ws=A, size=need):
        return L.tq_int8_decode(k or _cache(L), v or _cache(L), page, table, width, lens, n, q, type, stride, heads, scale,
                                out, ws, size, None)

    assert call(n=0) == L.TQ_OK
    for kw in (dict(page=0), dict(page=12), dict(page=1 << 17), dict(page=-16), dict(width=0), dict(heads=6),
               dict(heads=0), dict(stride=1000), dict(stride=1028), dict(scale=float("nan")), dict(type=5),
               dict(width=1 << 27), dict(n=-1), dict(n=1 << 25), dict(v=_cache(L, n_kv_heads=2)),
               dict(v=_cache(L, n_cells=1)), dict(n=1 << 24, heads=1024, stride=1 << 20)):
        assert call(**{"n": 0, **kw}) == L.TQ_ERR_INVALID_ARG, kw
        assert call(**kw) == L.TQ_ERR_INVALID_ARG, kw
    assert call(type=0) == L.TQ_ERR_UNSUPPORTED
    assert call(v=_cache(L, head_dim=256)) == L.TQ_ERR_UNSUPPORTED
    for kw in (dict(table=None), dict(lens=A + 2), dict(q=A + 8), dict(out=None)):
        assert call(**kw) == L.TQ_ERR_INVALID_ARG, kw
    for kw in (dict(ws=None), dict(ws=A + 128), dict(size=need - 1)):
        assert call(**kw) == L.TQ_ERR_WORKSPACE, kw


# ---------------------------------------------------------------- refusals of the Python calls

def test_python_refusals():
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    z = lambda *s, t=torch.float16: torch.zeros(s, dtype=t)  # noqa: E731
    rope = tq.Rope(32, device="cpu")
    pos, slots = z(3, t=torch.int32), z(3, t=torch.int64)
    kc, vc = tq.Int8Cache(2, 64, 40, device="cpu"), tq.Int8Cache(2, 64, 40, device="cpu")
    assert kc.rows.shape == (40, 2, 64) and kc.scales.shape == (40, 2)
    assert tq.Int8Cache.from_planes(kc.rows, kc.scales).head_dim == 64

    def no(call):
        with pytest.raises(ValueError) as e:
            call()
        assert "CUDA device" not in str(e.value)

    no(lambda: tq.Int8Cache(2, 72, 40, device="cpu"))
    no(lambda: tq.Int8Cache.from_planes(kc.rows, kc.scales.float()))
    no(lambda: tq.Int8Cache.from_planes(kc.rows, kc.scales[:, :1]))
    no(lambda: tq.Rope(32, layout="other", device="cpu"))
    no(lambda: tq.Rope(32, scaling="other", device="cpu"))
    no(lambda: tq.Rope(32, frequencies=[1.0], device="cpu"))
    with pytest.raises(tq.TQError):
        tq.Rope(31, device="cpu")
    q, k = z(3, 4, 64), z(3, 2, 64)
    # tensors of the host: refused for that, after everything else was found in order
    with pytest.raises(ValueError, match="CUDA device"):
        tq.rope_rows(rope, pos, q, k)
    with pytest.raises(ValueError, match="CUDA device"):
        tq.int8_rope_set_rows(kc, vc, rope, pos, q, k, k, slots)
    with pytest.raises(ValueError, match="CUDA device"):
        tq.int8_set_rows(kc, vc, k, k, slots)
    for call in (lambda: tq.rope_rows(rope, pos.long(), q), lambda: tq.rope_rows(rope, pos[:2], q),
                 lambda: tq.rope_rows(rope, pos, q, k.float()), lambda: tq.rope_rows(rope, pos, q.double()),
                 lambda: tq.rope_rows(rope, pos, q, z(2, 2, 64)), lambda: tq.rope_rows(rope, pos, q, z(3, 2, 32)),
                 lambda: tq.rope_rows(rope, pos, q.transpose(1, 2)), lambda: tq.rope_rows(rope, pos, q[0]),
                 lambda: tq.rope_rows(rope, pos, q, q_out=q.float()), lambda: tq.rope_rows(rope, pos, q, q_out=k),
                 lambda: tq.rope_rows(rope, pos, q, q_norm=z(64)), lambda: tq.rope_rows(rope, pos, q, k_out=k),
                 lambda: tq.rope_rows(rope, pos, q, q_norm=z(32, t=torch.float32)),
                 lambda: tq.rope_rows(rope, pos, q, dev_status=z(1)),
                 lambda: tq.int8_set_rows(kc, vc, k, k.float(), slots), lambda: tq.int8_set_rows(kc, vc, k, q, slots),
                 lambda: tq.int8_set_rows(kc, vc, k, k, slots.int()),
                 lambda: tq.int8_get_rows(kc, vc, slots, dtype=torch.float32, k_out=k),
                 lambda: tq.int8_get_rows(kc, vc, slots, k_out=k, v_out=k.float()),
                 lambda: tq.int8_rope_set_rows(kc, vc, rope, pos, q, k, k.float(), slots),
                 lambda: tq.int8_rope_set_rows(kc, vc, rope, pos, q.float(), k, k, slots),
                 lambda: tq.int8_rope_set_rows(kc, vc, rope, pos, None, k, k, slots, q_out=q),
                 lambda: tq.int8_rope_set_rows(kc, vc, rope, pos, z(3, 4, 32), k, k, slots),
                 lambda: tq.int8_decode(kc, vc, z(3, 5, t=torch.int32), pos, q.float()),
                 lambda: tq.int8_decode(kc, vc, z(3, 5, t=torch.int64), pos, q),
                 lambda: tq.int8_decode(kc, vc, z(3, 5, t=torch.int32), pos[:2], q),
                 lambda: tq.int8_decode(kc, vc, z(3, 5, t=torch.int32), pos, q, out=q.float()),
                 lambda: tq.int8_decode(kc, vc, z(3, 5, t=torch.int32), pos, q, ws=q)):
        no(call)
