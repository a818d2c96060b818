"""Rotary positions and the int8 cache on the GPU against the plain formulas of
oracle/int8.py.

Codes, scales and read-back rows are compared exactly where no rotation precedes
them.  Rotated rows are held to half a step of their type plus the errors of
fp32 arithmetic; attention outputs to half a step (2^-8 bfloat16, 2^-11 binary16,
relative) plus the bound that oracle.int8.attention derives."""
import math

import numpy as np
import pytest

from oracle import int8 as I

pytestmark = pytest.mark.gpu

HALF = {"float32": 2.0 ** -24, "float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}
TINY = {"float32": 2.0 ** -149, "float16": 2.0 ** -25, "bfloat16": 2.0 ** -133}


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _rows(rng, n, h, d):
    """N(0, 1) with an offset per channel and a few channels eight times as large."""
    x = rng.standard_normal((n, h, d)) + 0.3 * rng.standard_normal((h, d))
    x[:, :, rng.permutation(d)[:max(1, d // 32)]] *= 8
    return x.astype(np.float32)


def _gpu(x, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(getattr(torch, dtype))


def _turn_error(y, rope, positions):
    """What fp32 may be off by in rows of norm-scaled elements y: each product and sum of the pair rounds, 2^-24 of
    (|a| + |b|) each, and the sine and cosine carry 2^-22 (their own error and the reduced angle's, at most a
    quarter turn's 2^-24) and the angle's own: 1.5 2^-32 of a turn cut off, and 2^-51 of the whole angle, which both
    sides compute in 64 bits."""
    y = np.abs(y)
    f = np.abs(np.asarray(rope.frequencies))
    rot = rope.rot_dim
    first = np.arange(rot // 2) if rope.layout == "half" else np.arange(0, rot, 2)
    second = first + rot // 2 if rope.layout == "half" else first + 1
    angle = 2 * math.pi * 1.5 * 2.0 ** -32 + np.maximum(positions, 0)[:, None] * f * 2.0 ** -51
    both = (y[..., first] + y[..., second]) * (2.0 ** -22 + 4 * 2.0 ** -24 + angle[:, None]) * abs(rope.magnitude)
    err = np.zeros_like(y)
    err[..., first] = err[..., second] = both
    return err


def _check_turned(got, x, positions, rope, dtype, norm=None, eps=0.0, inverse=False):
    ref = I.turned(x, positions, rope.frequencies, rope.layout, np.float32(rope.magnitude), norm, eps, inverse)
    y = np.asarray(x, np.float64)
    if norm is not None:
        y = I.turned(x, np.zeros_like(positions), rope.frequencies, rope.layout, 1.0, norm, eps)
    err = _turn_error(y, rope, np.asarray(positions, np.float64))
    if norm is not None:
        # the reciprocal root's 2^-22, the sum of squares' d roundings (2^-24 each, halved by the root), two products
        err = err + np.abs(ref) * (2.0 ** -22 + x.shape[-1] * 2.0 ** -25 + 2.0 ** -22)
        rot = rope.rot_dim
        err[..., :rot] += np.abs(y[..., :rot]).max(-1, keepdims=True) * (2.0 ** -21 + x.shape[-1] * 2.0 ** -25)
    tol = HALF[dtype] * (np.abs(ref) + err) + err + TINY[dtype]
    live = np.asarray(positions) >= 0
    d = np.abs(_np(got) - ref)[live] / tol[live]
    assert np.all(np.isfinite(d)) and d.max(initial=0.0) <= 1.0, f"{d.max():.2f} times the tolerance"


# ---------------------------------------------------------------- rotary positions

@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rot", [(128, 128), (128, 64), (80, 20), (96, 24), (64, 64), (256, 256), (8, 8), (8, 2),
                                   (40, 24), (192, 64), (248, 246), (16, 16), (128, 16)])
def test_rope_rows(dtype, layout, d, rot):
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    rng = np.random.default_rng(d + rot)
    n, hq, hk = 45, 6, 3
    rope = tq.Rope(rot, 10000.0, layout=layout, scaling="linear", factor=2.5, magnitude=1.25)
    x, y = _gpu(_rows(rng, n, hq, d), dtype), _gpu(_rows(rng, n, hk, d), dtype)
    pos = rng.integers(0, 40000, n).astype(np.int32)
    pos[:5] = [0, 1, 2 ** 31 - 1, -1, 1 << 20]
    pos[-1] = -1
    q, k = torch.full_like(x, 7.0), torch.full_like(y, 7.0)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = tq.rope_rows(rope, _gpu(pos), x, y, q_out=q, k_out=k, dev_status=st)
    assert got[0] is q and got[1] is k and int(st) == 0
    for src, out in ((x, q), (y, k)):
        _check_turned(out, _np(src), pos, rope, dtype)
        assert torch.equal(out[..., rot:][pos >= 0], src[..., rot:][pos >= 0])         # what does not turn, bit for bit
        assert bool((out[pos < 0] == 7).all())
        assert torch.equal(out[0, :, :rot], (src[0, :, :rot].float() * 1.25).to(src.dtype))    # position 0
    # in place, and queries alone; new outputs begin as zeros
    z = x.clone()
    tq.rope_rows(rope, _gpu(pos), z, q_out=z)
    assert torch.equal(z[pos >= 0], q[pos >= 0]) and torch.equal(z[pos < 0], x[pos < 0])
    w = tq.rope_rows(rope, _gpu(pos), x)
    assert torch.equal(w[pos >= 0], q[pos >= 0]) and not w[pos < 0].any()


@pytest.mark.parametrize("n", [1, 2, 33, 700, 5000])
@pytest.mark.parametrize("hq,hk,d,rot,layout,dtype", [(1, 1, 64, 64, "half", "bfloat16"), (7, 1, 64, 64, "half", "bfloat16"),
                                                      (32, 8, 128, 128, "half", "float16"), (9, 3, 80, 20, "half", "float16"),
                                                      (16, 16, 48, 24, "interleaved", "bfloat16"),
                                                      (5, 2, 256, 256, "half", "float32"), (6, 2, 40, 20, "half", "float32"),
                                                      (8, 4, 128, 64, "interleaved", "float32")])
def test_rope_rows_of_any_number(n, hq, hk, d, rot, layout, dtype):
    # every split of rows and heads over threads gives the same bits as a row and a head by themselves
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    g = torch.Generator(device="cuda").manual_seed(n)
    rope = tq.Rope(rot, 500000.0, layout=layout, scaling="pairs", factor=8.0, original_len=8192.0)
    q = torch.randn((n, hq, d), generator=g, device="cuda").to(getattr(torch, dtype))
    k = torch.randn((n, hk, d), generator=g, device="cuda").to(q.dtype)
    pos = torch.randint(0, 1 << 20, (n,), generator=g, device="cuda", dtype=torch.int32)
    if n > 5:
        pos[n // 3::7] = -1
    live = (pos >= 0).tolist()
    a, b = tq.rope_rows(rope, pos, q, k, q_out=torch.full_like(q, 7.0), k_out=torch.full_like(k, 7.0))
    at = [i for i in range(n) if live[i]]
    at = sorted({at[(len(at) - 1) * i // 40] for i in range(41)})
    for x, y in ((q, a), (k, b)):
        _check_turned(y[at], _np(x[at]), pos[at].cpu().numpy(), rope, dtype)
        assert bool((y[pos < 0] == 7).all()) and bool((y[pos >= 0] != 7).any(-1).all())
    for i in at[::8]:
        for h in {0, hq - 1}:
            assert torch.equal(tq.rope_rows(rope, pos[i:i + 1], q[i:i + 1, h:h + 1].contiguous())[0, 0], a[i, h])
        assert torch.equal(tq.rope_rows(rope, pos[i:i + 1], k[i:i + 1])[0], b[i])
    # in place, all at once
    c, e = q.clone(), k.clone()
    tq.rope_rows(rope, pos, c, e, q_out=c, k_out=e)
    assert torch.equal(c[pos >= 0], a[pos >= 0]) and torch.equal(e[pos >= 0], b[pos >= 0])
    assert torch.equal(c[pos < 0], q[pos < 0]) and torch.equal(e[pos < 0], k[pos < 0])


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("layout,d,rot", [("half", 128, 128), ("interleaved", 96, 48), ("half", 80, 20), ("half", 24, 16),
                                          ("interleaved", 8, 6), ("half", 256, 64)])
def test_rope_rows_normed(dtype, layout, d, rot):
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    rng = np.random.default_rng(d)
    n, hq, hk = 30, 4, 2
    rope = tq.Rope(rot, 10000.0, layout=layout)
    x, y = _gpu(_rows(rng, n, hq, d), dtype), _gpu(0.01 * _rows(rng, n, hk, d), dtype)
    x[3], y[4] = 0.0, 0.0
    wq, wk = rng.standard_normal(d).astype(np.float32), 1 + rng.random(d).astype(np.float32)
    pos = rng.integers(0, 9000, n).astype(np.int32)
    q, k = tq.rope_rows(rope, _gpu(pos), x, y, q_norm=_gpu(wq), k_norm=_gpu(wk), eps=1e-5)
    _check_turned(q, _np(x), pos, rope, dtype, wq, 1e-5)
    _check_turned(k, _np(y), pos, rope, dtype, wk, 1e-5)
    assert not q[3].any() and not k[4].any()
    # one of the two normed; a row of zeros without eps stays one
    q, k = tq.rope_rows(rope, _gpu(pos), x, y, k_norm=_gpu(wk), eps=0.0)
    _check_turned(q, _np(x), pos, rope, dtype)
    y[4] = 1.0
    _check_turned(k[5:], _np(y[5:]), pos[5:], rope, dtype, wk, 0.0)
    assert not k[4].any()


def test_rope_rows_strided_slices_in_place():
    # queries and keys as slices of one projection's output, turned where they are; the values beside them stay
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    rng = np.random.default_rng(3)
    n, hq, hk, d = 50, 8, 2, 64
    wide = _gpu(_rows(rng, n, 1, (hq + 2 * hk) * d + 24)[:, 0], "float16")
    was = wide.clone()
    q = wide[:, 8:8 + hq * d].unflatten(1, (hq, d))
    k = wide[:, 8 + hq * d:8 + (hq + hk) * d].unflatten(1, (hk, d))
    pos = torch.arange(n, dtype=torch.int32, device="cuda") * 37
    for rot in (64, 20):                                       # (20: halves that end inside eight elements)
        wide.copy_(was)
        rope = tq.Rope(rot)
        want = tq.rope_rows(rope, pos, q.contiguous(), k.contiguous())
        tq.rope_rows(rope, pos, q, k, q_out=q, k_out=k)
        assert torch.equal(q, want[0]) and torch.equal(k, want[1])
        rest = torch.cat([wide[:, :8], wide[:, 8 + (hq + hk) * d:]], 1)
        assert torch.equal(rest, torch.cat([was[:, :8], was[:, 8 + (hq + hk) * d:]], 1))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_inverse_is_the_gradient(layout):
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    rng = np.random.default_rng(5)
    n, h, d, rot = 12, 3, 32, 24
    rope = tq.Rope(rot, 10000.0, layout=layout, magnitude=0.75)
    pos = rng.integers(0, 5000, n).astype(np.int32)
    x, g = rng.standard_normal((n, h, d)).astype(np.float32), rng.standard_normal((n, h, d)).astype(np.float32)
    got = tq.rope_rows(rope, _gpu(pos), _gpu(g), inverse=True)
    _check_turned(got, g, pos, rope, "float32", inverse=True)
    # against differences of the loss sum(g * rope(x)), which is linear: any step serves
    base = _np(tq.rope_rows(rope, _gpu(pos), _gpu(x)))
    for e in (0, 5, rot // 2, rot - 1, rot, d - 1):
        up = x.copy()
        up[:, :, e] += 1.0
        step = (up[:, :, e].astype(np.float64) - x[:, :, e])
        diff = ((_np(tq.rope_rows(rope, _gpu(pos), _gpu(up))) - base) * g).sum(-1) / step
        # two results of magnitude up to 5, fp32 rounded, times gradients up to 5, over the d terms
        assert np.all(np.abs(diff - _np(got)[:, :, e]) <= d * 2 * 25 * 2.0 ** -22)
    # there and back
    one = tq.Rope(rot, layout=layout)
    back = tq.rope_rows(one, _gpu(pos), tq.rope_rows(one, _gpu(pos), _gpu(x)), inverse=True)
    assert np.all(np.abs(_np(back) - x) <= 2.0 ** -19 * np.abs(x).max())


@pytest.mark.parametrize("d,rot", [(64, 64), (40, 20)])
def test_rope_bad_positions_and_values_that_are_not_finite(d, rot):
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    rope = tq.Rope(rot)
    x = torch.ones((4, 2, d), device="cuda")
    x[1, 0, rot // 2 - 1], x[1, 1, 3] = float("inf"), float("nan")
    x[2, :, rot:] = float("inf")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = tq.rope_rows(rope, torch.tensor([3, 0, 5, -7], dtype=torch.int32, device="cuda"), x, dev_status=st)
    assert int(st) == 6 and not y[3].any()
    assert bool(torch.isinf(y[2, :, rot:]).all()) and bool(torch.isfinite(y[2, :, :rot]).all())
    bad = ~torch.isfinite(y[1])
    pairs = {0: {rot // 2 - 1, rot - 1}, 1: {3, 3 + rot // 2}}
    for h, at in pairs.items():                              # only the pairs that hold them are touched
        assert {int(i) for i in bad[h].nonzero().flatten()} <= at and bool(bad[h].any())
    # without a status word
    assert not tq.rope_rows(rope, torch.full((4,), -2, dtype=torch.int32, device="cuda"), x).any()


def test_rope_no_rows():
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    q = torch.empty((0, 2, 64), device="cuda")
    assert tq.rope_rows(tq.Rope(64), torch.empty(0, dtype=torch.int32, device="cuda"), q).shape == (0, 2, 64)


# ---------------------------------------------------------------- rows of the int8 cache

def _upload(c: I.Cache):
    import quantized_kv_cache_tq_gb300 as tq
    return tq.Int8Cache.from_planes(_gpu(c.rows.copy()), _gpu(c.scales.copy()))


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (80, 96), (128, 128), (192, 128), (256, 256), (16, 48), (240, 16)])
def test_set_and_get_rows(dtype, dk, dv):
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    rng = np.random.default_rng(dk + dv)
    n, hk, hv, cells = 77, 3, 2, 205
    # rows are slices of one wide buffer, as of a fused projection
    wide = _gpu(_rows(rng, n, 1, hk * dk + hv * dv + 16)[:, 0], dtype)
    xk = wide[:, 8:8 + hk * dk].unflatten(1, (hk, dk))
    xv = wide[:, 8 + hk * dk:8 + hk * dk + hv * dv].unflatten(1, (hv, dv))
    xk[3], xv[4] = -2.5, 0.0                                 # constant rows
    slots = rng.permutation(cells)[:n].astype(np.int64)
    slots[5], slots[9] = -1, -1
    kc, vc = I.Cache(hk, dk, cells), I.Cache(hv, dv, cells)
    kc.set_rows(_np(xk), slots)
    vc.set_rows(_np(xv), slots)
    gk, gv = tq.Int8Cache(hk, dk, cells), tq.Int8Cache(hv, dv, cells)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    gs = _gpu(slots)
    tq.int8_set_rows(gk, gv, xk, xv, gs, dev_status=st)
    for g, c in ((gk, kc), (gv, vc)):
        assert np.array_equal(g.rows.cpu().numpy(), c.rows)
        assert np.array_equal(g.scales.cpu().numpy().view(np.int16), c.scales.view(np.int16))
    # back: scale * code is exact in fp32, rounded once; skipped rows keep what they had
    out = torch.full((n, hk * dk + hv * dv + 8), 5.0, dtype=xk.dtype, device="cuda")
    ok, ov = out[:, :hk * dk].unflatten(1, (hk, dk)), out[:, hk * dk:hk * dk + hv * dv].unflatten(1, (hv, dv))
    tq.int8_get_rows(gk, gv, gs, k_out=ok, v_out=ov, dev_status=st)
    for o, c in ((ok, kc), (ov, vc)):
        want = torch.from_numpy(I.values(c.rows[slots], c.scales[slots]).astype(np.float32)).to(o.dtype)
        want[slots < 0] = 5.0
        assert torch.equal(o.cpu(), want)
    assert bool((out[:, -8:] == 5).all()) and int(st) == 0
    k2, v2 = tq.int8_get_rows(gk, gv, gs)
    assert k2.dtype == torch.float16 and not k2[5].any() and v2.shape == (n, hv, dv)


@pytest.mark.parametrize("n,hk,hv,dk,dv,dtype", [(5000, 8, 8, 128, 128, "float16"), (3001, 3, 1, 80, 256, "bfloat16"),
                                                 (2500, 2, 5, 256, 16, "float32"), (12000, 1, 1, 64, 64, "float16")])
def test_rows_of_large_calls(n, hk, hv, dk, dv, dtype):
    # shares that begin and end anywhere, rows without cells among them
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    rng = np.random.default_rng(n)
    cells = n + 100
    xk, xv = _gpu(_rows(rng, n, hk, dk), dtype), _gpu(_rows(rng, n, hv, dv), dtype)
    slots = rng.permutation(cells)[:n].astype(np.int64)
    slots[::9] = -1
    kc, vc = I.Cache(hk, dk, cells), I.Cache(hv, dv, cells)
    kc.set_rows(_np(xk), slots)
    vc.set_rows(_np(xv), slots)
    gk, gv, gs = tq.Int8Cache(hk, dk, cells), tq.Int8Cache(hv, dv, cells), _gpu(slots)
    tq.int8_set_rows(gk, gv, xk, xv, gs)
    out = tq.int8_get_rows(gk, gv, gs, k_out=torch.full_like(xk, 5.0), v_out=torch.full_like(xv, 5.0))
    for g, c, o in ((gk, kc, out[0]), (gv, vc, out[1])):
        assert np.array_equal(g.rows.cpu().numpy(), c.rows)
        assert np.array_equal(g.scales.cpu().numpy().view(np.int16), c.scales.view(np.int16))
        want = torch.from_numpy(I.values(c.rows[slots], c.scales[slots]).astype(np.float32)).to(o.dtype)
        want[slots < 0] = 5.0
        assert torch.equal(o.cpu(), want)


def test_every_scale():
    # rows whose scale is each binary16 number from 2^-16 on: the codes' quotients are the correctly rounded ones
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    s = np.arange(0x0100, 0x7c00, dtype=np.uint16).view(np.float16).astype(np.float32)
    rng = np.random.default_rng(1)
    x = (rng.integers(-254, 255, (len(s), 1, 32)) / 2 + rng.choice([0, 2.0 ** -16, -2.0 ** -16], (len(s), 1, 32))) * s[:, None, None]
    x = x.astype(np.float32)                                 # codes' borders, and just beside them
    x[:, :, 3] = 127 * s[:, None]
    c = I.Cache(1, 32, len(s))
    c.set_rows(x, np.arange(len(s)))
    g, h = tq.Int8Cache(1, 32, len(s)), tq.Int8Cache(1, 32, len(s))
    tq.int8_set_rows(g, h, _gpu(x), _gpu(x), torch.arange(len(s), device="cuda"))
    assert np.array_equal(g.scales.cpu().numpy().view(np.int16), c.scales.view(np.int16))
    assert np.array_equal(g.rows.cpu().numpy(), c.rows)


def test_rows_out_of_range_and_special_values():
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    rng = np.random.default_rng(8)
    x = _rows(rng, 9, 2, 64)
    x[0, 0, 5], x[1, 1, 0], x[2, 0, 63] = np.nan, np.inf, -np.inf
    x[3] = np.nan
    x[4] *= 1e-8                                             # scales in binary16's subnormal range, and 0
    x[5] *= 1e-6
    x[6] *= 1e30                                             # beyond what a scale can say
    x[7] *= 3e-7
    slots = np.array([3, 4, 5, 6, 7, 8, 9, 10, 99], np.int64)
    kc, vc = I.Cache(2, 64, 50), I.Cache(2, 64, 50)
    for c in (kc, vc):
        c.set_rows(x, slots)
    gk, gv = tq.Int8Cache(2, 64, 50), tq.Int8Cache(2, 64, 50)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tq.int8_set_rows(gk, gv, _gpu(x), _gpu(x), _gpu(slots), dev_status=st)
    assert int(st) == 6
    for g, c in ((gk, kc), (gv, vc)):
        assert np.array_equal(g.rows.cpu().numpy(), c.rows)
        assert np.array_equal(g.scales.cpu().numpy().view(np.int16), c.scales.view(np.int16))
    st.zero_()
    k, _ = tq.int8_get_rows(gk, gv, _gpu(slots), dev_status=st)
    assert int(st) == 6 and not k[8].any()


def test_rows_past_32_bit_offsets():
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    cells = (1 << 32) // (8 * 128) + 1000                    # the planes' last rows begin beyond 2^32 bytes
    k, v = tq.Int8Cache(8, 128, cells), tq.Int8Cache(1, 16, cells)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, y = torch.randn((40, 8, 128), generator=g, device="cuda"), torch.randn((40, 1, 16), generator=g, device="cuda")
    slots = torch.arange(cells - 40, cells, device="cuda")
    tq.int8_set_rows(k, v, x, y, slots)
    c, s = I.quantise(x.cpu().numpy())
    assert np.array_equal(k.rows[-40:].cpu().numpy(), c) and not k.rows[:40].any()
    a, b = tq.int8_get_rows(k, v, slots, dtype=torch.float32)
    assert np.array_equal(a.cpu().numpy(), I.values(c, s).astype(np.float32))
    # and decode from there, through pages and through single cells
    q = torch.randn((1, 16, 128), generator=g, device="cuda").half()
    kv = tq.Int8Cache(8, 128, cells)
    kv.rows[-40:], kv.scales[-40:] = k.rows[-40:], k.scales[-40:]
    one = slots.to(torch.int32)[None].contiguous()
    got = tq.int8_decode(k, kv, one, torch.tensor([40], dtype=torch.int32, device="cuda"), q)
    oc = I.Cache(8, 128, 40)
    oc.rows[:], oc.scales[:] = c, s
    ref, bound = I.attention(oc, oc, [np.arange(40)], [40], 1, _np(q), 128 ** -0.5, 22)
    _check(got, ref, bound, "float16")


# ---------------------------------------------------------------- a step's rows

@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("layout,dk,dv,rot,norm", [("half", 128, 128, 128, False), ("half", 128, 64, 64, True),
                                                   ("interleaved", 80, 96, 40, False), ("half", 80, 80, 20, True),
                                                   ("interleaved", 256, 128, 256, True), ("half", 16, 16, 16, False)])
def test_rope_set_rows(dtype, layout, dk, dv, rot, norm):
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    rng = np.random.default_rng(dk + rot)
    n, hq, hk, hv, cells = 90, 6, 3, 3, 300
    rope = tq.Rope(rot, 10000.0, layout=layout, magnitude=1.1)
    q, k, v = (_gpu(_rows(rng, n, h, d), dtype) for h, d in ((hq, dk), (hk, dk), (hv, dv)))
    k[7] = 0.0
    wq, wk = ((_gpu(1 + rng.random(dk).astype(np.float32)) if norm else None) for _ in range(2))
    pos = rng.integers(0, 40000, n).astype(np.int32)
    slots = rng.permutation(cells)[:n].astype(np.int64)
    pos[4], slots[6], pos[-1], slots[-1] = -1, -1, -1, -1     # row 4 without a position, 6 without a cell
    gp, gs = _gpu(pos), _gpu(slots)
    kc, vc = tq.Int8Cache(hk, dk, cells), tq.Int8Cache(hv, dv, cells)
    kc.rows.fill_(3)
    q_out = torch.full_like(q, 7.0)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    more = dict(q_norm=wq, k_norm=wk, eps=1e-5)
    assert tq.int8_rope_set_rows(kc, vc, rope, gp, q, k, v, gs, q_out=q_out, dev_status=st, **more) is q_out
    assert int(st) == 0
    # the queries are rope_rows', the values int8_set_rows', bit for bit
    assert torch.equal(q_out, tq.rope_rows(rope, gp, q, q_norm=wq, eps=1e-5, q_out=torch.full_like(q, 7.0)))
    live = (pos >= 0) & (slots >= 0)
    k2, v2 = tq.Int8Cache(hk, dk, cells), tq.Int8Cache(hv, dv, cells)
    tq.int8_set_rows(k2, v2, k, v, torch.where(gp >= 0, gs, torch.full_like(gs, -1)))
    assert torch.equal(vc.rows, v2.rows) and torch.equal(vc.scales, v2.scales)
    # the keys: codes of the exact rows, but next to a border between two codes or two scales
    w = None if wk is None else _np(wk)
    y = I.turned(_np(k), pos, rope.frequencies, layout, np.float32(rope.magnitude), w, 1e-5)[live]
    step = np.abs(y).max(-1, keepdims=True) / 127
    scale = kc.scales[gs][live].cpu().numpy().astype(np.float64)[..., None]
    assert np.all(np.abs(scale - step) <= 2.0 ** -11 * step * (1 + 2.0 ** -9) + 2.0 ** -25)
    code = kc.rows[gs][live].cpu().numpy().astype(np.float64)
    far = np.abs(code - y / np.where(scale > 0, scale, 1.0))
    assert np.all(far <= 0.5 + 127 * 2.0 ** -18) and not code[scale[..., 0] == 0].any()
    off = np.rint(y / np.where(scale > 0, scale, 1.0)) != code
    assert off.mean() <= 4 * 127 * 2.0 ** -18                 # (a border is met within 2^-18 of the row's largest)
    others = np.ones(cells, bool)
    others[slots[live]] = False
    assert bool((kc.rows[_gpu(others)] == 3).all())
    # without queries, and in place
    k3, v3 = tq.Int8Cache(hk, dk, cells), tq.Int8Cache(hv, dv, cells)
    assert tq.int8_rope_set_rows(k3, v3, rope, gp, None, k, v, gs, k_norm=wk, eps=1e-5) is None
    assert torch.equal(k3.scales, kc.scales) and torch.equal(k3.rows[gs[_gpu(live)]], kc.rows[gs[_gpu(live)]])
    z = q.clone()
    tq.int8_rope_set_rows(k3, v3, rope, gp, z, k, v, gs, q_out=z, **more)
    assert torch.equal(z[pos >= 0], q_out[pos >= 0]) and torch.equal(z[pos < 0], q[pos < 0])


@pytest.mark.parametrize("hq,hk,d,dv,rot,layout,dtype", [(32, 8, 128, 128, 128, "half", "bfloat16"),
                                                         (9, 3, 80, 64, 20, "half", "float16"),
                                                         (4, 1, 64, 256, 32, "interleaved", "float32")])
def test_rope_set_rows_of_large_calls(hq, hk, d, dv, rot, layout, dtype):
    # a large call's rows are those of single ones, bit for bit
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    g = torch.Generator(device="cuda").manual_seed(d)
    n, cells = 3333, 4000
    rope = tq.Rope(rot, layout=layout)
    q, k, v = (torch.randn((n, h, e), generator=g, device="cuda").to(getattr(torch, dtype)) for h, e in ((hq, d), (hk, d), (hk, dv)))
    norm = 1 + 0.1 * torch.randn((d,), generator=g, device="cuda")
    pos = torch.randint(0, 100000, (n,), generator=g, device="cuda", dtype=torch.int32)
    slots = torch.randperm(cells, generator=g, device="cuda")[:n]
    pos[5::11], slots[7::13] = -1, -1
    kc, vc = tq.Int8Cache(hk, d, cells), tq.Int8Cache(hk, dv, cells)
    out = tq.int8_rope_set_rows(kc, vc, rope, pos, q, k, v, slots, q_norm=norm, k_norm=norm)
    k1, v1 = tq.Int8Cache(hk, d, cells), tq.Int8Cache(hk, dv, cells)
    alone = torch.zeros_like(q)
    for i in range(0, n, 101):
        one = slice(i, i + 7)
        alone[one] = tq.int8_rope_set_rows(k1, v1, rope, pos[one], q[one], k[one], v[one], slots[one], q_norm=norm, k_norm=norm)
        assert torch.equal(out[one], alone[one])
        at = slots[one][(slots[one] >= 0) & (pos[one] >= 0)]
        for x, y in ((kc, k1), (vc, v1)):
            assert torch.equal(x.rows[at], y.rows[at]) and torch.equal(x.scales[at], y.scales[at])
    live = (pos >= 0) & (slots >= 0)
    held = torch.zeros(cells, dtype=torch.bool, device="cuda")
    held[slots[live]] = True
    assert bool(vc.rows[held].any(-1).any(-1).all()) and not vc.rows[~held].any() and not kc.rows[~held].any()
    assert not out[pos < 0].any()


def test_rope_set_rows_bad_slots_and_positions():
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    x = torch.ones((3, 2, 32), device="cuda")
    for pos, slots in (([0, 1, -5], [1, 2, 3]), ([0, 1, 2], [1, 2, 40]), ([0, 1, 2], [1, 2, -3])):
        kc, vc = tq.Int8Cache(2, 32, 40), tq.Int8Cache(2, 32, 40)
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        q = tq.int8_rope_set_rows(kc, vc, tq.Rope(32), torch.tensor(pos, dtype=torch.int32, device="cuda"), x, x, x,
                                  torch.tensor(slots, device="cuda"), dev_status=st)
        assert int(st) == 6 and bool(vc.rows[1:3].all()) and not vc.rows[3:].any() and not kc.rows[3:].any()
        assert bool(q[2].any()) == (pos[2] >= 0)


# ---------------------------------------------------------------- decode

def _check(out, ref, bound, dtype):
    got = _np(out)
    assert got.shape == ref.shape
    tol = HALF[dtype] * (np.abs(ref) + bound) + bound + TINY[dtype] + 1e-30
    if dtype == "float16":
        # binary16 rounds numbers from 65520 on to infinity: there is no finite result to be near to
        over = np.isinf(got) & (np.sign(got) == np.sign(ref)) & (np.abs(ref) + bound >= 65520)
        assert not np.any(np.abs(ref) - bound >= 65520, where=~over)
        got = np.where(over, ref, got)
    assert np.all(np.isfinite(got))
    worst = float(np.max(np.abs(got - ref) / tol, initial=0.0))
    assert worst <= 1.0, f"{worst:.2f} times the tolerance"


class Batch:
    """Caches filled for sequences of `lens` cells; other cells hold NaN scales and random codes."""

    def __init__(self, seed, lens, hkv, dk, dv, page, spare=2, v_gain=1.0, k_gain=1.0, extra_cells=0):
        rng = np.random.default_rng(seed)
        self.rng, self.lens, self.page = rng, list(lens), page
        need = [-(-n // page) for n in lens]
        pool = sum(need) + spare
        perm = rng.permutation(pool)
        self.table = np.full((len(lens), max(need + [1]) + 1), 0x7ffffff0, np.int32)
        at = 0
        self.k, self.v = I.Cache(hkv, dk, pool * page + extra_cells), I.Cache(hkv, dv, pool * page + extra_cells)
        for c in (self.k, self.v):
            c.rows[:] = rng.integers(-128, 128, c.rows.shape, dtype=np.int8)
            c.scales[:] = np.nan
        for s, n in enumerate(lens):
            self.table[s, :need[s]] = perm[at:at + need[s]]
            at += need[s]
            t = np.arange(n)
            slots = self.table[s][t // page].astype(np.int64) * page + t % page
            self.k.set_rows(k_gain * _rows(rng, n, hkv, dk), slots)
            self.v.set_rows(v_gain * _rows(rng, n, hkv, dv), slots)
        self.gk, self.gv = _upload(self.k), _upload(self.v)
        self.gt = _gpu(self.table)
        self.gl = _gpu(np.array(self.lens, np.int32))

    def query(self, heads, dtype, gain=1.0):
        return _gpu(gain * _rows(self.rng, len(self.lens), heads, self.k.head_dim), dtype)

    def check(self, out, q, scale, dtype, lens=None, table=None):
        ref, bound = I.attention(self.k, self.v, self.table if table is None else table,
                                 self.lens if lens is None else lens, self.page, _np(q), scale,
                                 22 if dtype == "float16" else 11)
        _check(out, ref, bound, dtype)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("dk,dv,hkv,group,page", [(64, 64, 2, 1, 16), (128, 128, 2, 4, 16), (128, 128, 1, 7, 1),
                                                  (128, 128, 8, 8, 64), (80, 96, 3, 2, 4), (192, 128, 2, 4, 32),
                                                  (256, 256, 1, 16, 1), (256, 240, 2, 3, 256), (128, 112, 1, 33, 2),
                                                  (16, 64, 5, 12, 8), (144, 256, 3, 9, 1), (64, 48, 1, 16, 128)])
def test_decode(dtype, dk, dv, hkv, group, page):
    import quantized_kv_cache_tq_gb300 as tq
    lens = [1, 0, 300, 17, 64, 129, 1000, 0, 15]
    b = Batch(dk + group, lens, hkv, dk, dv, page)
    q = b.query(hkv * group, dtype)
    out = tq.int8_decode(b.gk, b.gv, b.gt, b.gl, q, 0.7 * dk ** -0.5, page_size=page)
    b.check(out, q, 0.7 * dk ** -0.5, dtype)
    assert not out[1].any() and not out[7].any()


@pytest.mark.parametrize("group", [1, 8, 9, 20])
@pytest.mark.parametrize("page", [1, 16, 64])
@pytest.mark.parametrize("dk,dv", [(80, 80), (96, 96), (96, 80), (80, 96), (112, 80), (160, 128), (192, 96), (192, 112),
                                   (208, 128), (144, 144)])
def test_decode_widths(dk, dv, page, group):
    # rows that fill their kernel's width, or end before it; items alone and shared, one sequence of two pages' odd ends
    import quantized_kv_cache_tq_gb300 as tq
    b = Batch(dk + 3 * dv + group, [700, 0, 33, 2, 513], 2, dk, dv, page)
    for dtype in ("bfloat16", "float16"):
        q = b.query(2 * group, dtype)
        b.check(tq.int8_decode(b.gk, b.gv, b.gt, b.gl, q, dk ** -0.5, page_size=page), q, dk ** -0.5, dtype)


@pytest.mark.parametrize("n_seq,length", [(1, 1), (1, 15), (1, 16), (1, 4097), (1, 40000), (3, 9000), (300, 40), (700, 1)])
def test_decode_splits(n_seq, length):
    import quantized_kv_cache_tq_gb300 as tq
    rng = np.random.default_rng(length)
    lens = [length] + [int(x) for x in rng.integers(0, length + 1, n_seq - 1)]
    b = Batch(length, lens, 1, 64, 64, 16)
    q = b.query(2, "float16")
    b.check(tq.int8_decode(b.gk, b.gv, b.gt, b.gl, q, 0.125, page_size=16), q, 0.125, "float16")


@pytest.mark.parametrize("lens", [[511], [512], [513], [576, 0, 512], [577, 65], [64] * 31 + [640], [130] * 32,
                                  [130] * 33, [0] * 32, [0] * 40, [0] * 33 + [1], [700] + [0] * 254 + [3],
                                  [5] * 256 + [900]])
def test_decode_at_the_edges_of_the_split(lens):
    # sequences that one CTA takes alone or several share, batches laid out by a warp, a CTA or in turns
    import quantized_kv_cache_tq_gb300 as tq
    for d, page in ((64, 16), (128, 1)):
        b = Batch(len(lens) + lens[0] + d, lens, 2, d, d, page)
        q = b.query(4, "float16")
        b.check(tq.int8_decode(b.gk, b.gv, b.gt, b.gl, q, d ** -0.5, page_size=page), q, d ** -0.5, "float16")


@pytest.mark.parametrize("dk,dv,hkv,group,page,dtype", [(128, 128, 8, 4, 32, "bfloat16"), (64, 64, 4, 8, 16, "float16"),
                                                        (128, 128, 4, 12, 1, "float16"), (256, 256, 2, 3, 16, "bfloat16"),
                                                        (192, 128, 6, 2, 8, "float16"), (80, 80, 8, 1, 64, "bfloat16")])
def test_decode_of_batches_that_take_heads_side_by_side(dk, dv, hkv, group, page, dtype):
    # enough work for several heads a CTA, items that many CTAs share, empty sequences among them
    import quantized_kv_cache_tq_gb300 as tq
    rng = np.random.default_rng(dk * group)
    lens = [3000] + [int(x) for x in rng.integers(0, 3000, 30)] + [0, 1, 0, 64, 65] + [int(x) for x in rng.integers(1, 90, 8)]
    if hkv * group < 10:
        lens = lens + lens
    b = Batch(dk, lens, hkv, dk, dv, page)
    q = b.query(hkv * group, dtype)
    out = tq.int8_decode(b.gk, b.gv, b.gt, b.gl, q, dk ** -0.5, page_size=page)
    b.check(out, q, dk ** -0.5, dtype)


@pytest.mark.parametrize("gain", [0.05, 1.0])
def test_decode_error_in_binary16_is_the_outputs_own(gain):
    # weights of 22 bits and exact values leave little but the rounding of the output: 2^-11 / sqrt(3) relative rms of
    # numbers spread over a binade's half steps (at most), and a tenth for the fp32 sums
    import quantized_kv_cache_tq_gb300 as tq
    b = Batch(31, [20000], 2, 128, 128, 16)
    q = b.query(8, "float16", gain)
    out = _np(tq.int8_decode(b.gk, b.gv, b.gt, b.gl, q, 128 ** -0.5, page_size=16))
    ref, _ = I.attention(b.k, b.v, b.table, b.lens, 16, _np(q), 128 ** -0.5, 22)
    assert np.sqrt(((out - ref) ** 2).mean()) <= 1.1 * 2.0 ** -11 / 3 ** 0.5 * np.sqrt((ref ** 2).mean())


@pytest.mark.parametrize("v_gain,k_gain,q_gain,scale", [(1e-6, 1.0, 1.0, 0.1), (2e4, 1.0, 1.0, 0.1), (1.0, 1.0, 1e3, 1e-4),
                                                        (1.0, 1e3, 6e-6, 20.0), (1.0, 1.0, 1.0, -0.2),
                                                        (1.0, 1.0, 1.0, 0.0), (1.0, 1.0, 1.0, 3.0)])
def test_decode_ranges(v_gain, k_gain, q_gain, scale):
    import quantized_kv_cache_tq_gb300 as tq
    for dtype in ("bfloat16", "float16"):
        b = Batch(5, [500, 70], 2, 128, 128, 16, v_gain=v_gain, k_gain=k_gain)
        q = b.query(8, dtype, q_gain)
        b.check(tq.int8_decode(b.gk, b.gv, b.gt, b.gl, q, scale, page_size=16), q, scale, dtype)


def test_decode_value_scales_far_apart():
    # keys of like weight whose value rows are 2^30 apart, in one tile and in different ones
    import quantized_kv_cache_tq_gb300 as tq
    for where in (slice(0, 3), slice(100, 101), slice(5, 200, 2)):
        b = Batch(6, [400], 1, 128, 128, 16, v_gain=1e-5)
        t = np.arange(400)
        cells = b.table[0][t // 16].astype(np.int64) * 16 + t % 16
        b.v.scales[cells[where]] = np.float16(500.0)
        gv = _upload(b.v)
        for dtype in ("bfloat16", "float16"):
            q = b.query(4, dtype, 0.1)
            b.check(tq.int8_decode(b.gk, gv, b.gt, b.gl, q, 0.1, page_size=16), q, 0.1, dtype)


def test_decode_strided_queries_and_given_out():
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    b = Batch(7, [33, 200, 5], 2, 64, 64, 16)
    wide = torch.zeros((3, 8 * 64 + 72), dtype=torch.bfloat16, device="cuda")
    q = wide[:, 72:].unflatten(1, (8, 64))
    q.copy_(b.query(8, "bfloat16"))
    out = torch.full((3, 8, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    ws = tq.workspace(tq.int8_decode_workspace(b.gk, b.gv, 8, 3))
    assert tq.int8_decode(b.gk, b.gv, b.gt, b.gl, q, 0.1, page_size=16, out=out, ws=ws) is out
    b.check(out, q, 0.1, "bfloat16")
    assert torch.equal(out, tq.int8_decode(b.gk, b.gv, b.gt, b.gl, q.contiguous(), 0.1, page_size=16))


@pytest.mark.parametrize("page", [1, 8, 16, 64])
def test_decode_bad_pages_and_lengths_are_reported(page):
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    # (cells behind the last whole page belong to no page)
    b = Batch(8, [100, 100, 100], 1, 64, 64, page, extra_cells=page - 1)
    q = b.query(4, "float16")
    ws = tq.workspace(tq.int8_decode_workspace(b.gk, b.gv, 4, 3))
    status = lambda: tq._lib.tq_workspace_status(ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)  # noqa: E731
    out = tq.int8_decode(b.gk, b.gv, b.gt, b.gl, q, 0.1, page_size=page, ws=ws)
    assert status() == 0
    table = b.table.copy()
    table[0, 0], table[1, 99 // page], table[2, 50 // page] = -1, b.k.n_cells // page, 0x7fffffff
    got = tq.int8_decode(b.gk, b.gv, _gpu(table), b.gl, q, 0.1, page_size=page, ws=ws)
    assert status() == 6
    b.check(got, q, 0.1, "float16", table=table)
    # lengths beyond the table, or negative, are cut to what it holds
    wide = b.table.shape[1] * page
    lens = _gpu(np.array([-4, 100, wide + 1], np.int32))
    table = b.table.copy()
    table[2, 100 // page:] = table[2, 0]
    t = np.arange(100, -(-100 // page) * page)
    cells = b.table[2][t // page].astype(np.int64) * page + t % page
    b.k.scales[cells], b.v.scales[cells] = 1.0, 1.0
    table[2, -(-100 // page) - (1 if 100 % page else 0)] = b.table[2, -(-100 // page) - (1 if 100 % page else 0)]
    gk, gv = _upload(b.k), _upload(b.v)
    got = tq.int8_decode(gk, gv, _gpu(table), lens, q, 0.1, page_size=page, ws=ws)
    assert status() == 6 and not got[0].any() and torch.equal(got[1], out[1])
    b.check(got, q, 0.1, "float16", lens=[0, 100, wide], table=table)


def test_decode_no_sequences():
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    c = tq.Int8Cache(2, 64, 16)
    q = torch.empty((0, 4, 64), dtype=torch.float16, device="cuda")
    z = torch.empty((0, 3), dtype=torch.int32, device="cuda")
    assert tq.int8_decode(c, c, z, z[:, 0].contiguous(), q, page_size=16).shape == (0, 4, 64)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_decode_repeats_bit_for_bit(dtype):
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    b = Batch(9, [5000, 3, 900, 2500, 70], 2, 128, 128, 16)
    q = b.query(8, dtype)
    ws = tq.workspace(tq.int8_decode_workspace(b.gk, b.gv, 8, 5))
    first = tq.int8_decode(b.gk, b.gv, b.gt, b.gl, q, page_size=16, ws=ws)
    for _ in range(20):
        assert torch.equal(first, tq.int8_decode(b.gk, b.gv, b.gt, b.gl, q, page_size=16, ws=ws))


def test_decode_graph_follows_lengths_and_shares_a_workspace():
    # two captured graphs and eager calls of both page caches, one workspace, any order
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    b = Batch(10, [700, 2000, 40], 2, 128, 128, 16)
    c = Batch(11, [3000], 1, 128, 128, 1)
    qb, qc = b.query(8, "bfloat16"), c.query(4, "float16")
    ws = tq.workspace(max(tq.int8_decode_workspace(b.gk, b.gv, 8, 3), tq.int8_decode_workspace(c.gk, c.gv, 4, 1)))
    ob, oc = torch.empty((3, 8, 128), dtype=torch.bfloat16, device="cuda"), torch.empty((1, 4, 128), dtype=torch.float16, device="cuda")
    run_b = lambda: tq.int8_decode(b.gk, b.gv, b.gt, b.gl, qb, page_size=16, out=ob, ws=ws)  # noqa: E731
    run_c = lambda: tq.int8_decode(c.gk, c.gv, c.gt, c.gl, qc, out=oc, ws=ws)  # noqa: E731
    p = tq.Paged4Cache(1, 128, 16, 4)
    p.scales[..., 0] = 1.0
    p.codes.random_(0, 256)
    pt, pl = torch.tensor([[3, 1, 0]], dtype=torch.int32, device="cuda"), torch.tensor([41], dtype=torch.int32, device="cuda")
    run_p = lambda: tq.paged4_decode(p, p, pt, pl, qc, 0.01, ws=ws)  # noqa: E731
    run_b(), run_c()
    want_p = run_p().clone()
    torch.cuda.synchronize()
    graphs = []
    for run in (run_b, run_c):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        graphs.append(g)
    for lens in ([700, 2000, 40], [1, 0, 33], [699, 1, 0], [700, 1999, 17]):
        b.gl.copy_(torch.tensor(lens, dtype=torch.int32))
        c.gl.fill_(lens[1])
        ob.fill_(9), oc.fill_(9)
        for g in graphs + graphs[::-1]:
            g.replay()
        assert torch.equal(run_p(), want_p)
        graphs[0].replay()
        b.check(ob, qb, 128 ** -0.5, "bfloat16", lens=lens)
        c.check(oc, qc, 128 ** -0.5, "float16", lens=[lens[1]])


def test_calls_on_two_streams_at_once():
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    b = Batch(12, [6000, 900], 2, 64, 64, 16)
    q = b.query(8, "float16")
    want = tq.int8_decode(b.gk, b.gv, b.gt, b.gl, q, page_size=16)
    rope = tq.Rope(64)
    pos = torch.arange(2, dtype=torch.int32, device="cuda") + 5
    turned = tq.rope_rows(rope, pos, q)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):                      # workspaces and outputs made for the call's own stream
            got[i].append((tq.int8_decode(b.gk, b.gv, b.gt, b.gl, q, page_size=16, stream=s),
                           tq.rope_rows(rope, pos, q, stream=s)))
    torch.cuda.synchronize()
    for x in got[0] + got[1]:
        assert torch.equal(x[0], want) and torch.equal(x[1], turned)


def test_sequences_that_share_pages():
    import quantized_kv_cache_tq_gb300 as tq
    b = Batch(13, [320, 320, 200], 2, 64, 64, 16)
    b.table[1, :12], b.table[2, :12] = b.table[0, :12], b.table[0, :12]
    q = b.query(4, "bfloat16")
    b.check(tq.int8_decode(b.gk, b.gv, _gpu(b.table), b.gl, q, 0.1, page_size=16), q, 0.1, "bfloat16")


# ---------------------------------------------------------------- together

def test_serving_steps_in_one_captured_graph():
    """Plan -> rows with positions into the cache -> decode, captured once; prompts before it, and prompt attention
    over the same cells afterwards."""
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    rng = np.random.default_rng(21)
    n, hq, hkv, d, page, pages, width, steps = 4, 8, 2, 128, 16, 40, 12, 5
    rope = tq.Rope(d, 10000.0, scaling="rotations", factor=4.0, original_len=64.0, beta_fast=8.0)
    kc, vc = tq.Int8Cache(hkv, d, pages * page), tq.Int8Cache(hkv, d, pages * page)
    table = torch.zeros((n, width), dtype=torch.int32, device="cuda")
    free = torch.randperm(pages, device="cuda").to(torch.int32)
    count = torch.tensor([pages], dtype=torch.int32, device="cuda")
    lens = torch.zeros(n, dtype=torch.int32, device="cuda")
    history = [[] for _ in range(n)]                          # (k, v) rows of each sequence, as projected

    def project(rows, counts):
        x = _rows(rng, rows, hq + 2 * hkv, d)
        at = 0
        for s, c in enumerate(counts):
            history[s] += list(x[at:at + c])
            at += c
        return x

    def check_rows(s, length):
        """The sequence's cells stand for its whole history, turned: half a code, the scale's rounding, fp32."""
        h, p = np.array(history[s])[:length], np.arange(length)
        slots = table[s].long().cpu().numpy()[p // page] * page + p % page
        k, v = (_np(t) for t in tq.int8_get_rows(kc, vc, _gpu(slots), dtype=torch.float32))
        for got, want in ((k, I.turned(h[:, hq:hq + hkv], p, rope.frequencies)), (v, h[:, hq + hkv:])):
            step = np.abs(want).max(-1, keepdims=True) / 127
            assert np.all(np.abs(got - want) <= step * (0.5 + 127 * (2.0 ** -11 + 2.0 ** -18)))

    def down(c):
        o = I.Cache(hkv, d, pages * page)
        o.rows[:], o.scales[:] = c.rows.cpu().numpy(), c.scales.cpu().numpy()
        return o

    # prompts
    prompts = [37, 5, 16, 60]
    rows = sum(prompts) + 10
    plan = tq.page_plan(lens, torch.tensor(prompts, dtype=torch.int32, device="cuda"), page, table, free, count,
                        n_rows=rows, in_place=True)
    x = np.zeros((rows, hq + 2 * hkv, d), np.float32)
    x[:sum(prompts)] = project(sum(prompts), prompts)
    gx = _gpu(x, "float16")
    for s in range(n):
        history[s] = [r.astype(np.float16).astype(np.float32) for r in history[s]]
    q = tq.int8_rope_set_rows(kc, vc, rope, plan.positions, gx[:, :hq], gx[:, hq:hq + hkv], gx[:, hq + hkv:], plan.slots)
    # prompt attention over the cells that the plan named
    cells = plan.slots[:prompts[0]].to(torch.int32).contiguous()
    out = tq.int8_prompt_attn(kc.rows, kc.scales, vc.rows, vc.scales, cells, prompts[0], q[:prompts[0]].contiguous())
    for s in range(n):
        check_rows(s, prompts[s])
    oc, ov = down(kc), down(vc)
    ref, _ = I.attention(oc, ov, [cells.cpu().numpy()], [prompts[0]], 1, _np(q[prompts[0] - 1:prompts[0]]), d ** -0.5, 11)
    assert ((_np(out[-1:]) - ref) ** 2).mean() <= 1e-6 * (ref ** 2).mean()         # (prompt attention's own tolerance)

    # decode steps in one graph
    ones = torch.ones(n, dtype=torch.int32, device="cuda")
    step = tq.PagePlan(n, 8)
    proj = torch.zeros((8, hq + 2 * hkv, d), dtype=torch.float16, device="cuda")
    q_out, att = torch.zeros((8, hq, d), dtype=torch.float16, device="cuda"), torch.zeros((n, hq, d), dtype=torch.float16, device="cuda")
    ws = tq.workspace(tq.int8_decode_workspace(kc, vc, hq, n))

    def one():
        tq.page_plan(lens, ones, page, table, free, count, plan=step, in_place=True)
        tq.int8_rope_set_rows(kc, vc, rope, step.positions, proj[:, :hq], proj[:, hq:hq + hkv], proj[:, hq + hkv:],
                              step.slots, q_out=q_out)
        tq.int8_decode(kc, vc, table, lens, q_out[:n], page_size=page, out=att, ws=ws)

    keep = [t.clone() for t in (lens, table, free, count)]
    one()                                                     # (a first call outside: its changes are taken back)
    for t, u in zip((lens, table, free, count), keep):
        t.copy_(u)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        one()
    for t, u in zip((lens, table, free, count), keep):
        t.copy_(u)
    for i in range(steps):
        x = project(n, [1] * n).astype(np.float16).astype(np.float32)
        for s in range(n):
            history[s][-1] = x[s]
        proj[:n].copy_(_gpu(x, "float16"))
        g.replay()
        assert lens.tolist() == [p + i + 1 for p in prompts]
        now = [p + i + 1 for p in prompts]
        _check_turned(q_out[:n], x[:, :hq], [m - 1 for m in now], rope, "float16")
        ref, bound = I.attention(down(kc), down(vc), table.cpu().numpy(), now, page, _np(q_out[:n]), d ** -0.5, 22)
        _check(att, ref, bound, "float16")
    for s in range(n):
        check_rows(s, prompts[s] + steps)
    assert not q_out[n:].any()


def test_the_turn_step_of_cached_keys():
    """Keys whose cells move to other positions: read back, turned by the difference, written again."""
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    rng = np.random.default_rng(22)
    n, h, d = 40, 2, 64
    rope = tq.Rope(d)
    kc, vc = tq.Int8Cache(h, d, n), tq.Int8Cache(h, d, n)
    x = _gpu(_rows(rng, n, h, d))
    pos, slots = torch.arange(n, dtype=torch.int32, device="cuda") + 100, torch.arange(n, device="cuda")
    tq.int8_rope_set_rows(kc, vc, rope, pos, None, x, x, slots)
    back, _ = tq.int8_get_rows(kc, vc, slots, dtype=torch.float32)
    moved = tq.rope_rows(rope, torch.full_like(pos, 60), back, inverse=True)
    want = I.turned(_np(x), np.arange(n) + 40, rope.frequencies)
    # the codes' half step (and the scale's rounding, 127 2^-11), turned: both of a pair count
    step = np.abs(I.turned(_np(x), np.arange(n) + 100, rope.frequencies)).max(-1, keepdims=True) / 127
    assert np.all(np.abs(_np(moved) - want) <= 2 ** 0.5 * step * (0.5 + 127 * 2.0 ** -11) + 1e-4)
