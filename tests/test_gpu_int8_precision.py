"""How many bits the int8 cache's calls and rotations keep: inputs on which one
rounding too many, or a number that runs out of range, shows in the result."""
import numpy as np
import pytest

from oracle import int8 as I
from tests.test_gpu_int8_cache import _check_turned

pytestmark = pytest.mark.gpu

HALF = {"float32": 2.0 ** -24, "float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _gpu(x, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(getattr(torch, dtype))


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("nats", [14.0, 16.3, 18.0])
def test_decode_faint_keys_beside_a_heavy_one(dtype, nats, first):
    """One key `nats` above 100000 equal ones, ahead of them or behind: where its values are zero, theirs alone are the
    result, however small their weights are.  So many sequences that a warp has half of one's keys."""
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    n, n_seq, h, d = 100001, 304, 4, 64
    rng = np.random.default_rng(7)
    k, v = I.Cache(h, d, n), I.Cache(h, d, n)
    k.rows[:, :, 0], k.scales[:] = 1, 2.0 ** -7
    v.rows[:], v.scales[:] = rng.integers(20, 127, v.rows.shape), 0.01
    k.rows[0, :, 0], v.rows[0, :, :d // 2] = 127, 0
    q = np.zeros((1, h, d))
    q[..., 0] = 1.0
    scale = nats * 128 / 126
    ref, bound = I.attention(k, v, [np.arange(n)], [n], 1, q, scale, 22 if dtype == "float16" else 11)
    gk, gv = (tq.Int8Cache.from_planes(_gpu(c.rows), _gpu(c.scales)) for c in (k, v))
    cells = torch.arange(n, dtype=torch.int32, device="cuda")
    table = (cells if first else cells.flip(0)).expand(n_seq, n).contiguous()
    lens = torch.full((n_seq,), n, dtype=torch.int32, device="cuda")
    out = _np(tq.int8_decode(gk, gv, table, lens, _gpu(q, dtype).expand(n_seq, h, d).contiguous(), scale))
    # Beyond what `bound` counts: it takes 2^11 roundings in a row, but a warp has half of the keys here.  Its products
    # add 16 keys at a time (binary16 results twice, the weights being in two parts), each sum cut by up to 2^-23 of
    # itself, that is 2^-24 of the last one in the mean of a sum that grows evenly; its weights are summed 4 at a time
    # in each of 8 lanes, every sum rounded by up to 2^-24.
    steps = n / 2 / 16 * (2 if dtype == "float16" else 1) + n / 2 / 32
    bound = bound + steps * 2.0 ** -24 * np.abs(ref)
    tol = HALF[dtype] * (np.abs(ref) + bound) + bound
    worst = (np.abs(out - ref) / tol).max()
    assert worst <= 1.0, f"{worst:.2f} times the tolerance, in the mean {(out / ref - 1).mean():+.1e}"


@pytest.mark.parametrize("dk,dv,group", [(128, 128, 4), (64, 64, 8), (128, 128, 16), (256, 256, 2)])
def test_decode_in_bfloat16_is_the_exact_result_rounded(dk, dv, group):
    """A result off by e rounds to another number with probability 2 e / step, and a step of bfloat16 is at least 2^-8 of
    the number.  fp32 arithmetic and weights of 22 bits leave e at 2^-20 or so: 2^-11 of the results, and a few times
    that for results near zero.  Weights of 11 bits, 2^-13 in the mean and independent: 2^-4."""
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    rng = np.random.default_rng(dk + group)
    lens, hkv = [700, 3000, 9000], 2
    k, v = I.Cache(hkv, dk, sum(lens)), I.Cache(hkv, dv, sum(lens))
    for c in (k, v):
        c.set_rows(rng.standard_normal((sum(lens), hkv, c.head_dim)), np.arange(sum(lens)))
    table = np.zeros((3, 9000), np.int32)
    at = rng.permutation(sum(lens))
    for s, n in enumerate(lens):
        table[s, :n], at = at[:n], at[n:]
    q = _gpu(rng.standard_normal((3, hkv * group, dk)), "bfloat16")
    gk, gv = (tq.Int8Cache.from_planes(_gpu(c.rows), _gpu(c.scales)) for c in (k, v))
    out = tq.int8_decode(gk, gv, _gpu(table), _gpu(np.array(lens, np.int32)), q)
    ref, _ = I.attention(k, v, table, lens, 1, _np(q), dk ** -0.5, 22)
    want = torch.from_numpy(ref).to(torch.bfloat16)
    off = (out.cpu() != want).double().mean().item()
    assert off <= 2.0 ** -8, f"{off:.2%} of the results"


@pytest.mark.parametrize("layout,d,rot", [("half", 128, 128), ("half", 80, 20), ("interleaved", 96, 48)])
@pytest.mark.parametrize("dtype,gain,eps", [("float32", 1e30, 1e-6), ("float32", 1e19, 0.0), ("float32", 1e-19, 0.0),
                                            ("float32", 1e-30, 0.0), ("float32", 1e-41, 0.0), ("float32", 1e-25, 1e-44),
                                            ("float32", 1e-7, 1e30), ("bfloat16", 1e30, 1e-6), ("bfloat16", 1e-30, 0.0),
                                            ("float16", 5e3, 1e-6), ("float16", 6e-7, 0.0)])
def test_norm_of_rows_whose_squares_leave_the_range(layout, d, rot, dtype, gain, eps):
    # every other row as it mostly is, so that both kinds meet in a warp; tolerances as for those
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    rng = np.random.default_rng(d)
    n, h, eps = 41, 3, float(np.float32(eps))
    rows = rng.standard_normal((n, h, d))
    rows[1::2] *= gain
    x, pos = _gpu(rows.astype(np.float32), dtype), rng.integers(0, 9000, n).astype(np.int32)
    w = 1 + rng.random(d).astype(np.float32)
    rope, gp, gw = tq.Rope(rot, layout=layout), _gpu(pos), _gpu(w)
    y = tq.rope_rows(rope, gp, x, q_norm=gw, eps=eps)
    _check_turned(y, _np(x), pos, rope, dtype, w, eps)
    assert torch.equal(tq.rope_rows(rope, gp[::2].contiguous(), x[::2].contiguous(), q_norm=gw, eps=eps), y[::2])
    # and quantised: scales and codes of the exact rows, but next to a border between two of them
    k, v = tq.Int8Cache(h, d, n), tq.Int8Cache(h, d, n)
    tq.int8_rope_set_rows(k, v, rope, gp, None, x, x, torch.arange(n, device="cuda"), k_norm=gw, eps=eps)
    want = I.turned(_np(x), pos, rope.frequencies, layout, 1.0, w, eps)
    step = np.abs(want).max(-1, keepdims=True) / 127
    scale, code = _np(k.scales)[..., None], k.rows.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(scale - step) <= 2.0 ** -11 * step * (1 + 2.0 ** -9) + 2.0 ** -25)
    exact = np.clip(np.divide(want, scale, where=scale > 0, out=np.zeros_like(want)), -127, 127)
    assert np.all(np.abs(code - exact) <= 0.5 + 127 * 2.0 ** -18)


def test_norm_of_rows_that_are_not_finite_or_zero():
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    x = torch.ones((4, 2, 64), device="cuda")
    x[0, 0, 3], x[1, 1, 5], x[2] = float("inf"), float("nan"), 0.0
    y = tq.rope_rows(tq.Rope(64), torch.zeros(4, dtype=torch.int32, device="cuda"), x,
                     q_norm=torch.ones(64, device="cuda"), eps=0.0)
    assert bool(y[0, 0, 3].isnan()) and not y[0, 0, :3].any() and bool(y[1, 1].isnan().all()) and not y[2].any()
    # (position 0 turns nothing; one root's 2^-22 and two products)
    one = y.new_ones(64) * 1.0
    for row in (y[0, 1], y[1, 0], y[3, 0], y[3, 1]):
        assert bool(((row - one).abs() <= 2.0 ** -21).all())


@pytest.mark.parametrize("layout,d,rot", [("half", 128, 128), ("interleaved", 128, 128), ("half", 80, 20)])
@pytest.mark.parametrize("magnitude", [1.0, 1.2079441547393799])
@pytest.mark.parametrize("inverse", [False, True])
def test_rotations_in_fp32_round_as_little_as_they_can(layout, d, rot, magnitude, inverse):
    """Of N(0, 1) rows at all angles: a result is rounded once and one of its two products once; sine and cosine, each
    rounded once, count as much again as a result.  A rounding of numbers spread evenly over the logarithm is 2.53e-8
    rms (2^-23 / 12^0.5, times the rms of 1 / mantissa, 0.7355), of numbers just above a power of two 3.44e-8:
    2.53e-8 (1 + 1/2 + 1)^0.5 = 4.0e-8, and with sine and cosine reaching into [1, 1.21) 4.63e-8 at most."""
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    rng = np.random.default_rng(rot)
    n, h = 3000 * 128 // rot, 4
    rope = tq.Rope(rot, frequencies=rng.uniform(0.1, 3.0, rot // 2), layout=layout, magnitude=magnitude)
    x, pos = rng.standard_normal((n, h, d)).astype(np.float32), rng.integers(0, 1 << 20, n).astype(np.int32)
    out = _np(tq.rope_rows(rope, _gpu(pos), _gpu(x), inverse=inverse))
    ref = I.turned(x, pos, rope.frequencies, layout, float(np.float32(magnitude)), inverse=inverse)
    first = np.arange(rot // 2) if layout == "half" else np.arange(0, rot, 2)
    for at in (first, first + (rot // 2 if layout == "half" else 1)):
        e = np.sqrt(((out - ref)[..., at] ** 2).mean() / (ref[..., at] ** 2).mean())
        assert e <= (4.0e-8 if magnitude == 1.0 else 4.63e-8), f"{e:.3e}"


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("v_scale", [0x3fff, 0x43ff, 0x03ff, 0x7bff])
@pytest.mark.parametrize("sign", [1, -1])
def test_decode_scores_at_the_end_of_the_range(dtype, v_scale, sign):
    """Scores next to 2^24, growing from key to key by what fp32 resolves there, value scales just below a power of two:
    weights stay finite.  All keys have the same values, so that whatever the weights are, these are the result: weights
    of 22 bits, sums over 40 tiles of a warp at most."""
    import torch
    import quantized_kv_cache_tq_gb300 as tq
    n, h, d = 3000, 2, 64
    rng = np.random.default_rng(3)
    k, v = I.Cache(h, d, n), I.Cache(h, d, n)
    k.rows[:, :, 0], k.rows[:, :, 1], k.scales[:] = 127, (np.arange(n) * 127 // n)[:, None], 1.0
    v.rows[:] = rng.integers(-126, 127, (1, h, d))
    v.rows[:, :, 0] = 127
    v.scales[:] = np.uint16(v_scale).view(np.float16)
    q = torch.zeros((1, 4, d), dtype=getattr(torch, dtype), device="cuda")
    q[..., 0], q[..., 1] = sign, 3e-5
    gk, gv = (tq.Int8Cache.from_planes(_gpu(c.rows), _gpu(c.scales)) for c in (k, v))
    out = tq.int8_decode(gk, gv, torch.arange(n, dtype=torch.int32, device="cuda")[None],
                         torch.tensor([n], dtype=torch.int32, device="cuda"), q, (2.0 ** 24 - 2.0 ** 14) / 127)
    want = I.values(v.rows[0], v.scales[0]).repeat(2, 0)[None]
    over = np.abs(want) >= 65520 if dtype == "float16" else np.zeros_like(want, bool)
    got = _np(out)
    # (a binary16 result has steps of 2^-24 at least)
    tol = (HALF[dtype] + 2.0 ** -13) * np.abs(want) + (2.0 ** -25 if dtype == "float16" else 0.0)
    assert np.all(np.isfinite(got) | over) and np.all((np.abs(got - want) <= tol) | over)
