"""How many bits the int8 cache's calls and rotations keep: inputs on which one
rounding too many, or a number that runs out of range, shows in the result."""
import math

import numpy as np
import pytest

from oracle import int8 as I

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
