"""Attention over the 4-bit cache beside V cells of a huge scale that a row does not see, or hardly weighs.

Bound of a row's error, derived from the keys the row sees alone: half a step of the output; each weight P s
rounded to fp16, 2^-11 of itself or, subnormal, 2^-25 of the row's largest P s (which is at least 1 in the
units of the rounding), times |c - 7.5| <= 7.5; the scores' and sums' error as in test_gpu_kv4.py."""
import numpy as np
import pytest
import torch

from oracle import kv4 as O
from tests.test_gpu_kv4 import STEP, Cache, check, np64, spec_

pytestmark = pytest.mark.gpu


def rows_ref(q, k, v, vs, n_cached, parent=None, dtype=torch.float16):
    """Oracle output of one window [n, Hq, hd] over held k, v [keys, Hkv, hd] (V's scales vs [keys, Hkv]) and the bound."""
    out, probs = O.attention(q, k, v, n_cached, parent)
    n, Hq, hd = q.shape
    grp = Hq // k.shape[1]
    tol = STEP[dtype] * np.abs(out) + 2.0 ** -25
    for h, p in enumerate(probs):                            # [grp, n, keys]
        ps = p * vs[:, h]
        rnd = 7.5 * (2.0 ** -11 * ps.sum(-1) + 2.0 ** -25 * ps.max(-1) * (p > 0).sum(-1))
        mag = np.einsum("ngd,kd->gnk", np.abs(q[:, h * grp:(h + 1) * grp]), np.abs(k[:, h]) + 16 * np.abs(k[:, h]).max(-1, keepdims=True))
        e = 2.0 ** -22 * hd ** -0.5 * np.where(p > 2.0 ** -60, mag, 0).max(-1) + 2.0 ** -21
        dev = np.einsum("gnk,kd->gnd", p, np.abs(v[:, h])) + np.abs(np.einsum("gnk,kd->gnd", p, v[:, h]))
        tol[:, h * grp:(h + 1) * grp] += np.moveaxis(rnd[..., None] + 2 * e[..., None] * dev, 0, 1)
    return out, tol


def window(lens, W, Hkv, grp, hd, v_gain, dtype, seed=0):
    """Queries near one direction, K around zero, V of size v_gain."""
    g = torch.Generator().manual_seed(seed)
    way = torch.randn(Hkv, 1, hd, generator=g).sign()
    q = (0.3 * torch.randn(len(lens), W, Hkv, grp, hd, generator=g) + way).flatten(2, 3).to(dtype)
    n = max(lens) + W
    k = (0.5 * torch.randn(len(lens), n, Hkv, hd, generator=g)).to(dtype)
    v = (v_gain * torch.randn(len(lens), n, Hkv, hd, generator=g)).to(dtype)
    return q, k, v, way.squeeze(1)


def run(q, k, v, lens, W, parent, dtype, hint):
    spec = spec_()
    Hkv, hd = k.shape[2:]
    c = Cache([n + W for n in lens], Hkv, hd, seed=W)
    off = np.concatenate([[0], np.cumsum([n + W for n in lens])])
    flat = [torch.cat([x[b, :n + W] for b, n in enumerate(lens)]) for x in (k, v)]
    zero = torch.zeros(len(lens), dtype=torch.int32, device="cuda")
    spec.spec_kv4_write(flat[0].cuda(), flat[1].cuda(), zero, c.table, c.pool, row_off=torch.tensor(off, dtype=torch.int32, device="cuda"))
    got = spec.spec_kv4_attention(q.cuda(), c.pool, torch.tensor(lens, dtype=torch.int32, device="cuda"), c.table, parent=parent, max_kv_len=hint)
    return got, [(O.held(np64(k[b, :n + W])), O.held(np64(v[b, :n + W])), O.quantise(np64(v[b, :n + W]))[1][..., 0]) for b, n in enumerate(lens)]


# lengths, rows, heads: clusters, one CTA, pieces of one warp's pages and of the whole CTA's
SHAPES = [([70, 3], 3, 2, 2, 64), ([60, 130], 7, 1, 4, 128), ([500], 15, 2, 4, 128), ([3000, 900], 3, 2, 4, 128),
          ([9000], 2, 1, 4, 64), ([7000, 64], 10, 1, 4, 128)]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("lens,W,Hkv,grp,hd", SHAPES)
@pytest.mark.parametrize("what", ["hidden", "weightless", "both"])
def test_a_huge_value_that_has_no_weight_costs_nothing(dtype, lens, W, Hkv, grp, hd, what):
    """hidden: the values of a tree's first branch span +-65504, which the second branch's rows do not see;
    weightless: so do those of a cached token whose score is far below the others'."""
    if W < 3 and what != "weightless":
        pytest.skip("no second branch")
    q, k, v, way = window(lens, W, Hkv, grp, hd, 2e-3, dtype, seed=W)
    parent = None
    huge = torch.tensor([65504.0, -65504.0]).repeat(hd // 2).to(dtype)
    if what != "weightless":
        parent = [-1, 0, 0] + [(j - 1) // 2 for j in range(3, W)]
        for b, n in enumerate(lens):
            v[b, n + 1] = huge
    if what != "hidden":
        for b, n in enumerate(lens):
            v[b, n // 2], k[b, n // 2] = huge, (-30 * way).to(dtype)
    for hint in (0, max(lens)):
        got, held = run(q, k, v, lens, W, parent, dtype, hint)
        for b, n in enumerate(lens):
            check(got[b], *rows_ref(np64(q[b]), *held[b], n, parent, dtype))


@pytest.mark.parametrize("lens,W,Hkv,grp,hd", [s for s in SHAPES if s[1] > 2])
def test_rows_do_not_depend_on_cells_they_do_not_see(lens, W, Hkv, grp, hd):
    """Bit for bit: the second branch's rows, whatever the first branch's K and V."""
    parent = [-1, 0, 0] + [2] * (W - 3)
    q, k, v, _ = window(lens, W, Hkv, grp, hd, 1.0, torch.float16, seed=W + 1)
    a, _ = run(q, k, v, lens, W, parent, torch.float16, max(lens))
    for b, n in enumerate(lens):
        k[b, n + 1], v[b, n + 1] = 65504, -65504
        v[b, n + 1, :, ::2] = 65504
    z, _ = run(q, k, v, lens, W, parent, torch.float16, max(lens))
    keep = [j for j in range(W) if j != 1]
    assert torch.equal(a[:, keep], z[:, keep]) and not torch.equal(a[:, 1], z[:, 1])


@pytest.mark.parametrize("W,grp", [(1, 4), (4, 4), (8, 8)])
def test_scales_from_subnormal_to_the_largest(W, grp):
    """Tokens whose V scales span 2^-24 to 2^13, and some without spread, the smallest with the highest scores."""
    n, Hkv, hd = 700, 2, 128
    q, k, v, way = window([n], W, Hkv, grp, hd, 1.0, torch.float16, seed=5)
    e = torch.linspace(-24, 13, n + W)[torch.randperm(n + W, generator=torch.Generator().manual_seed(1))]
    v = (v.clamp(-3.9, 3.9) * 2.0 ** e.view(1, -1, 1, 1)).clamp(-65504, 65504)
    v[0, ::17] = 2.0 ** -3
    k = k.float() + (5 - e).view(1, -1, 1, 1) * way * (0.35 * hd ** -0.5)
    got, held = run(q, k.half(), v.half(), [n], W, None, torch.float16, 0)
    check(got[0], *rows_ref(np64(q[0]), *held[0], n))
