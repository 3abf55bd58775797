"""Attention over the 4-bit cache at scores so large that float32 does not hold their differences: all the
weight is on the token of the largest score, and the output is its value.

Bound: half a step of the output, and the weight P s rounded to fp16 (2^-11 of itself) times |c - 7.5| <= 7.5;
the sums have one term each."""
import numpy as np
import pytest
import torch

from oracle import kv4 as O
from tests.test_gpu_kv4 import STEP, Cache, np64, spec_

pytestmark = pytest.mark.gpu


def expect_argmax(got, q, held, n_cached, scale, dtype):
    (k, v), vs = held
    n, Hq, hd = q.shape
    grp = Hq // k.shape[1]
    got = np64(got)
    assert np.isfinite(got).all()
    for h in range(Hq):
        score = q[:, h] @ k[:, h // grp].T * scale                         # [n, keys]
        score = np.where(np.arange(len(k))[None] <= n_cached + np.arange(n)[:, None], score, -np.inf)
        top2 = np.sort(score, -1)[:, -2:]
        bound = np.abs(q[:, h]).sum(-1) * np.abs(k[:, h // grp]).max() * abs(scale)
        assert (top2[:, 1] - top2[:, 0] > 2.0 ** -18 * bound).all() and (top2[:, 1] - top2[:, 0] > 200).all()   # clear of rounding
        at = score.argmax(-1)
        want, s = v[at, h // grp], vs[at, h // grp]
        assert (np.abs(got[:, h] - want) <= STEP[dtype] * np.abs(want) + 7.5 * 2.0 ** -11 * s + 2.0 ** -20 * (np.abs(want) + 16 * s) + 2.0 ** -25).all()


# lengths, rows, heads: clusters, one CTA, pieces of one warp's pages and of the whole CTA's
SHAPES = [([70, 3], 3, 2, 2, 64), ([60, 130], 7, 1, 4, 128), ([500], 15, 2, 4, 128), ([3000, 900], 3, 2, 4, 128), ([9000], 2, 1, 4, 64),
          ([7000, 64], 10, 1, 4, 128)]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("lens,W,Hkv,grp,hd", SHAPES)
@pytest.mark.parametrize("scale,q_gain", [(2.0 ** 40, 1.0), (-2.0 ** 40, 1.0), (2.0 ** 27, 1.0), (2.0 ** 23, 1.0), (2.0 ** 20, 1.0),
                                          (2.0 ** 40, 8000.0), (1e7, 1000.0)])
def test_all_weight_on_the_largest_score(dtype, lens, W, Hkv, grp, hd, scale, q_gain):
    spec = spec_()
    g = torch.Generator().manual_seed(W + 3)
    c = Cache([n + W for n in lens], Hkv, hd, seed=W)
    held = c.fill(sum(lens) + W + 1)
    q = torch.empty(len(lens), W, Hkv * grp, hd, dtype=dtype)
    for b, n in enumerate(lens):                             # queries with a clear winner: near one of the keys they see
        (k, _), _ = held[b]
        for h in range(Hkv * grp):
            for j in range(W):
                unit = torch.from_numpy(k[:n + j + 1, h // grp])
                pick = int(torch.argmax((unit ** 2).sum(-1))) if (h + j) % 3 == 0 else int(torch.randint(n + j + 1, (1,), generator=g))
                x = unit[pick] * (1 if scale > 0 else -1)
                mean = unit.mean(0)
                x = x - (x @ mean) / max(float(mean @ mean), 1e-9) * mean * 0.5
                q[b, j, h] = (q_gain * x / x.abs().max()).to(dtype)
    kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for hint in (0, max(lens)):
        got = spec.spec_kv4_attention(q.cuda(), c.pool, kv_len, c.table, scale=scale, max_kv_len=hint)
        for b, n in enumerate(lens):
            expect_argmax(got[b], np64(q[b]), held[b], n, scale, dtype)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n,W", [(40, 1), (300, 4), (5000, 4), (5000, 12)])
def test_infinite_queries_and_keys(dtype, n, W):
    """Saturated on both sides: the token whose infinity meets the query's is the one attended to."""
    spec = spec_()
    hd = 128
    g = torch.Generator().manual_seed(n)
    k, v = (torch.randn(1, n + W, 1, hd, generator=g).to(dtype) for _ in range(2))
    q = torch.randn(1, W, 2, hd, generator=g).to(dtype)
    k[0, n // 3, 0, 5], q[0, :, :, 5] = float("inf"), float("inf")
    k[0, n // 2, 0, 5] = float("-inf")
    c = Cache([n + W], 1, hd)
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    spec.spec_kv4_write(k.cuda(), v.cuda(), z, c.table, c.pool)
    held = ((O.held(np64(k[0])), O.held(np64(v[0]))), O.quantise(np64(v[0]))[1])
    got = spec.spec_kv4_attention(q.cuda(), c.pool, z + n, c.table)
    expect_argmax(got[0], O.saturate(np64(q[0])), held, n, hd ** -0.5, dtype)
