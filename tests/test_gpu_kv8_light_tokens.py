"""Attention over the 8-bit cache: tokens of little weight, or of small values beside a sub-block of huge ones,
give the output their share, dim by dim."""
import numpy as np
import pytest
import torch

from oracle import kv4 as O4
from oracle import kv8 as O
from tests._gpu import need_gpu

pytestmark = pytest.mark.gpu
SUB = 16


@pytest.fixture(scope="module")
def spec():
    need_gpu()
    from speculative_decoding_verify_step_gb300 import spec
    spec.load_library()
    return spec


def held(x):
    """What a prompt's write holds of x [tokens, hd], and the exponent of each token's sub-block."""
    y = O.held(x)
    e = np.array([O.needed_exp(np.abs(O4.saturate(x[s:s + SUB])).max()) for s in range(0, len(x), SUB)])
    return y, np.repeat(e, SUB)[:len(x)]


def check(spec, q, k, v, grp, W):
    """W rows of grp heads (all rows alike: q [hd]) over a chain behind k, v [tokens, hd]; the last W tokens are the window's."""
    n, hd = k.shape
    q = q.to(torch.float16)
    pages = (n + 63) // 64
    pool = spec.spec_kv8_pool(pages, 1, hd)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").view(1, -1)
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    k16, v16 = (torch.from_numpy(x).to(torch.float16) for x in (k, v))
    spec.spec_kv8_write(k16.view(1, n, 1, hd).cuda(), v16.view(1, n, 1, hd).cuda(), z, table, pool)
    kk, _ = held(k16.double().numpy())
    vv, b = held(v16.double().numpy())
    out = spec.spec_kv8_attention(q.view(1, 1, 1, hd).expand(1, W, grp, hd).contiguous().cuda(), pool, z + (n - W), table, scale=1.0)
    qd = q.double().numpy()
    s = kk @ qd / np.log(2.0)                      # in log2 units
    # fp32 sums of hd exact products, each addition within 2^-23 of the largest partial sum, and the product's rounding
    mag = (np.abs(kk) @ np.abs(qd)).max() / np.log(2.0)
    for j in range(W):
        m = n - W + 1 + j
        p = np.exp2(s[:m] - s[:m].max())
        L = p.sum()
        ref = p @ vv[:m] / L
        share = p @ np.abs(vv[:m]) / L
        # numerator and denominator: the score's error and exp2's; additions in fp32, 16 tokens at once;
        # then the weight's rounding to fp16, half a step
        rel = 2 * ((hd + 2) * 2.0 ** -23 * mag + 2.0 ** -22 + (m / 16 + 64) * 2.0 ** -23) + 2.0 ** -11
        # a weight times 2^b below 2^-25 of the row's largest has fp16's subnormal steps: off by 2^-36 of the largest at
        # most (twice that, as the running maximum may lie a bit above it)
        flush = np.abs(vv[:m] / np.exp2(b[:m, None])).sum(0) * 2.0 ** -35 * np.exp2((s[:m] - s[:m].max() + b[:m]).max()) / L
        tol = share * rel + flush + np.abs(ref) * 2.0 ** -11 + 2.0 ** -25
        got = out[0, j].double().cpu().numpy()
        assert (np.abs(got - ref) <= tol).all(), (j, np.abs(got - ref).max(0)[:3], tol[:3], ref[:3])
    return out


@pytest.mark.parametrize("grp,W", [(1, 1), (4, 5), (8, 8)])
@pytest.mark.parametrize("n,below", [(65520, 25.3), (65520, 30.2), (700, 26.0), (1500, 20.0)])
def test_one_heavy_token_over_many_light_ones(spec, n, below, grp, W):
    """The heavy token's values are zero in every other dim, so those dims are the light tokens' alone."""
    rng = np.random.default_rng(n)
    hd = 64
    q = torch.zeros(hd)
    q[0] = 1.0
    k = rng.normal(size=(n, hd)) * 0.1
    k[:, 0] = -below * np.log(2.0) / 2             # held on e4m3's grid: the test takes what is held
    v = 1.0 + 0.3 * rng.random((n, hd))
    heavy = n // 3
    k[heavy, 0] = below * np.log(2.0) / 2
    v[heavy, ::2] = 0.0
    check(spec, q, k, v, grp, W)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("less", [0.0, 4.0, 8.0])
@pytest.mark.parametrize("n,at", [(8192, 100), (8192, 8100), (300, 0)])
def test_an_attended_outlier_in_one_dim(spec, n, at, less, hd):
    """A value 57344 in one dim of a token that is attended to: the others' values of 0.01, at `less` bits lower
    scores, make the other dims."""
    rng = np.random.default_rng(at)
    q = torch.zeros(hd)
    q[0] = 1.0
    k = rng.normal(size=(n, hd)) * 0.1
    k[:, 0] = 0.0
    k[at, 0] = less * np.log(2.0)
    v = 0.01 * (0.5 + rng.random((n, hd)))
    v[at] = 0.0
    v[at, 5] = 57344.0
    check(spec, q, k, v, 4, 2)


def test_huge_scores_keep_their_ties(spec):
    """Scores whose float steps are 2 to 2^17 log2 units, equal ones in sub-blocks of unlike exponents: each gets
    its share, and nothing overflows."""
    hd, n = 64, 256
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    pool = spec.spec_kv8_pool(4, 1, hd)
    k = torch.full((1, n, 1, hd), 1.0, dtype=torch.float16)
    v = torch.full((1, n, 1, hd), 0.25, dtype=torch.float16)
    ties = [3, 40, 77, 130, 200, 250]
    k[0, ties] = 4.0
    v[0, ties] = torch.tensor([60000.0, 1e-4, 448.0, 57344.0, 28672.0, 3.5]).view(6, 1, 1).to(torch.float16)
    table, z = i32([[2, 0, 3, 1]]), i32([0])
    spec.spec_kv8_write(k.cuda(), v.cuda(), z, table, pool)
    vv = np.stack([O.held(v[0, s:s + SUB, 0].double().numpy()) for s in range(0, n, SUB)]).reshape(n, hd)
    for sign in (1.0, -1.0):
        # keys of 1 are the best with the sign turned, in all sub-blocks
        best = np.array(ties) if sign > 0 else np.setdiff1d(np.arange(n), ties)
        want = vv[best].mean(0)
        for scale in [2.0 ** e for e in range(0, 41, 2)]:
            q = torch.full((1, 1, 4, hd), 2048.0, dtype=torch.float16, device="cuda")
            out = spec.spec_kv8_attention(q, pool, i32([n - 1]), table, scale=sign * scale).double().cpu().numpy()
            # equal scores: equal weights; sums of 256, and the output's rounding
            assert np.abs(out - want).max() <= want.max() * (2.0 ** -11 + 256 * 2.0 ** -23), (sign, scale, out.ravel()[0], want[0])
