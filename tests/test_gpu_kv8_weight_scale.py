"""Tokens' weights of the 8-bit attention where scores are large: a row gives one in all, and equal tokens equal shares."""
import numpy as np
import pytest
import torch

from tests._gpu import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def spec():
    need_gpu()
    from speculative_decoding_verify_step_gb300 import spec
    spec.load_library()
    return spec


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("grp,W", [(1, 1), (4, 2), (4, 3), (4, 16)])
@pytest.mark.parametrize("pages,hint", [(4, 0), (300, 0), (300, 64)])
def test_equal_best_tokens_share_alike(spec, pages, hint, grp, W, sign):
    """Up to 8 rows from kept scores, more from the keys once more; one cluster, and cut groups.  All numbers are powers of two
    (products and sums exact) and the best tokens' scores are equal, so that shares are 1/3 to fp32's roundings: exp2's
    2^-22, those of the sum of three, its inverse and the product, and one for each row that is added up."""
    hd, n = 64, pages * 64
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    pool = spec.spec_kv8_pool(pages, 1, hd)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").view(1, -1)
    k = torch.full((1, n, 1, hd), -sign, dtype=torch.float16, device="cuda")
    best = [7, 90, n - 40]
    k[0, best] = sign
    spec.spec_kv8_write(k, k, i32([0]), table, pool)
    q = torch.full((1, W, grp, hd), 1024.0, dtype=torch.float16, device="cuda")
    for scale in [sign * 2.0 ** e for e in (-16, -4, 0, 1, 4, 6, 8, 9, 10, 11, 12, 15, 20, 30, 40)]:
        weight = torch.zeros(1, 1, n, device="cuda")
        spec.spec_kv8_attention(q, pool, i32([n - W]), table, scale=scale, weight=weight, max_kv_len=hint)
        w = weight[0, 0].double().cpu().numpy()
        rows = W * grp
        if abs(scale) >= 2.0 ** -4:        # the others' scores are 2^13 or more below
            assert np.abs(w[best] - rows / 3).max() <= rows / 3 * (2.0 ** -21 + rows * 2.0 ** -23), (scale, w[best])
            assert np.abs(np.delete(w, best)).max() == 0
        else:
            assert np.abs(w[best] - w[best[0]]).max() == 0
            assert abs(w.sum() - rows) <= rows * (2.0 ** -21 + (rows + n / 64) * 2.0 ** -23)


@pytest.mark.parametrize("W", [2, 8])
def test_rows_add_up_to_one_at_large_scores(spec, W):
    """Random scores of some 10^5: whatever they are, a row's weights add up to one."""
    hd, n, grp = 64, 700, 4
    g = torch.Generator().manual_seed(W)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    pool = spec.spec_kv8_pool(11, 2, hd)
    table = torch.arange(11, dtype=torch.int32, device="cuda").view(1, -1)
    k = torch.randn(1, n, 2, hd, generator=g)
    k[..., 0] = 400.0                       # a common part of all scores
    k[..., 1:] *= 0.02
    k = k.to(torch.float16).cuda()
    spec.spec_kv8_write(k, k, i32([0]), table, pool)
    q = torch.randn(1, W, 2 * grp, hd, generator=g)
    q[..., 0] = 300.0
    weight = torch.zeros(1, 2, n, device="cuda")
    spec.spec_kv8_attention(q.to(torch.float16).cuda(), pool, i32([n - W]), table, scale=1.0, weight=weight)
    got = weight.double().sum(-1).cpu().numpy()
    # exp2 and the products with 1/l: 2^-21 of each weight; sums of n in fp32, 32 at once, then rows
    assert np.abs(got - W * grp).max() <= W * grp * (2.0 ** -21 + (n / 16 + 64 + W * grp) * 2.0 ** -23), got
