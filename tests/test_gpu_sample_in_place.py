"""q written over its own logits: the same tokens and the same q as into another tensor."""
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


@pytest.mark.parametrize("rows,V", [(1, 128256), (5, 50257), (40, 33001), (300, 1003)])
def test_q_in_place_of_the_logits(spec, rows, V):
    g = torch.Generator().manual_seed(V)
    x = (3 * torch.randn(rows, V, generator=g)).cuda()
    x[0, 5] = float("nan")
    u = torch.rand(rows, generator=g).cuda()
    for kw in (dict(), dict(temperature=0.0), dict(top_k=20), dict(top_k=700), dict(top_p=0.9), dict(top_k=900, top_p=0.99, min_p=0.001),
               dict(min_p=0.2), dict(top_k=-1)):
        tok, q = spec.spec_sample(x, u, return_probs=True, **kw)
        y, out = x.clone(), torch.empty_like(tok)
        t2, q2 = spec.spec_sample(y, u, outs=(out, y), **kw)
        assert q2 is y and torch.equal(t2, tok) and torch.equal(y, q), kw
