"""Settings of spec_sample given in other types than the kernel's: they mean what they say."""
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


@pytest.fixture(scope="module")
def logits():
    return torch.randn(3, 5000, generator=torch.Generator().manual_seed(1)).cuda()


LAST = 1.0 - 2.0 ** -24                          # fp32's last number below one


def test_uniforms_in_64_bits_next_to_one(spec, logits):
    want = spec.spec_sample(logits, torch.full((3,), LAST, device="cuda"), top_k=40)[0]
    assert (want >= 0).all()
    for near in (1.0 - 2.0 ** -25, 1.0 - 2.0 ** -26, 1.0 - 2.0 ** -53):
        forms = [torch.full((3,), near, dtype=torch.float64, device="cuda"), torch.full((3,), near, dtype=torch.float64), [near] * 3, near,
                 np.full(3, near)]
        for u in forms:
            assert torch.equal(spec.spec_sample(logits, u, top_k=40)[0], want), (near, type(u))


def test_uniforms_out_of_range_stay_so(spec, logits):
    for u in (1.0, 2.0, -1e-3, float("nan"), 1.0 + 2.0 ** -40):
        for form in (torch.full((3,), u, dtype=torch.float64, device="cuda"), [u] * 3, u):
            assert (spec.spec_sample(logits, form)[0] == -1).all(), u
