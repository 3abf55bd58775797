"""top_k, top_p, min_p and temperature of spec_sample as 64-bit numbers and tensors, and numpy's numbers: what they say
counts, not what is left of them in 32 bits."""
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
    return torch.randn(3, 5000, generator=torch.Generator().manual_seed(1)).cuda(), torch.tensor([0.9, 0.5, 0.99]).cuda()


def test_a_top_k_past_the_vocabulary_is_off(spec, logits):
    x, u = logits
    want, q = spec.spec_sample(x, u, 2.0, return_probs=True)
    for k in (5000, 2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 63 - 1):
        for form in (k, [k] * 3, torch.full((3,), k), torch.full((3,), k, device="cuda"), np.full(3, k, np.int64)):
            got, p = spec.spec_sample(x, u, 2.0, top_k=form, return_probs=True)
            assert torch.equal(got, want) and torch.equal(p, q), (k, type(form))


def test_negative_top_k_is_out_of_range(spec, logits):
    x, u = logits
    for k in (-1, -2 ** 32 + 7, -2 ** 63):
        for form in (k, [k] * 3, torch.full((3,), k, device="cuda")):
            assert (spec.spec_sample(x, u, 2.0, top_k=form)[0] == -1).all(), k


def test_numbers_below_fp32_are_not_zero(spec, logits):
    x, u = logits
    best = x.argmax(1).int()
    for tiny in (1e-50, 1e-320):
        for form in (lambda v: v, lambda v: [v] * 3, lambda v: torch.full((3,), v, dtype=torch.float64, device="cuda")):
            assert torch.equal(spec.spec_sample(x, u, 1.0, top_p=form(tiny))[0], best)      # the first token reaches it
            assert (spec.spec_sample(x, u, [tiny] * 3)[0] == -1).all()                       # neither 0 nor in range
        with pytest.raises(spec.SpecError):
            spec.spec_sample(x, u, tiny)


def test_numpy_numbers_count_for_all_rows(spec, logits):
    x, u = logits
    want = spec.spec_sample(x, u, 0.5, top_k=7, top_p=0.75, min_p=0.25)[0]
    for f, i in ((np.float32, np.int64), (np.float64, np.int32)):
        got = spec.spec_sample(x, u, f(0.5), top_k=i(7), top_p=f(0.75), min_p=f(0.25))[0]
        assert torch.equal(got, want)
    assert torch.equal(spec.spec_sample(x, np.float32(0.5), 0.5)[0], spec.spec_sample(x, 0.5, 0.5)[0])
