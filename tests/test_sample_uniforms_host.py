"""Uniforms of other types than fp32: the draw takes floor(2^24 u), and a number below one stays below one."""
import numpy as np
import pytest
import torch

from speculative_decoding_verify_step_gb300.spec import _uniforms

CPU = torch.device("cpu")


def test_fp32_is_taken_as_it_is():
    u = torch.rand(5)
    assert _uniforms(u, 5, CPU) is u and _uniforms(None, 5, CPU) is None


def test_64_bits_keep_their_first_24():
    x = np.concatenate([np.random.default_rng(0).random(1000), [0.0, 1 - 2.0 ** -53, 1 - 2.0 ** -25, 1 - 2.0 ** -24, 0.5 + 3 * 2.0 ** -26, 2.0 ** -60]])
    want = torch.from_numpy(np.floor(x * 2 ** 24) / 2 ** 24).float()
    assert (want < 1).all()
    for form in (x, torch.from_numpy(x), x.tolist()):
        got = _uniforms(form, len(x), CPU)
        assert got.dtype is torch.float32 and torch.equal(got, want)
    for v in x[-6:]:
        assert torch.equal(_uniforms(float(v), 2, CPU), torch.full((2,), math_floor(v)))


def math_floor(v):
    return float(np.float32(np.floor(v * 2 ** 24) / 2 ** 24))


@pytest.mark.parametrize("v", [1.0, 1.0 + 2.0 ** -40, 2.0, -1e-30, -0.5, float("inf"), -float("inf"), float("nan")])
def test_out_of_range_stays_so(v):
    for form in (v, [v] * 3, torch.full((3,), v, dtype=torch.float64)):
        got = _uniforms(form, 3, CPU)
        assert not ((got >= 0) & (got < 1)).any()
