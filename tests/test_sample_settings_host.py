"""Settings of spec_sample as the kernel gets them, from every type that a caller may hold them in."""
import math

import numpy as np
import pytest
import torch

from speculative_decoding_verify_step_gb300.spec import _setting

CPU = torch.device("cpu")


@pytest.mark.parametrize("dt", [torch.uint8, torch.int8, torch.int16, torch.int32, torch.int64, torch.float16, torch.bfloat16, torch.float32,
                                torch.float64])
def test_top_k_of_any_type(dt):
    got = _setting(torch.tensor([5, 0, 120], dtype=dt), torch.int32, 3, CPU, "top_k")
    assert got.dtype is torch.int32 and got.tolist() == [5, 0, 120]
    if dt.is_signed:
        assert (_setting(torch.tensor([-3, -1], dtype=dt), torch.int32, 2, CPU, "top_k") < 0).all()


@pytest.mark.parametrize("k,want", [(7, 7), (2 ** 31, 2 ** 31 - 1), (2 ** 63 - 1, 2 ** 31 - 1), (-2 ** 63, -1), (np.int64(9), 9), (True, 1),
                                    (math.inf, 2 ** 31 - 1), (math.nan, -1), (40.0, 40)])
def test_top_k_numbers(k, want):
    for form in (k, [k, k], torch.tensor([k, k]), np.array([k, k])):
        assert _setting(form, torch.int32, 2, CPU, "top_k").tolist() == [want] * 2, type(form)


@pytest.mark.parametrize("x", [0.0, 1e-50, -1e-50, 0.7, math.nan, math.inf, 1e300, -1e300, 1, np.float32(0.5), np.float64(0.25)])
def test_other_numbers(x):
    for form in (x, [x], np.array([x]), torch.tensor([float(x)], dtype=torch.float64)):
        got = _setting(form, torch.float32, 1, CPU, "top_p")
        assert got.dtype is torch.float32
        y = got.item()
        if x != x:
            assert y != y
        elif 0 < abs(x) < 2.0 ** -149:
            assert abs(y) == 2.0 ** -149 and (y > 0) == (x > 0)
        elif abs(x) > 3.5e38:
            assert y == math.copysign(math.inf, x)
        else:
            assert y == torch.tensor(float(x)).item()


def test_what_is_right_already_is_taken_as_it_is():
    for t in (torch.rand(4), torch.arange(4, dtype=torch.int32)):
        assert _setting(t, t.dtype, 4, CPU, "x") is t
    assert _setting(None, torch.float32, 4, CPU, "x") is None
    with pytest.raises(ValueError):
        _setting(torch.rand(3), torch.float32, 4, CPU, "x")
