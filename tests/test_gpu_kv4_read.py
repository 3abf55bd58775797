"""Reads of the 4-bit cache are s * c + m rounded once: equality with the 64-bit value, rounded once."""
import numpy as np
import pytest
import torch

from oracle import kv4 as O
from tests.test_gpu_kv4 import Cache, np64, spec_

pytestmark = pytest.mark.gpu


def to_bf16(v):
    """fp64 (0, or of bf16's normal range) to the nearest bf16 number, ties to even, in one rounding."""
    f, e = np.frexp(v)
    return np.ldexp(np.rint(np.ldexp(f, 8)), e - 8)


def read_back(x, dtype, as_dtype, hd):
    spec = spec_()
    y = torch.from_numpy(np.ascontiguousarray(x)).to(dtype).view(1, -1, 1, hd)
    c = Cache([y.shape[1]], 1, hd)
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    spec.spec_kv4_write(y.cuda(), y.cuda(), z, c.table, c.pool)
    return [np64(t) for t in spec.spec_kv4_read(c.pool, z, c.table, y.shape[1], dtype=as_dtype)], O.held(np64(y))


def test_rounding_of_the_test_itself():
    assert to_bf16(np.array([0.0, 1.0, 1 + 2.0 ** -8, 1 + 2.0 ** -8 + 2.0 ** -40, 1 + 3 * 2.0 ** -8, -116.25000066])).tolist() == [
        0.0, 1.0, 1.0, 1 + 2.0 ** -7, 1 + 2.0 ** -6, -116.5]


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("n", [200, 40000])
def test_bf16_read_next_to_a_tie_is_rounded_once(hd, n):
    """s c is half way between two bf16 numbers and m a last bit on either side of it: rounded to fp32 first,
    the sum would be that tie."""
    rng = np.random.default_rng(hd)
    s = (2 * rng.integers(32, 64, n) + 1) * 2.0 ** rng.integers(-3, 3, n)     # 7 bits, odd
    m = 2.0 ** -24 * rng.integers(1, 4, n) * rng.choice([1, -1], n)
    x = np.stack([m + 0 * s, 15 * s], 1)
    x = np.concatenate([x] + [(s * c)[:, None] for c in range(1, 15)] * (hd // 16) + [x] * hd, 1)[:, :hd]
    got, held = read_back(x, torch.float16, torch.bfloat16, hd)
    want = to_bf16(held)
    assert (to_bf16(held.astype(np.float32).astype(np.float64)) != want).mean() > 0.02    # the rows show it
    for y in got:
        assert np.array_equal(y, want)


@pytest.mark.parametrize("hd", [64, 128])
def test_bf16_read_of_one_known_cell(hd):
    x = np.full((1, hd), 6.5565e-7)
    x[0, 1], x[0, 2:12] = 217.875, np.linspace(100, 130, 10)
    got, held = read_back(x, torch.float16, torch.bfloat16, hd)
    for y in got:
        assert np.array_equal(y, to_bf16(held))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("as_dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("hd", [64, 128])
def test_reads_of_any_scale_and_offset_are_rounded_once(dtype, as_dtype, hd):
    rng = np.random.default_rng(7)
    n = 30000
    x = rng.normal(size=(n, hd)) * 2.0 ** rng.uniform(-20, 8, (n, 1)) + rng.normal(size=(n, 1)) * 2.0 ** rng.uniform(-24, 8, (n, 1))
    x[:50] *= 200                                           # up to and past fp16's largest
    x = np.clip(x, -O.HALF_MAX, O.HALF_MAX)
    got, held = read_back(x, dtype, as_dtype, hd)
    if as_dtype == torch.float16:
        want = np.clip(held, -O.HALF_MAX, O.HALF_MAX).astype(np.float16).astype(np.float64)
    else:
        want = to_bf16(held)
    for y in got:
        assert np.array_equal(y, want)
