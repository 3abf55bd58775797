"""Codes of the 4-bit cache where a quotient lies on or next to a half, against the fp64 oracle.

A row's codes show in what a read gives: s * c + m rounded once, and another code is s away, more than the
rounding.  So the values read are compared for equality."""
import numpy as np
import pytest
import torch

from oracle import kv4 as O
from tests.test_gpu_kv4 import Cache, np64, spec_

pytestmark = pytest.mark.gpu


def held_bits(x, dtype, hd):
    """x [rows, 64] written as `dtype` (repeated to head_dim hd) and read back as fp16: (what K and V give,
    what the oracle holds, rounded to fp16)."""
    spec = spec_()
    y = torch.from_numpy(np.ascontiguousarray(x)).to(dtype)
    assert np.array_equal(np64(y), x)                       # the values are numbers of the type
    y = y.repeat(1, hd // 64).view(1, -1, 1, hd)
    c = Cache([y.shape[1]], 1, hd)
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    spec.spec_kv4_write(y.cuda(), y.cuda(), z, c.table, c.pool)
    want = np.clip(O.held(np64(y)), -O.HALF_MAX, O.HALF_MAX).astype(np.float16)
    return [t.cpu().numpy() for t in spec.spec_kv4_read(c.pool, z, c.table, y.shape[1])], want


def rows_at_halves(dtype):
    """Rows with s = 2^e and m = -(k + 1/2) s, whose tiny values have quotients next to k + 1/2."""
    least = 24 if dtype == torch.float16 else 100
    rows = []
    for e in range(-10, 14):
        s = 2.0 ** e
        for k in range(15):
            m, top = -(k + 0.5) * s, (14.5 - k) * s
            if max(-m, top) > O.HALF_MAX:
                continue
            tiny = [0.0] + [sg * 2.0 ** (e - j) for j in range(4, 34) for sg in (1, -1) if j - e <= least]
            rows.append([m, top] + (tiny + [0.0] * 62)[:62])
    return np.array(rows)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("copies", [1, 60])
def test_every_half_of_every_power_of_two_scale(dtype, hd, copies):
    """One copy is few rows, sixty are more than warps hold at once."""
    x = np.tile(rows_at_halves(dtype), (copies, 1))
    got, want = held_bits(x, dtype, hd)
    for y in got:
        assert np.array_equal(y, want)


def test_a_value_just_below_half_a_step():
    """min -1, max 29, so s = 2: -2^-24 is below 1/2 step and is held as -1, not as 1."""
    x = np.zeros((1, 64))
    x[0, :3] = -1, 29, -2.0 ** -24
    got, want = held_bits(x, torch.float16, 64)
    assert want[0, 0, 0, 2] == -1
    for y in got:
        assert np.array_equal(y, want)


def neighbours(v, dtype):
    """Four numbers of the type (fp64) around v: the third is the nearest, or next to it."""
    if dtype == torch.float16:
        h = v.astype(np.float16)
        lo, hi = np.nextafter(h, np.float16(-np.inf)), np.nextafter(h, np.float16(np.inf))
        near = [np.nextafter(lo, np.float16(-np.inf)), lo, h, hi]
    else:
        f = np.where(np.abs(v) < 1e-30, 1e-30, v).astype(np.float32).view(np.int32) & -65536     # towards zero
        near = [(f + d * 65536).view(np.float32) for d in (2, -1, 0, 1)]
    return [a.astype(np.float64) for a in near]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("n", [300, 40000])
def test_neighbours_of_every_border(dtype, hd, n):
    """Rows of any scale, most of them with -m/s far from a half: the numbers on both sides of every border
    m + (c + 1/2) s, c = 0..14."""
    rng = np.random.default_rng(n + hd)
    s0 = 2.0 ** rng.uniform(-9, 11, n)
    m = neighbours(s0 * rng.uniform(-25, 10, n), dtype)[2]
    top = neighbours(m + 15 * s0, dtype)[2]
    _, s, lo = (a[..., 0] if a.shape[-1] == 1 else a for a in O.quantise(np.stack([m, top], 1)))
    x = [m, top]
    for c in range(15):
        x += neighbours(lo + (c + 0.5) * s, dtype)
    x = np.stack(x + [m, top], 1)
    x = np.where((x < m[:, None]) | (x > top[:, None]), m[:, None], x)
    frac = np.abs((-lo / s) % 1 - 0.5)
    assert (frac > 0.02).mean() > 0.9                       # the rows that need no second look
    got, want = held_bits(x, dtype, hd)
    for y in got:
        assert np.array_equal(y, want)
