"""What is no number stays none in the 4-bit attention's output: NaN rows are how a call without a status word
tells of a wait that ran out, so the output's saturation must let them through.  Here the NaN come from
cells that hold no numbers (never written, in a pool of 0xff)."""
import pytest
import torch

from tests.test_gpu_kv4 import Cache, check, np64, rows_ref, spec_

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("lens,W,grp,hd", [([64, 70], 1, 4, 64), ([500, 640], 2, 4, 128), ([700, 650], 12, 4, 128), ([5000, 3000], 3, 4, 128),
                                           ([9000, 40], 12, 4, 64)])
def test_rows_over_cells_without_numbers_are_nan(dtype, lens, W, grp, hd):
    """A cluster, one CTA, and merged pieces: the rows of the sequence with such a cell are NaN, those of the other are right."""
    spec = spec_()
    c = Cache([n + W for n in lens], 2, hd, seed=W)
    held = c.fill(W)
    page = int(c.table[0, (lens[0] - 1) // 64])
    c.pool[page] = 0xff
    q = torch.randn(2, W, 2 * grp, hd, generator=torch.Generator().manual_seed(W)).to(dtype)
    for hint in (0, max(lens)):
        got = spec.spec_kv4_attention(q.cuda(), c.pool, torch.tensor(lens, dtype=torch.int32, device="cuda"), c.table, max_kv_len=hint)
        assert got[0].isnan().all()
        check(got[1], *rows_ref(np64(q[1]), held[1], lens[1], dtype=dtype))


def test_values_past_the_largest_are_still_held_to_it():
    """V of 65504 everywhere, held as it is: the output is fp16's largest, not an infinity."""
    spec = spec_()
    c = Cache([130], 1, 64)
    k, v = torch.randn(1, 130, 1, 64).half().cuda(), torch.full((1, 130, 1, 64), 65504.0, dtype=torch.float16, device="cuda")
    v[0, ::2] *= -1
    v[0, ::2, 0, 0] = 65504                                 # 15 s + m passes 65504 in these rows
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    spec.spec_kv4_write(k, v, z, c.table, c.pool)
    got = spec.spec_kv4_attention(torch.randn(1, 2, 2, 64).half().cuda(), c.pool, z + 128, c.table)
    assert got.isfinite().all() and (got[..., 0] == 65504).all()
