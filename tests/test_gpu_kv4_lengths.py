"""Attention over the 4-bit cache where kv_len lies outside the page table: window row j is token
kv_len + j, and a token before position 0 or past the table has no cell."""
import numpy as np
import pytest
import torch

from tests.test_gpu_kv4 import Cache, check, np64, rows_ref, spec_

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("grp,W", [(1, 4), (4, 8), (2, 16)])
def test_a_window_that_starts_before_the_first_token(grp, W, tree):
    """The rows before position 0 have no cell: the others see what is left of their window."""
    spec = spec_()
    Hkv, hd = 2, 128
    lens = [-1, -3, -W + 1, -W, -W - 1, -(1 << 31), 0, 40]
    parent = [-1] + [(j - 1) // 2 for j in range(1, W)] if tree else None
    c = Cache([max(n, 0) + W for n in lens], Hkv, hd, seed=W)
    held = c.fill(W)
    q = torch.randn(len(lens), W, Hkv * grp, hd, generator=torch.Generator().manual_seed(W)).half()
    kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for hint in (0, 40, 5000):
        got = spec.spec_kv4_attention(q.cuda(), c.pool, kv_len, c.table, parent=parent, max_kv_len=hint)
        for b, n in enumerate(lens):
            if n >= 0:
                check(got[b], *rows_ref(np64(q[b]), held[b], n, parent))
                continue
            cut = min(-n, W)                                 # rows without a cell
            (k, v), vs = held[b]
            pad = [np.concatenate([np.zeros((cut,) + x.shape[1:]), x[:W - cut]]) for x in (k, v, vs)]
            ok = np.arange(W) >= cut
            ref, tol = rows_ref(np64(q[b]), ((pad[0], pad[1]), pad[2]), 0, parent, key_ok=ok)
            check(got[b], ref, tol)
            if cut == W or not tree:
                assert (got[b, :cut] == 0).all()


def test_the_three_calls_agree_on_a_window_that_starts_before_the_first_token():
    """Rows written from position -2 on: the third is token 0, and alone is what the window sees."""
    spec = spec_()
    c = Cache([64], 1, 64)
    k, v = (torch.randn(1, 3, 1, 64).half().cuda() for _ in range(2))
    at = torch.tensor([-2], dtype=torch.int32, device="cuda")
    spec.spec_kv4_write(k, v, at, c.table, c.pool)
    held = spec.spec_kv4_read(c.pool, at, c.table, 3)[1]
    got = spec.spec_kv4_attention(torch.randn(1, 3, 1, 64).half().cuda(), c.pool, at, c.table)
    assert (got[0, :2] == 0).all() and (got[0, 2] - held[0, 2]).abs().max() <= 2.0 ** -9 * held[0, 2].abs().max()


def test_a_window_past_the_table():
    spec = spec_()
    c = Cache([128], 2, 64)                                  # a table of three entries, two with a page
    held = c.fill(3)
    tab = c.table[:, :2].contiguous()
    q = torch.randn(1, 4, 2, 64).half()
    for n in (126, 128, 129, 1 << 20, (1 << 31) - 1):
        got = spec.spec_kv4_attention(q.cuda(), c.pool, torch.tensor([n], dtype=torch.int32, device="cuda"), tab)
        pad = max(0, min(n, 128) + 4 - 128)
        (k, v), vs = held[0]
        at = min(n, 128)
        ext = [np.concatenate([x, np.zeros((pad,) + x.shape[1:])]) for x in (k, v, vs)]
        ok = np.arange(128 + pad) < 128
        check(got[0], *rows_ref(np64(q[0]), ((ext[0], ext[1]), ext[2]), at, key_ok=ok))
