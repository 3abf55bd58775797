"""Drafts that are rejected: what the caller clears of the accumulated weights, and what stays in the cache."""
import numpy as np
import pytest
import torch

from oracle import kv4 as O4
from oracle import kv8 as O
from tests._gpu import need_gpu
from tests.test_gpu_kv8 import Cache, run_evict

pytestmark = pytest.mark.gpu
H, HD, GRP = 2, 64, 2


@pytest.fixture(scope="module")
def spec():
    need_gpu()
    from speculative_decoding_verify_step_gb300 import spec
    spec.load_library()
    return spec


class Drafter:
    """Decode steps over one sequence, and the weights that they give in 64 bits."""

    def __init__(self, spec, n):
        self.spec, self.c, self.n = spec, Cache(spec, 1, H, HD, 4, spare=4), n
        self.c.write([0], [self.c.values(n)], [self.c.values(n)])
        self.weight = torch.zeros(1, H, 256, device="cuda")
        self.ref = np.zeros((H, 256))

    def step(self, gain=1.0):
        self.c.write([self.n], [self.c.values(1, gain)], [self.c.values(1, gain)])
        q = torch.from_numpy(self.c.rng.normal(size=(1, 1, H * GRP, HD))).to(torch.float16)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        out = self.spec.spec_kv8_attention(q.cuda(), self.c.pool, i32([self.n]), self.c.table, weight=self.weight)
        k, v = self.c.held(0, self.n + 1)
        ref, probs = O4.attention(q[0].double().numpy(), k, v, self.n)
        assert np.abs(out[0].double().cpu().numpy() - ref).max() <= np.abs(v).max() * 2.0 ** -8
        for h in range(H):
            self.ref[h, :self.n + 1] += probs[h].sum((0, 1))
        self.n += 1

    def check(self):
        assert np.abs(self.weight[0].double().cpu().numpy() - self.ref).max() <= 1e-4


def test_weights_of_rejected_tokens_are_cleared_by_the_caller(spec):
    d = Drafter(spec, 100)
    for _ in range(2):
        d.step()
    for _ in range(3):                                    # drafts, of which the first is accepted
        d.step()
    d.n = 103
    assert (d.weight[0, :, 103:105] > 0).all()            # a call only adds: the rejected ones' entries are there
    d.weight[:, :, d.n:] = 0
    d.ref[:, d.n:] = 0
    for _ in range(4):
        d.step()
    d.check()                                             # tokens written over them have their own weights alone
    run_evict(spec, d.c, [d.n], d.weight, 40, 4)


def test_a_copy_takes_back_the_rejected_rows_shares_too(spec):
    d = Drafter(spec, 60)
    d.step()
    kept, ref = d.weight.clone(), d.ref.copy()
    for _ in range(2):                                    # rejected, both
        d.step()
    d.n, d.ref = 61, ref
    d.weight.copy_(kept)
    for _ in range(5):
        d.step()
    d.check()


def test_a_rejected_outlier_leaves_its_exponent(spec):
    """Until a write starts the sub-block anew, what comes next is held on the outlier's grid (Cache.write
    follows that rule bit for bit)."""
    d = Drafter(spec, 70)
    d.step(gain=5000.0)                                   # at 70, in the sub-block from 64 on
    coarse = [d.c.v[0][h].e[4] for h in range(H)]
    d.n = 70
    d.weight[:, :, 70:] = 0
    d.c.write([70], [d.c.values(3)], [d.c.values(3)])
    assert [d.c.v[0][h].e[4] for h in range(H)] == coarse and min(coarse) > O.needed_exp(10.0)
    d.c.check_read([0], [73], "fp16")
    d.c.write([64], [d.c.values(9)], [d.c.values(9)])     # from its first token on
    assert max(d.c.v[0][h].e[4] for h in range(H)) < min(coarse)
    d.c.check_read([0], [73], "fp16")
