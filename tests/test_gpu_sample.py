"""Sampling from logits on the GPU against the oracle: tokens and kept sets exactly, q to fp32's roundings.
Masses are good to about 2^-42 of themselves before their floor, so each may be a unit (2^-40) off and a
sum of V of them V units: where a decision lies nearer than that to another outcome, the other one is as
good, and the row is held to that distance."""
import numpy as np
import pytest
import torch

from oracle import sample as O
from tests._gpu import need_gpu

pytestmark = pytest.mark.gpu
DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def spec():
    need_gpu()
    from speculative_decoding_verify_step_gb300 import spec
    spec.load_library()
    return spec


def logits_of(rows, V, dt, seed, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, V, generator=g) * spread
    x.scatter_add_(1, torch.randint(0, V, (rows, min(V, 30)), generator=g), 6 * torch.rand(rows, min(V, 30), generator=g))
    return x.to(DT[dt]), torch.rand(rows, generator=g)


def check(spec, x, u, t=1.0, k=None, p=None, m=None, per=1, probs=True):
    """x [rows, V] on the CPU or a CUDA view; settings: numbers or one per setting."""
    xg = x if x.is_cuda else x.cuda()
    rows, V = xg.shape
    tok, q = spec.spec_sample(xg, u.cuda(), t, k, p, m, rows_per_setting=per, return_probs=probs)
    again, _ = spec.spec_sample(xg, u.cuda(), t, k, p, m, rows_per_setting=per)
    assert torch.equal(tok, again)
    at = lambda s, r, default: default if s is None else (s[r // per] if isinstance(s, (list, tuple)) else s)  # noqa: E731
    f32 = lambda v: float(np.float32(v))  # noqa: E731
    xc = xg.double().cpu().numpy()
    eps = 2 * V * 2.0 ** -40
    for r in range(rows):
        ur, kw = u[r].item(), dict(temperature=f32(at(t, r, 1.0)), top_k=int(at(k, r, 0)), top_p=f32(at(p, r, 1.0)), min_p=f32(at(m, r, 0.0)))
        ref, qr, near = O.sample(xc[r], ur, **kw)
        v, got = int(tok[r]), q[r].double().cpu().numpy() if probs else None
        if near < eps and v != ref:
            cum, want = np.cumsum(qr), np.floor(ur * 2 ** 24) / 2 ** 24
            assert cum[v] - qr[v] - eps <= want <= cum[v] + eps, (r, v, ref, near)
        else:
            assert v == ref, (r, v, ref, near)
        if probs:
            other = (got > 0) != (qr > 0)
            assert (near < eps and np.maximum(got, qr)[other].sum() <= eps) or not other.any(), r
            # R / Z: R to 2^-42 and a unit, then roundings of R, Z, 1/Z and the product to fp32
            assert (np.abs(got - qr)[~other] <= qr[~other] * (2.0 ** -21 + 2 * eps * (near < eps)) + 2.0 ** -39).all(), r
    return tok, q


@pytest.mark.parametrize("dt", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("V", [1, 2, 7, 31, 300, 4096, 4097, 10007, 50257, 128256])
def test_vocabularies(spec, V, dt):
    x, u = logits_of(5, V, dt, V)
    check(spec, x, u, 0.7)
    check(spec, x, u, 1.0, k=[1, 3, 50, 0, V + 5], p=0.9)
    check(spec, x, u, 1.3, k=40, m=[0.0, 0.01, 0.1, 0.5, 1.0])
    check(spec, x, u, 0.9, p=[0.5, 0.95, 1.0, 0.999999, 1e-6], m=0.001)


def test_largest_vocabulary(spec):
    x, u = logits_of(2, 393216, "fp32", 1)
    check(spec, x, u, 1.0, p=0.95)
    check(spec, x, u, 1.0, k=[1000, 393215])


@pytest.mark.parametrize("rows,V", [(700, 1003), (300, 5001), (33, 33000)])
def test_many_rows(spec, rows, V):
    x, u = logits_of(rows, V, "bf16", rows)
    check(spec, x, u, 0.8, k=60, p=0.9, m=0.01)


def test_peaked_and_flat_rows(spec):
    for spread in (0.0, 1e-3, 30.0, 1e4, 1e30):
        x, u = logits_of(3, 3000, "fp32", 4, spread)
        if spread == 0.0:
            x.zero_()                                   # all equal: ranks by index alone
        for kw in (dict(), dict(k=100), dict(p=0.5), dict(k=1000, p=0.3), dict(m=0.5)):
            check(spec, x, u, 1.0, **kw)
    x, u = logits_of(3, 3000, "fp32", 5)
    for t in (1e-6, 1e-3, 50.0, 1e6, 1e30):
        check(spec, x, u, t, k=500, p=0.9)
        check(spec, x, u, t, p=0.9)


def test_ties_go_to_the_lower_index(spec):
    g = torch.Generator().manual_seed(0)
    x = torch.randint(-2, 3, (6, 40000), generator=g).float()          # five values: thousands of ties at each cut
    u = torch.rand(6, generator=g)
    for kw in (dict(k=100), dict(k=9000), dict(p=0.3), dict(k=20000, p=0.7), dict(k=20000, p=0.01), dict(m=0.4)):
        check(spec, x, u, 1.0, **kw)
    z = x.clone()
    z[:, ::2] = 0.0
    z[:, 1::2] = -0.0                                                  # equal numbers
    check(spec, z, u, 1.0, k=777)


def test_a_bin_that_holds_every_scale_of_floats(spec):
    """Logits around zero, from 1e-30 to 1e-3 and of both signs, in one bin of the first histogram."""
    g = torch.Generator().manual_seed(2)
    x = torch.randn(4, 6000, generator=g).sign() * 10.0 ** (-3 - 27 * torch.rand(4, 6000, generator=g))
    u = torch.rand(4, generator=g)
    for kw in (dict(k=10), dict(k=3000), dict(p=0.5), dict(k=4000, p=0.5)):
        check(spec, x, u, 1.0, **kw)


def test_not_a_number_and_infinities(spec):
    inf, nan = float("inf"), float("nan")
    x, u = logits_of(8, 5000, "fp32", 9)
    x[0, :] = -inf
    x[1, :] = nan
    x[2, 100:] = -inf
    x[3, ::3] = nan
    x[4, [7, 4000]] = inf
    x[5, 4999] = inf
    x[6, :] = -inf
    x[6, 4321] = -3e38
    x[7, 0] = 3.4e38
    x[7, 1] = -3.4e38
    for kw in (dict(), dict(k=5), dict(p=0.9), dict(k=500, p=0.9, m=0.01)):
        tok, q = check(spec, x, u, 1.0, **kw)
        assert tok[:2].tolist() == [-1, -1] and (q[:2] == 0).all()
    tok, _ = check(spec, x, u, 0.0)
    assert tok[4] == 7 and tok[6] == 4321


@pytest.mark.parametrize("dt", ["fp32", "fp16"])
@pytest.mark.parametrize("none", [float("nan"), -float("inf")])
def test_top_k_that_ends_among_tokens_without_mass(spec, none, dt):
    x, u = logits_of(2, 5000, dt, 14)
    x[0, 4590:4990] = none
    x[1, torch.randperm(5000, generator=torch.Generator().manual_seed(2))[:700]] = none
    for k in (4299, 4300, 4301, 4599, 4600, 4601, 4800, 4999):
        check(spec, x, u, 1.0, k=k)
        check(spec, x, u, 2.0, k=k, p=0.99)


@pytest.mark.parametrize("spread", [0.01, 0.3, 5.0])
def test_limits_among_neighbours(spec, spread):
    """Where the limits end in bins of few, of many and of a thousand tokens."""
    x, u = logits_of(3, 20000, "fp32", 15)
    x = x.clamp(max=3.0) * spread
    for kw in (dict(k=40), dict(k=120), dict(k=130), dict(k=300), dict(k=513), dict(k=900), dict(p=0.002), dict(p=0.05), dict(p=0.5),
               dict(k=200, p=0.3), dict(k=1500, p=0.6), dict(k=60, p=0.9, m=0.3)):
        check(spec, x, u, 1.0, **kw)


@pytest.mark.parametrize("rows,V", [(1, 128256), (3, 50257)])
def test_infinities_of_one_slice(spec, rows, V):
    """+infinity in one CTA's slice of a row, the first one's among them, with a small top_k."""
    x, u = logits_of(rows, V, "fp32", 12)
    for at in ([0], [7, 11], [V // 2], [V // 3, V // 3 + 1], [V - 1]):
        y = x.clone()
        y[:, at] = float("inf")
        for k in (1, 2, 5):
            tok, q = check(spec, y, u, 1.0, k=k)
            assert all(int(t) in at for t in tok)
            check(spec, y, u, 0.7, k=k, p=0.9)


def test_greedy(spec):
    x, u = logits_of(6, 20011, "bf16", 3)
    tok, q = check(spec, x, u, 0.0, k=5, p=0.5)
    got, none = spec.spec_sample(x.cuda(), temperature=0.0)
    assert none is None and torch.equal(got, tok) and torch.equal(q.argmax(1).int(), tok) and (q.sum(1) == 1).all()
    check(spec, x, u, [0.0, 1.0, 0.0, 0.5, 0.0, 2.0], p=0.9)


def test_settings_out_of_range(spec):
    inf, nan = float("inf"), float("nan")
    x, u = logits_of(1, 500, "fp32", 3)
    rows = x.expand(12, 500).contiguous()
    us = u.expand(12).clone()
    us[10], us[11] = 1.0, nan
    t = [1.0, -1.0, inf, nan, 1e-7] + [1.0] * 7
    k = [0, 0, 0, 0, 0, -1, 0, 0, 0, 0, 0, 0]
    p = [1.0] * 6 + [0.0, 1.5, 1.0, 1.0, 1.0, 1.0]
    m = [0.0] * 8 + [-0.1, 1.01, 0.0, 0.0]
    tok, q = check(spec, rows, us, t, k=k, p=p, m=m)
    assert (tok[1:] == -1).all() and (q[1:] == 0).all() and tok[0] >= 0


def test_temperatures_at_their_ends(spec):
    x, u = logits_of(6, 3000, "fp32", 5)
    x[1:3] *= 1e30
    x[3:] *= 1e-6
    check(spec, x, u, [1e-6, 1e30, 3e30, 1e-6, 2e-6, 1e-4], p=0.9)
    check(spec, x, u, 1e30)
    check(spec, x, u, 1e-6, k=7)


def test_uniforms_at_their_ends(spec):
    x, _ = logits_of(4, 9000, "fp32", 8)
    x[:, 0] = x[:, -1] = x.max() + 1                      # so that neither end is a decision near another
    u = torch.tensor([0.0, 2.0 ** -24, 1 - 2.0 ** -24, 0.5])
    tok, _ = spec.spec_sample(x.cuda(), u.cuda(), 1.0)
    assert tok[0] == 0 and tok[2] == 8999
    for r in (1, 3):
        assert int(tok[r]) == O.sample(x[r].double().numpy(), u[r].item())[0]


def test_strided_rows_settings_per_group_and_outputs(spec):
    x, u = logits_of(6, 1001, "bf16", 12)
    wide = torch.full((6, 1037), 99.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 3:1004] = x.cuda()
    check(spec, wide[:, 3:1004], u, [0.5, 1.0, 2.0], k=[5, 0, 30], p=[1.0, 0.8, 0.9], per=2)
    outs = (torch.empty(6, dtype=torch.int32, device="cuda"), torch.full((6, 1001), 5.0, device="cuda"))
    tok, q = spec.spec_sample(x.cuda(), u.cuda(), 0.8, top_k=20, outs=outs)
    assert tok is outs[0] and q is outs[1] and ((q > 0).sum(1) == 20).all() and torch.allclose(q.sum(1), torch.ones(6, device="cuda"), atol=1e-5)
    y = x.view(2, 3, 1001).cuda()
    t3, q3 = spec.spec_sample(y, u.view(2, 3).cuda(), 0.8, top_k=20, return_probs=True)
    assert t3.shape == (2, 3) and torch.equal(t3.view(-1), tok) and torch.equal(q3.view(6, -1), q)


def test_binding_refusals_on_the_device(spec):
    x = torch.zeros(2, 8, device="cuda")
    u = torch.zeros(2, device="cuda")
    for bad in (lambda: spec.spec_sample(x.double(), u), lambda: spec.spec_sample(x.t(), u), lambda: spec.spec_sample(x, u[:1]),
                lambda: spec.spec_sample(x, u, [1.0, 1.0, 1.0]), lambda: spec.spec_sample(x, u, top_k=[1]),
                lambda: spec.spec_sample(x, u, rows_per_setting=0),
                lambda: spec.spec_sample(x, u, outs=(torch.empty(2, device="cuda"), None)),
                lambda: spec.spec_sample(x, u, outs=(torch.empty(2, dtype=torch.int32, device="cuda"), torch.empty(2, 7, device="cuda")))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(spec.SpecError):
        spec.spec_sample(x, None, 1.0)
    with pytest.raises(spec.SpecError):
        spec.spec_sample(x, u, -1.0)
    assert spec.spec_sample(x[:0], u[:0])[0].shape == (0,)
