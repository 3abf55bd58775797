"""Sampling from logits without a GPU: the oracle's pins and every refusal of the C ABI and the binding."""
import numpy as np
import pytest
import torch

from oracle import accept as A
from oracle import sample as O


@pytest.fixture(scope="module")
def spec():
    from speculative_decoding_verify_step_gb300 import build
    from speculative_decoding_verify_step_gb300 import spec
    spec.load_library(build.build())
    return spec


def test_draw_is_the_acceptance_draw():
    rng = np.random.default_rng(0)
    for _ in range(50):
        R = np.floor(rng.random(37) ** 8 * 2.0 ** 40)
        u = np.float32(rng.random())
        assert O.draw(R, u)[0] == A.draw_index(R.astype(np.uint64), u)


def test_kept_tokens_by_hand():
    l = np.log(np.array([0.1, 0.4, 0.2, 0.25, 0.05]))
    kept = lambda **kw: np.nonzero(O.kept_masses(l, 1.0, **kw)[0])[0].tolist()  # noqa: E731
    assert kept() == [0, 1, 2, 3, 4] and kept(top_k=2) == [1, 3] and kept(top_p=0.6) == [1, 3]
    assert kept(top_p=0.66) == [1, 2, 3] and kept(min_p=0.5) == [1, 2, 3] and kept(top_k=3, top_p=0.7) == [1, 3]
    assert kept(min_p=1.0) == [1] and kept(top_k=9) == [0, 1, 2, 3, 4]
    assert np.nonzero(O.kept_masses(np.zeros(6), 1.0, top_k=2)[0])[0].tolist() == [0, 1]      # ties: lower index


def test_law():
    """Over all u of a grid the draws are q, to the grid."""
    l = np.array([0.3, -1.0, 2.0, 0.0, 1.5])
    q = O.sample(l, 0.0, 0.8, top_k=4, min_p=0.05)[1]
    n = 4000
    got = np.bincount([O.sample(l, np.float32((i + 0.5) / n), 0.8, top_k=4, min_p=0.05)[0] for i in range(n)], minlength=5) / n
    assert np.abs(got - q).max() <= 1.0 / n + 1e-6


def test_degenerate_rows():
    inf, nan = np.inf, np.nan
    assert O.sample([-inf, nan], 0.5)[0] == -1
    assert O.sample([nan, 1.0, -inf], 0.9)[0] == 1
    assert O.sample([inf, 5.0, inf], 0.75)[0] == 2 and O.sample([1.0, 3.0, 3.0], 0.2, 0.0)[0] == 1
    for kw in (dict(temperature=-1.0), dict(temperature=inf), dict(temperature=1e-9), dict(top_k=-1), dict(top_p=0.0),
               dict(top_p=1.5), dict(min_p=-0.1), dict(min_p=1.1)):
        assert O.sample([0.0, 1.0], 0.5, **kw)[0] == -1
    assert O.sample([0.0, 1.0], 1.0)[0] == -1 and O.sample([0.0, 1.0], nan)[0] == -1


def _call(spec, **kw):
    a = dict(rows=2, V=100, logits=4096, dtype=2, stride=100, u=4096, t_all=1.0, t=None, k=None, p=None, m=None, per=1,
             tokens=4096, probs=None)
    a.update(kw)
    return spec._lib.spec_sample(a["rows"], a["V"], a["logits"], a["dtype"], a["stride"], a["u"], a["t_all"], a["t"], a["k"],
                                 a["p"], a["m"], a["per"], a["tokens"], a["probs"], None)


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(rows=(1 << 24) + 1), dict(V=0), dict(V=393217, stride=393217), dict(dtype=3), dict(dtype=-1),
    dict(stride=99), dict(per=0), dict(t_all=-1.0), dict(t_all=float("nan")), dict(t_all=float("inf")), dict(t_all=1e-7), dict(t_all=1.1e30),
    dict(logits=None), dict(tokens=None), dict(u=None), dict(u=None, t_all=0.0, t=4096), dict(logits=4098),
    dict(logits=4097, dtype=1)])
def test_refusals(spec, kw):
    assert _call(spec, **kw) == 1
    assert spec._lib.spec_last_error() != b""


def test_no_rows_is_no_work(spec):
    assert _call(spec, rows=0) == 0


def test_binding_refusals(spec):
    with pytest.raises(ValueError):
        spec.spec_sample(torch.zeros(2, 8), torch.zeros(2))          # host tensor
