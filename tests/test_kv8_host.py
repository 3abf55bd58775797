"""8-bit KV cache without a GPU: the oracle's pins and every refusal of the C ABI and the binding."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import kv8 as O


@pytest.fixture(scope="module")
def spec():
    from speculative_decoding_verify_step_gb300 import build
    from speculative_decoding_verify_step_gb300 import spec
    spec.load_library(build.build())
    return spec


# ------------------------------------------------------------------------- the oracle
def test_e4m3_against_torch():
    """All codes are fixed points, and numbers between two codes go where torch's conversion takes them."""
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    codes = codes[~torch.isnan(codes)].double().numpy()
    assert np.array_equal(O.e4m3(codes), codes)
    rng = np.random.default_rng(0)
    y = np.concatenate([rng.uniform(-448, 448, 4000), rng.uniform(-0.1, 0.1, 4000), (np.sort(codes)[1:] + np.sort(codes)[:-1]) / 2])
    y = y.astype(np.float32)
    ref = torch.from_numpy(y).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(O.e4m3(y), ref)


def test_exponents():
    assert O.needed_exp(0.0) == -15 and O.needed_exp(448.0) == 0 and O.needed_exp(448.1) == 1
    assert O.needed_exp(65504.0) == 8 and O.needed_exp(224.0) == -1 and O.needed_exp(448 * 2.0 ** -15) == -15


def test_raising_keeps_what_is_normal():
    c = O.HeldSeq(16, 4)
    x = np.array([[1.0, -0.5, 0.25, 448.0]])
    c.write(0, x)
    before = c.y.copy()
    c.write(1, np.array([[30000.0, 1.0, 2.0, -3.0]]))
    assert c.e[0] == 7 and np.array_equal(c.y[0, 3], before[0, 3])
    assert np.allclose(c.y[0], before[0], atol=2.0 ** -10 * 2 ** 7)   # half a subnormal step of the new grid
    c.write(0, x)                                                      # the first token starts it anew
    assert c.e[0] == 0 and np.array_equal(c.y[0], before[0])


def test_keep_tokens():
    w = np.array([0.5, 0.1, 0.5, np.nan, 0.9, 0.0, -np.inf])
    assert O.keep_tokens(w, 7, 3, 0).tolist() == [0, 2, 4]
    assert O.keep_tokens(w, 7, 3, 1).tolist() == [0, 4, 6]
    assert O.keep_tokens(w, 7, 6, 0).tolist() == [0, 1, 2, 4, 5, 6]    # NaN last
    assert O.keep_tokens(w, 2, 5, 5).tolist() == [0, 1]


# ------------------------------------------------------------------------- refusals (C ABI)
def _write(spec, **kw):
    a = dict(B=2, n=3, total=6, row_off=None, start=4096, table=4096, max_pages=4, num_pages=8, H=2, hd=64, dtype=0,
             k=4096, v=4096, ks=128, vs=128, pool=4096)
    a.update(kw)
    return spec._lib.spec_kv8_write(a["B"], a["n"], a["total"], a["row_off"], a["start"], a["table"], a["max_pages"],
                                    a["num_pages"], a["H"], a["hd"], a["dtype"], a["k"], a["v"], a["ks"], a["vs"],
                                    a["pool"], None)


def _read(spec, **kw):
    a = dict(B=2, n=3, total=6, row_off=None, start=4096, table=4096, max_pages=4, num_pages=8, H=2, hd=64, dtype=0,
             k=4096, v=4096, pool=4096)
    a.update(kw)
    return spec._lib.spec_kv8_read(a["B"], a["n"], a["total"], a["row_off"], a["start"], a["table"], a["max_pages"],
                                   a["num_pages"], a["H"], a["hd"], a["dtype"], a["pool"], a["k"], a["v"], None)


def _attend(spec, **kw):
    a = dict(B=2, n=3, total=6, row_off=None, start=4096, table=4096, max_pages=4, num_pages=8, Hq=4, H=2, hd=64,
             dtype=0, q=4096, qs=256, parent=None, scale=0.125, hint=0, pool=4096, out=4096, weight=None, T=0, ws=4096,
             ws_bytes=1 << 40)
    a.update(kw)
    return spec._lib.spec_kv8_attention(a["B"], a["n"], a["total"], a["row_off"], a["start"], a["table"],
                                        a["max_pages"], a["num_pages"], a["Hq"], a["H"], a["hd"], a["dtype"], a["q"],
                                        a["qs"], a["parent"], a["scale"], a["hint"], a["pool"], a["out"], a["weight"],
                                        a["T"], a["ws"], a["ws_bytes"], None)


def _evict(spec, **kw):
    a = dict(B=2, start=4096, table=4096, max_pages=4, dst=4096, dst_pages=2, num_pages=8, H=2, hd=64, keep=100, recent=10,
             weight=1 << 20, T=256, pool=4096, new_len=1 << 16, kept=4096, wout=1 << 30, To=256)
    a.update(kw)
    return spec._lib.spec_kv8_evict(a["B"], a["start"], a["table"], a["max_pages"], a["dst"], a["dst_pages"], a["num_pages"],
                                    a["H"], a["hd"], a["keep"], a["recent"], a["weight"], a["T"], a["pool"], a["new_len"],
                                    a["kept"], a["wout"], a["To"], None)


COMMON = [(dict(hd=96), 7), (dict(hd=0), 7), (dict(B=0, total=0), 1), (dict(B=65536, total=65536 * 3), 1),
          (dict(H=0), 1), (dict(num_pages=0), 1), (dict(max_pages=0), 1), (dict(max_pages=1 << 25), 1),
          (dict(num_pages=1 << 25), 1), (dict(start=None), 1), (dict(table=None), 1), (dict(pool=None), 1),
          (dict(pool=4100), 1)]
ROWS = [(dict(dtype=2), 1), (dict(dtype=-1), 1), (dict(total=5), 1), (dict(total=-1, row_off=4096), 1)]


@pytest.mark.parametrize("call", [_write, _read, _attend])
@pytest.mark.parametrize("kw,status", COMMON + ROWS)
def test_common_refusals(spec, call, kw, status):
    assert call(spec, **kw) == status
    assert spec._lib.spec_last_error() != b""


@pytest.mark.parametrize("kw,status", [(k, s) for k, s in COMMON])
def test_evict_common_refusals(spec, kw, status):
    kw = {k: v for k, v in kw.items() if k != "total"}
    assert _evict(spec, **kw) == status


@pytest.mark.parametrize("kw", [
    dict(keep=0), dict(keep=-3), dict(keep=129), dict(recent=-1), dict(recent=101), dict(dst_pages=0), dict(dst_pages=1),
    dict(T=0), dict(T=(1 << 30) + 1), dict(To=99), dict(To=(1 << 30) + 1), dict(dst=None), dict(weight=None), dict(new_len=None),
    dict(kept=None), dict(wout=None), dict(weight=(1 << 20) + 2), dict(wout=(1 << 30) + 1), dict(wout=1 << 20),
    dict(wout=(1 << 20) + 2 * 2 * 256 * 4 - 4)])
def test_evict_refusals(spec, kw):
    assert _evict(spec, **kw) == 1


@pytest.mark.parametrize("at", [4096, 4100, 4092])
def test_evict_new_len_is_not_kv_len(spec, at):
    assert _evict(spec, new_len=at) == 1
    assert b"new_len overlaps kv_len" in spec._lib.spec_last_error()


@pytest.mark.parametrize("kw", [dict(), dict(out=4096 + 6 * 512 - 16), dict(q=4096 + 6 * 512 - 16),
                                dict(qs=512, out=4096 + 5 * 1024 + 496)])
def test_attention_with_weights_is_not_in_place(spec, kw):
    assert _attend(spec, weight=1 << 20, T=64, **kw) == 1
    assert b"out overlaps q" in spec._lib.spec_last_error()


@pytest.mark.parametrize("kw", [dict(k=None), dict(v=None), dict(k=4104), dict(v=4098), dict(ks=120), dict(vs=120),
                                dict(ks=132), dict(n=-1, total=-2)])
def test_write_refusals(spec, kw):
    assert _write(spec, **kw) == 1


@pytest.mark.parametrize("kw", [dict(k=None), dict(v=None), dict(k=4104), dict(v=4098), dict(n=-1, total=-2)])
def test_read_refusals(spec, kw):
    assert _read(spec, **kw) == 1


@pytest.mark.parametrize("kw,status", [
    (dict(n=0, total=0), 1), (dict(n=17, total=34), 1), (dict(Hq=5), 1), (dict(Hq=0), 1), (dict(q=None), 1),
    (dict(out=None), 1), (dict(q=4104), 1), (dict(out=4104), 1), (dict(qs=248), 1), (dict(qs=260), 1),
    (dict(scale=float("inf")), 1), (dict(scale=float("nan")), 1), (dict(scale=1.2e12), 1), (dict(hint=-1), 1),
    (dict(ws=None, max_pages=4096), 1), (dict(ws=4100, max_pages=4096), 1), (dict(weight=4096, T=0), 1), (dict(weight=4098, T=64), 1),
    (dict(n=9, total=18, Hq=16), 7),                                  # 9 rows x 8 heads of a group
    (dict(H=1 << 14, Hq=1 << 14, max_pages=1 << 16), 7),
    (dict(parent=(ctypes.c_int32 * 3)(0, 0, 1)), 1), (dict(parent=(ctypes.c_int32 * 3)(-1, 1, 0)), 1)])
def test_attention_refusals(spec, kw, status):
    assert _attend(spec, **kw) == status


@pytest.mark.parametrize("call", [_write, _read, _attend])
def test_no_rows_is_no_work(spec, call):
    n = 1 if call is _attend else 0
    assert call(spec, n=n, total=0, row_off=4096) == 0


def test_block_bytes_and_workspace(spec):
    assert [spec._lib.spec_kv8_block_bytes(h) for h in (64, 128, 96, 0)] == [8256, 16448, 0, 0]
    for bad in ((0, 1, 1, 4, 2, 64, 4, 0, 0), (1, 17, 1, 4, 2, 64, 4, 0, 0), (1, 1, 1, 5, 2, 64, 4, 0, 0),
                (1, 1, 1, 4, 2, 96, 4, 0, 0), (1, 16, 16, 16, 2, 64, 4, 0, 0), (1, 1, -1, 4, 2, 64, 4, 0, 0),
                (1, 1, 1, 4, 2, 64, 4, -1, 0)):
        assert spec._lib.spec_kv8_attention_workspace(*bad) == -1


# ------------------------------------------------------------------------- refusals (binding)
def test_binding_refusals(spec):
    pool = torch.zeros(4, 2, 8256, dtype=torch.uint8)
    i32 = dict(dtype=torch.int32)
    start, table = torch.zeros(2, **i32), torch.zeros(2, 2, **i32)
    k = torch.zeros(2, 3, 2, 64, dtype=torch.float16)
    with pytest.raises(ValueError):                       # host tensors
        spec.spec_kv8_write(k, k, start, table, pool)
    with pytest.raises(ValueError):
        spec.spec_kv8_pool(4, 2, 96)
    with pytest.raises(ValueError):                       # a 4-bit pool
        spec.spec_kv8_read(torch.zeros(4, 2, 4608, dtype=torch.uint8), start, table, 3)
    with pytest.raises(ValueError):
        spec.spec_kv8_read(pool, start.long(), table, 3)
    with pytest.raises(ValueError):
        spec.spec_kv8_evict(pool, torch.zeros(2, 2, 64), start, table[:1], table, 4)
