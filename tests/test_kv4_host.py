"""4-bit KV cache without a GPU: the oracle's pins and every refusal of the C ABI and the binding."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import kv4 as O


@pytest.fixture(scope="module")
def spec():
    from speculative_decoding_verify_step_gb300 import build
    from speculative_decoding_verify_step_gb300 import spec
    spec.load_library(build.build())
    return spec


# ------------------------------------------------------------------------- the oracle
def test_hand_values():
    x = np.array([0.0, 1.0, 7.0, 15.0])
    c, s, m = O.quantise(x)
    assert s.item() == 1.0 and m.item() == 0.0 and c.tolist() == [0, 1, 7, 15]
    x = np.array([-1.0, -1.0, 0.5, 2.0])              # s = 0.2 rounded up to fp16
    c, s, m = O.quantise(x)
    assert m.item() == -1.0 and 0.2 <= s.item() <= 0.2 * (1 + 2 ** -10) and c.tolist() == [0, 0, 7, 15]
    assert O.held(np.array([3.0, 3.0, 3.0])).tolist() == [3.0, 3.0, 3.0]        # no spread: the value itself
    assert O.held(np.array([np.nan, np.inf])).tolist()[0] == -65504.0
    c, _, _ = O.quantise(np.array([0.0, 0.5, 1.5, 15.0]))                     # halves go up
    assert c.tolist() == [0, 1, 2, 15]


def test_held_values_are_within_half_a_step():
    rng = np.random.default_rng(0)
    for scale in (1e-7, 1e-3, 1.0, 300.0, 2e4):
        x = (rng.normal(size=(500, 64)) * scale).astype(np.float16).astype(np.float64)
        c, s, m = O.quantise(x)
        assert c.min() >= 0 and c.max() <= 15
        assert (np.abs(O.held(x) - O.saturate(x)) <= s / 2 * (1 + 1e-12)).all()


def test_window_mask_chain_and_tree():
    assert np.array_equal(O.window_mask(4), np.tril(np.ones((4, 4), bool)))
    see = O.window_mask(5, [-1, 0, 0, 1, 1])
    assert see[3].tolist() == [True, True, False, True, False] and see[2].tolist() == [True, False, True, False, False]


def test_attention_of_one_token_is_its_value():
    rng = np.random.default_rng(1)
    v = rng.normal(size=(1, 2, 64))
    out, _ = O.attention(rng.normal(size=(1, 4, 64)), rng.normal(size=(1, 2, 64)), v, 0)
    assert np.allclose(out[0], np.repeat(v[0], 2, 0))
    out, _ = O.attention(rng.normal(size=(1, 4, 64)), rng.normal(size=(1, 2, 64)), v, 0, key_ok=np.array([False]))
    assert (out == 0).all()


# ------------------------------------------------------------------------- refusals (C ABI)
def _write(spec, **kw):
    a = dict(B=2, n=3, total=6, row_off=None, start=4096, table=4096, max_pages=4, num_pages=8, H=2, hd=64, dtype=0,
             k=4096, v=4096, ks=128, vs=128, pool=4096)
    a.update(kw)
    return spec._lib.spec_kv4_write(a["B"], a["n"], a["total"], a["row_off"], a["start"], a["table"], a["max_pages"],
                                    a["num_pages"], a["H"], a["hd"], a["dtype"], a["k"], a["v"], a["ks"], a["vs"],
                                    a["pool"], None)


def _read(spec, **kw):
    a = dict(B=2, n=3, total=6, row_off=None, start=4096, table=4096, max_pages=4, num_pages=8, H=2, hd=64, dtype=0,
             k=4096, v=4096, pool=4096)
    a.update(kw)
    return spec._lib.spec_kv4_read(a["B"], a["n"], a["total"], a["row_off"], a["start"], a["table"], a["max_pages"],
                                   a["num_pages"], a["H"], a["hd"], a["dtype"], a["pool"], a["k"], a["v"], None)


def _attend(spec, **kw):
    a = dict(B=2, n=3, total=6, row_off=None, start=4096, table=4096, max_pages=4, num_pages=8, Hq=4, H=2, hd=64,
             dtype=0, q=4096, qs=256, parent=None, scale=0.125, hint=0, pool=4096, out=4096, ws=4096, ws_bytes=1 << 40)
    a.update(kw)
    return spec._lib.spec_kv4_attention(a["B"], a["n"], a["total"], a["row_off"], a["start"], a["table"],
                                        a["max_pages"], a["num_pages"], a["Hq"], a["H"], a["hd"], a["dtype"], a["q"],
                                        a["qs"], a["parent"], a["scale"], a["hint"], a["pool"], a["out"], a["ws"],
                                        a["ws_bytes"], None)


COMMON = [(dict(hd=96), 7), (dict(hd=0), 7), (dict(B=0, total=0), 1), (dict(B=65536, total=65536 * 3), 1),
          (dict(H=0), 1), (dict(num_pages=0), 1), (dict(max_pages=0), 1), (dict(max_pages=1 << 25), 1),
          (dict(num_pages=1 << 25), 1), (dict(dtype=2), 1), (dict(dtype=-1), 1), (dict(total=5), 1),
          (dict(total=-1, row_off=4096), 1), (dict(start=None), 1), (dict(table=None), 1), (dict(pool=None), 1),
          (dict(pool=4100), 1)]


@pytest.mark.parametrize("call", [_write, _read, _attend])
@pytest.mark.parametrize("kw,status", COMMON)
def test_common_refusals(spec, call, kw, status):
    assert call(spec, **kw) == status
    assert spec._lib.spec_last_error() != b""


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
    (dict(scale=float("inf")), 1), (dict(scale=float("nan")), 1), (dict(scale=1.2e12), 1), (dict(scale=-1.2e12), 1), (dict(hint=-1), 1), (dict(ws=None, max_pages=4096), 1), (dict(ws=4100, max_pages=4096), 1),
    (dict(n=9, total=18, Hq=16), 7),                                  # 9 rows x 8 heads of a group
    (dict(parent=(ctypes.c_int32 * 3)(0, 0, 1)), 1), (dict(parent=(ctypes.c_int32 * 3)(-1, 1, 0)), 1)])
def test_attention_refusals(spec, kw, status):
    assert _attend(spec, **kw) == status


@pytest.mark.parametrize("call", [_write, _read, _attend])
def test_no_rows_is_no_work(spec, call):
    assert call(spec, total=0, row_off=4096) == 0


def test_block_bytes(spec):
    assert [spec._lib.spec_kv4_block_bytes(h) for h in (64, 128, 32, 0, 256)] == [4608, 8704, 0, 0, 0]
    assert spec.spec_kv4_pool(3, 2, 128, device="cpu").shape == (3, 2, 8704)
    with pytest.raises(ValueError):
        spec.spec_kv4_pool(3, 2, 96, device="cpu")


# ------------------------------------------------------------------------- refusals (binding)
def test_binding_refuses_host_and_misshapen_tensors(spec):
    pool = spec.spec_kv4_pool(4, 2, 64, device="cpu")
    i32 = dict(dtype=torch.int32)
    start, table = torch.zeros(2, **i32), torch.zeros(2, 3, **i32)
    k = torch.zeros(2, 5, 2, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA device"):
        spec.spec_kv4_write(k, k, start, table, pool)
    for bad in (dict(pool=pool.float()), dict(pool=pool[:, :, :100]), dict(pool=pool[:, :1]), dict(start=start.long()),
                dict(table=table.long()), dict(table=torch.zeros(3, 3, **i32)), dict(table=table.t()),
                dict(row_off=torch.zeros(2, **i32)), dict(row_off=torch.zeros(3))):
        a = dict(pool=pool, start=start, table=table, row_off=None)
        a.update(bad)
        with pytest.raises(ValueError):
            spec._kv4_geometry(a["pool"], a["start"], a["table"], a["row_off"])


def test_binding_row_geometry(spec):
    dev = torch.device("cpu")
    rows = lambda x, heads=2, ragged=False: spec._kv4_rows(x, "x", 2, heads, 64, ragged, dev)   # noqa: E731
    assert rows(torch.zeros(2, 5, 2, 64, dtype=torch.float16)) == (10, 5, 128)
    fused = torch.zeros(2, 5, 6, 64, dtype=torch.bfloat16)
    assert rows(fused[:, :, 2:4]) == (10, 5, 384)                      # a view into q | k | v
    assert rows(fused[:, :1, 2:4]) == (2, 1, 5 * 384)
    assert rows(torch.zeros(7, 2, 64, dtype=torch.float16), ragged=True) == (7, 0, 128)
    assert rows(torch.zeros(0, 2, 64, dtype=torch.float16), ragged=True)[0] == 0
    for bad in (torch.zeros(2, 5, 2, 64), torch.zeros(3, 5, 2, 64).half(), torch.zeros(2, 5, 3, 64).half(),
                torch.zeros(2, 5, 2, 128).half(), torch.zeros(2, 5, 64, 2).half().transpose(2, 3),
                torch.zeros(2, 2, 5, 64).half().transpose(1, 2), torch.zeros(2, 9, 2, 64).half()[:, :5],
                torch.zeros(10, 2, 64).half()):
        with pytest.raises(ValueError):
            rows(bad)


def test_model_refuses_an_unknown_cache_format(spec):
    from speculative_decoding_verify_step_gb300 import synth
    d = synth.TINY
    cfg = spec.spec_config(d.n_layers, d.d_model, d.n_heads, d.n_kv_heads, d.head_dim, d.ffn_dim, d.vocab, d.rms_eps,
                           d.rope_theta, 64, 2, 4, 256, 8)
    h = ctypes.c_void_p()
    assert spec._lib.spec_model_create_kv(ctypes.byref(cfg), 2, ctypes.byref(h)) == 1 and not h.value
    assert spec._lib.spec_model_create_kv(None, 1, ctypes.byref(h)) == 1
    with pytest.raises(ValueError):
        spec.SpecModel(d, max_batch=2, max_width=4, max_seq_len=256, num_pages=8, kv_format="int3")
