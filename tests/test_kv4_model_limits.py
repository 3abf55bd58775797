"""Pages of a model with a 4-bit cache: slots (page * 64 + offset) are 32-bit numbers."""
import ctypes

import pytest


@pytest.mark.parametrize("num_pages", [(1 << 24) + 1, 1 << 25, (1 << 31) - 1])
def test_more_pages_than_slots_can_name_are_refused(num_pages):
    from speculative_decoding_verify_step_gb300 import build, spec, synth
    lib = spec.load_library(build.build())
    d = synth.TINY
    cfg = spec.spec_config(d.n_layers, d.d_model, d.n_heads, d.n_kv_heads, d.head_dim, d.ffn_dim, d.vocab, d.rms_eps, d.rope_theta, 64, 2, 4,
                           256, num_pages)
    h = ctypes.c_void_p()
    assert lib.spec_model_create_kv(ctypes.byref(cfg), 1, ctypes.byref(h)) == 1 and not h.value
    assert b"num_pages" in lib.spec_last_error()
