"""The per-kernel record of a model with a 4-bit cache holds every launch that its attention class names."""
import pytest
import torch

from speculative_decoding_verify_step_gb300 import synth
from tests._gpu import need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,per_layer", [("fp16", 1), ("int4", 2)])
@pytest.mark.parametrize("B,W", [(1, 1), (2, 4)])
def test_the_write_of_the_window_is_recorded(fmt, per_layer, B, W):
    """int4: the window's cells are written by a launch of their own, over their fp16 rows and their bytes."""
    need_gpu()
    from speculative_decoding_verify_step_gb300 import spec
    d = synth.TINY
    m = spec.SpecModel(d, max_batch=2, max_width=4, max_seq_len=256, num_pages=12, kv_format=fmt)
    m.load_weights((k, v.cuda()) for k, v in synth.make_weights(d, seed=1).items())
    m.kv_fill_random(list(range(B)), [70] * B, seed=1, scale=0.5)
    tok = torch.ones(B, W, dtype=torch.int32)
    m.set_profiling(True)
    m.read_profile()
    m.verify_step(list(range(B)), tok)
    m.sync_status()
    ms, n, by = m.read_profile()["attention"]
    m.close()
    assert n == per_layer * d.n_layers and ms > 0
    tokens = B * (70 + W) * d.n_kv_heads
    if fmt == "fp16":
        assert by == d.n_layers * tokens * 4 * d.head_dim
    else:
        cell = d.head_dim + 8
        assert by == d.n_layers * (tokens * cell + B * W * d.n_kv_heads * (4 * d.head_dim + cell))
