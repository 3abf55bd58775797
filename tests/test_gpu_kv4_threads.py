"""Calls of the 4-bit cache's operators from another host thread do not count as a model's launches."""
import threading

import pytest
import torch

from speculative_decoding_verify_step_gb300 import synth
from tests.test_gpu_kv4 import Cache, spec_

pytestmark = pytest.mark.gpu


def test_launch_count_of_a_round_beside_another_thread():
    spec = spec_()
    d = synth.TINY
    m = spec.SpecModel(d, max_batch=1, max_width=4, max_seq_len=512, num_pages=8, kv_format="int4")
    m.load_weights((k, v.cuda()) for k, v in synth.make_weights(d, seed=1).items())
    tok = torch.ones(1, 4, dtype=torch.int32, device="cuda")
    m.kv_fill_random([0], [70], seed=1, scale=0.5)
    m.verify_step([0], tok)
    m.sync_status()
    alone = m.last_launch_count()
    c = Cache([64], 1, 64)
    c.fill(1)
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    stop = threading.Event()

    def read():
        with torch.cuda.stream(torch.cuda.Stream()):
            while not stop.is_set():
                for _ in range(20):
                    spec.spec_kv4_read(c.pool, z, c.table, 4)
                torch.cuda.current_stream().synchronize()

    other = threading.Thread(target=read)
    other.start()
    counts = set()
    try:
        for i in range(400):
            if i % 20 == 0:
                m.kv_fill_random([0], [70], seed=1, scale=0.5)
            m.verify_step([0], tok)
            counts.add(m.last_launch_count())
        m.sync_status()
    finally:
        stop.set()
        other.join()
    m.close()
    assert counts == {alone}
