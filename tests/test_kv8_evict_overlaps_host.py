"""spec_kv8_evict refuses outputs that overlap each other or what the call reads: positions and pages are read back from
them between its two kernels."""
import pytest


@pytest.fixture(scope="module")
def spec():
    from speculative_decoding_verify_step_gb300 import build
    from speculative_decoding_verify_step_gb300 import spec
    spec.load_library(build.build())
    return spec


MB = 1 << 20
# bytes of each argument: B = 2, 3 heads of 64, 4 and 2 pages, 8 in the pool, 100 kept of 200 weights, 128 out
SIZES = dict(new_len=8, kept=2 * 3 * 100 * 4, wout=2 * 3 * 128 * 4, start=8, table=2 * 4 * 4, dst=2 * 2 * 4, weight=2 * 3 * 200 * 4,
             pool=8 * 3 * (128 * 64 + 64))
PLACE = {n: (i + 1) * MB for i, n in enumerate(SIZES)}


def evict(spec, **kw):
    a = dict(PLACE, **kw)
    return spec._lib.spec_kv8_evict(2, a["start"], a["table"], 4, a["dst"], 2, 8, 3, 64, 100, 10, a["weight"], 200, a["pool"], a["new_len"],
                                    a["kept"], a["wout"], 128, None)


@pytest.mark.parametrize("out", ["new_len", "kept", "wout"])
@pytest.mark.parametrize("other", list(SIZES))
def test_overlaps_are_refused(spec, out, other):
    if out == other:
        return
    last = PLACE[other] + SIZES[other] - 4              # the output's first entry on the other's last, and the other way round
    for at in (PLACE[other], last, PLACE[other] - SIZES[out] + 4):
        assert evict(spec, **{out: at}) == 1, at
        assert b"overlap" in spec._lib.spec_last_error()
