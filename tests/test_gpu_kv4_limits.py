"""The workspace size of the 4-bit attention is -1 exactly where the call refuses the shape."""
import pytest

from tests.test_gpu_kv4 import spec_

pytestmark = pytest.mark.gpu

GOOD = dict(B=2, W=3, Hq=4, H=2, hd=64, max_pages=4, hint=0)


def both(**kw):
    """(workspace bytes, status of the call without rows)."""
    spec = spec_()
    a = dict(GOOD, **kw)
    lib = spec.load_library()
    size = lib.spec_kv4_attention_workspace(a["B"], a["W"], a["Hq"], a["H"], a["hd"], a["max_pages"], a["hint"])
    # with row_off and no rows a call that is not refused is no work
    status = lib.spec_kv4_attention(a["B"], a["W"], 0, 4096, 4096, 4096, a["max_pages"], 8, a["Hq"], a["H"], a["hd"], 0, 4096, a["Hq"] * a["hd"],
                                    None, 0.125, a["hint"], 4096, 4096, 4096, 1 << 40, None)
    return size, status


@pytest.mark.parametrize("kw", [dict(), dict(B=65535), dict(B=4096, H=8, Hq=8, max_pages=32768), dict(W=16, Hq=8), dict(max_pages=1 << 24, B=1)])
def test_shapes_that_are_served(kw):
    size, status = both(**kw)
    assert size >= 0 and status == 0


@pytest.mark.parametrize("kw", [dict(B=0), dict(B=65536), dict(H=65536, Hq=65536, B=1), dict(H=0), dict(Hq=5), dict(hd=96), dict(W=0),
                                dict(W=17), dict(W=16, Hq=16), dict(max_pages=0), dict(max_pages=(1 << 24) + 1, B=1), dict(hint=-1),
                                dict(B=4096, H=8, Hq=8, max_pages=32769)])
def test_shapes_that_are_refused(kw):
    size, status = both(**kw)
    assert size == -1 and status != 0
