"""The 8-bit cache's calls and spec_sample refuse arrays of 4-byte numbers that are not 4-byte aligned: a kernel's
access to one would be an error of the GPU."""
import pytest

from tests import test_kv8_host as K
from tests import test_sample_host as S

spec = K.spec


@pytest.mark.parametrize("by", [1, 2, 3])
@pytest.mark.parametrize("call,names", [(K._write, ["row_off", "start", "table"]), (K._read, ["row_off", "start", "table"]),
                                        (K._attend, ["row_off", "start", "table", "weight"]),
                                        (K._evict, ["start", "table", "dst", "new_len", "kept", "wout", "weight"]),
                                        (S._call, ["u", "t", "k", "p", "m", "tokens", "probs"])])
def test_misaligned(spec, call, names, by):
    for name in names:
        kw = {name: (1 << 22) + by}
        if name == "weight" and call is K._attend:
            kw["T"] = 64
        assert call(spec, **kw) == 1, name
        assert b"must be 4-byte aligned" in spec._lib.spec_last_error(), name
