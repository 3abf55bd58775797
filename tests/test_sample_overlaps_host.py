"""spec_sample refuses outputs that overlap each other or an input, but for q in place of its logits."""
import pytest

from tests import test_kv8_host as K
from tests import test_sample_host as S

spec = K.spec
MB = 1 << 20
# 6 rows of 100 fp32 logits 120 apart, a setting for every 4 rows
SIZES = dict(tokens=24, probs=2400, logits=(5 * 120 + 100) * 4, u=24, t=8, k=8, p=8, m=8)
PLACE = {n: (i + 1) * MB for i, n in enumerate(SIZES)}


def call(spec, **kw):
    return S._call(spec, **{**PLACE, "rows": 6, "V": 100, "stride": 120, "per": 4, **kw})


@pytest.mark.parametrize("out", ["tokens", "probs"])
@pytest.mark.parametrize("other", list(SIZES))
def test_overlaps_are_refused(spec, out, other):
    if out == other:
        return
    for at in (PLACE[other], PLACE[other] + SIZES[other] - 4, PLACE[other] - SIZES[out] + 4):
        assert call(spec, **{out: at}) == 1, at
        assert b"overlap" in spec._lib.spec_last_error()


@pytest.mark.parametrize("kw", [dict(dtype=0), dict(dtype=1), dict(stride=101), dict(probs=4096 + 400), dict(probs=4096 - 400)])
def test_in_place_is_for_fp32_and_the_same_rows(spec, kw):
    assert S._call(spec, **dict(dict(logits=4096, probs=4096, tokens=1 << 22, u=1 << 23), **kw)) == 1
    assert b"probs overlaps logits" in spec._lib.spec_last_error()
