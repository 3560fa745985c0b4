"""rope_frequencies refuses what would make a table of zeros or infinities."""
import math

import pytest
import torch

from moe_expert_gemv_b200 import qmoe


@pytest.mark.parametrize("kw", [dict(base=math.inf), dict(kind="linear", factor=math.inf), dict(kind="ramp", factor=math.inf, trained=100),
                                dict(kind="base", factor=math.inf), dict(base=1e300, kind="base", factor=1e30),
                                dict(kind="bands", factor=2.0, trained=100, high=math.inf),
                                dict(kind="ramp", factor=2.0, trained=100, high=math.inf)], ids=str)
def test_infinite_arguments_refused(kw):
    with pytest.raises(qmoe.QmoeError) as e:
        qmoe.rope_frequencies(8, **kw)
    assert e.value.code == qmoe.ERR_INVALID_ARG


@pytest.mark.parametrize("kind", list(qmoe.ROPE_KINDS))
def test_the_widest_finite_ones(kind):
    f, scale = qmoe.rope_frequencies(64, 1e100, kind, 1e30, trained=2 ** 31 - 1, low=1e-30, high=1e30)
    assert torch.isfinite(f).all() and (f > 0).all() and math.isfinite(scale)
