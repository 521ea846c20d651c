"""The AdamW descriptor's ranges are those of the header (CPU, before any GPU call)."""
import math

import pytest

from test_block_abi import E_DEV, E_SHAPE, ad, pytestmark, step  # noqa: F401


@pytest.mark.parametrize("kw,want", [
    (dict(eps=1e-30), E_DEV), (dict(eps=1e30), E_DEV), (dict(eps=9.9e-31), E_SHAPE), (dict(eps=1.1e30), E_SHAPE),
    (dict(eps=-1e-8), E_SHAPE), (dict(eps=math.nan), E_SHAPE),
    # the step is fp32: a rate that it cannot hold would turn every parameter into a NaN
    (dict(lr=3.4e38), E_DEV), (dict(lr=-3.4e38), E_DEV), (dict(lr=1e39), E_SHAPE), (dict(lr=-1e300), E_SHAPE),
    (dict(lr=math.nan), E_SHAPE)])
def test_adamw_ranges(kw, want):
    assert step(ad(**kw)) == want
