"""Pins of oracle/cache.py for rows that are not finite (CPU)."""
import math

import pytest
import torch

from oracle import cache as oc


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_int8_rows_that_are_not_finite_have_logit_zero(bad):
    """Attention over an int8 cache with such a row is that over one with a row of zeros in its place,
    whose logit is 0 too, where the page's other rows decide its scale; a bf16 cache keeps the row."""
    g = torch.Generator().manual_seed(0)
    n, d, page = 9, 64, 16
    x, v = (torch.randn((1, 1, n, d), generator=g).bfloat16() for _ in range(2))
    table = torch.tensor([[0]], dtype=torch.int32)
    spoilt, zero = x.clone(), x.clone()
    spoilt[0, 0, 4, 7] = bad
    zero[0, 0, 4] = 0
    outs = []
    for rows in (spoilt, zero):
        c = oc.empty(1, 1, page, d, True)
        oc.append(c, rows, v, table, [0])
        assert float(c["key_inv_norm"][0, 0, 4]) == 0.0
        outs.append(oc.attend(c, x[:, :, 8:], table, [8]))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    c = oc.empty(1, 1, page, d, False)
    oc.append(c, spoilt, v, table, [0])
    assert math.isnan(float(c["key_inv_norm"][0, 0, 4])) == math.isnan(bad)
