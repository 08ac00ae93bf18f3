"""Pins of oracle/cache.py against things other than itself (CPU)."""
import math

import numpy as np
import pytest
import torch

import oracle
from oracle import cache as oc


def rows(*shape, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g)


@pytest.mark.parametrize("adjacent", [False, True])
def test_rotation_is_a_complex_product(adjacent):
    x = rows(1, 2, 5, 8)
    dims, freqs = (4, 2), torch.tensor([1.0, 0.25, 0.5])
    pos = torch.tensor([[0, 1, -2, 30, 7], [5, 4, 3, 2, 1]])
    y = oc.rope(x, pos, freqs, dims, adjacent)
    z = x.double()
    for t in range(5):
        for p, (a, lo, hi) in enumerate([(0, 0, 1 if adjacent else 2), (0, 2 if adjacent else 1, 3),
                                         (1, 4, 5)]):
            turn = complex(math.cos(int(pos[a, t]) * float(freqs[p])),
                           math.sin(int(pos[a, t]) * float(freqs[p])))
            for h in range(2):
                w = complex(z[0, h, t, lo], z[0, h, t, hi]) * turn
                assert abs(w - complex(y[0, h, t, lo], y[0, h, t, hi])) < 1e-14
    assert torch.equal(y[..., 6:], z[..., 6:])


def test_rotation_depends_on_differences_of_positions_and_keeps_norms():
    x = rows(1, 1, 2, 64)
    freqs = 10000.0 ** (-torch.arange(32) / 32)
    a = oc.rope(x, torch.tensor([[3, 10]]), freqs, (64,))[0, 0]
    b = oc.rope(x, torch.tensor([[1003, 1010]]), freqs, (64,))[0, 0]
    assert abs(float(a[0] @ a[1] - b[0] @ b[1])) < 1e-10
    assert torch.allclose(a.norm(dim=-1), x[0, 0].double().norm(dim=-1), rtol=1e-13)


def test_inverse_undoes_and_is_the_gradient():
    x = rows(2, 1, 3, 16).double().requires_grad_()
    pos = torch.tensor([[[1, 2, 3], [9, 8, 7]], [[0, 5, 6], [4, 4, 4]]])
    freqs, dims = torch.tensor([1.0, 0.5, 0.3, 0.7]), (4, 4)
    y = oc.rope(x, pos, freqs, dims)
    assert torch.allclose(oc.rope(y, pos, freqs, dims, inverse=True), x, atol=1e-14)
    g = rows(2, 1, 3, 16, seed=1).double()
    (y * g).sum().backward()
    assert torch.allclose(oc.rope(g, pos, freqs, dims, inverse=True), x.grad, atol=1e-14)


@pytest.mark.parametrize("n,split", [(1, [1]), (37, [37]), (37, [20, 1, 16]), (64, [33, 31])])
def test_attention_over_the_cache_is_the_dense_attention(n, split):
    """Appending a sequence piece by piece and attending with every piece gives the rows of dense
    causal attention over it."""
    H, d, P = 2, 64, 16
    x, v = rows(1, H, n, d).bfloat16(), rows(1, H, n, d, seed=1).bfloat16()
    ref, ref_lse = oracle.dense_sampled(x, v, True, np.arange(n, dtype=np.int32))
    cache = oc.empty(9, H, P, d, False)
    table = torch.tensor([[7, 2, 5, 0, 8]])
    at = 0
    for m in split:
        xs, vs = x[:, :, at:at + m], v[:, :, at:at + m]
        oc.append(cache, xs, vs, table, [at])
        out, lse, _ = oc.attend(cache, xs, table, [at])
        # 1/||x|| is held in fp32: half a step of it moves a logit by 2^-24 of its value, below 8
        # here, and an output by about twice that of |v| < 6
        assert np.abs(out.numpy() - ref[:, :, at:at + m]).max() < 6 * 2 * 8 * 2.0 ** -24
        # the lse of a row that sees itself alone is -1e5 on both sides
        assert np.abs(lse.numpy() - ref_lse.reshape(1, H, n)[:, :, at:at + m]).max() < 8 * 2.0 ** -23
        at += m


def test_int8_values_stay_within_the_last_scale():
    """However often a page's scale grows, a stored value is within one last step of the row: half
    for the last rounding and 1/4 + 1/8 + ... for those before it."""
    H, d, P = 1, 64, 16
    cache = oc.empty(2, H, P, d, True)
    table = torch.tensor([[1]])
    data = [(rows(1, H, 1, d, seed=s) * 2.0 ** s).bfloat16() for s in range(8)]
    for i, r in enumerate(data):
        oc.append(cache, r, r, table, [i])
    s = float(cache["k_scale"][1, 0])
    assert 127 * s >= data[-1].abs().max() > 127 * s / 2
    k, v, _ = oc.read(cache, table, 0, 0, 8)
    full = torch.cat(data, 2)[0, 0].double()
    assert (k - full).abs().max() <= s and (v - full).abs().max() <= s
    assert torch.equal(k[7], torch.round(full[7] / s) * s)
    # slots of later tokens are as they were
    assert (cache["k"][1, 0, 8:] == 99).all() and (cache["v"][1, 0, 0, :, 8:] == 99).all()


@pytest.mark.parametrize("amax,scale", [(127.0, 1.0), (127.5, 2.0), (1.0, 2.0 ** -6), (0.0, 2.0 ** -126),
                                        (3.0e38, 2.0 ** 121)])
def test_scale(amax, scale):
    assert oc.scale_for(amax) == scale
