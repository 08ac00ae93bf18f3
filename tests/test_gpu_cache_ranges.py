"""Rotary positions, the paged cache and attention over it where values, norms and scales lie far
apart, through the C ABI, against oracle/cache.py (float64).

Tolerances of the attention. With nq the largest ||x_t|| and r the largest ||k_j|| / ||x_j|| (1 but for
the rounding of a stored row), a logit is a sum of d products, off by d 2^-24 nq r ||x_j||, times
1 / (||x_j|| sqrt(d)): sqrt(d) 2^-24 nq r; its scalings and its difference to the row's reference are
six roundings of at most nq r / sqrt(d) <= nq r / 8: together below E = (sqrt(d) + 4) 2^-24 nq r. A weight is
off by E of itself, 2^-20 for the exponential and 2^-16 for its two bf16 parts; sums of n <= 4096 terms, sixteen
to a step, by n / 16 2^-23 <= 2^-15 of sum p |v|; the normaliser by as much. The output by
(2 E + 2^-13) sum p |v| and its own rounding, 2^-8; whatever the sizes of the values in other dimensions, of
other tokens, or behind the row. lse: E, 2^-14, and 2^-22 of itself. Both formats: the bounds of
test_gpu_cache.py for int8 are wider, derived for weights in f16 and keys with an offset.
"""
import math

import pytest
import torch

from lsh_attention_b200 import binding as lb
from oracle import cache as oc
from test_gpu_cache import bits, freqs_of, near, randn, same_cache, table_of, to_gpu

pytestmark = pytest.mark.gpu

DEV = "cuda"


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def filled(x, v, page, int8):
    """A cache of the rows x, v [1, H, n, d], its table, and both on the GPU."""
    _, H, n, d = x.shape
    per_seq = n // page + 1
    ref = oc.empty(per_seq + 1, H, page, d, int8)
    table = table_of(1, per_seq, per_seq + 1)
    oc.append(ref, x, v, table, [0])
    return ref, table, to_gpu(ref)


def check_attend(ref, table, gpu, q, length):
    d = q.shape[-1]
    out, lse = lb.lsh_cache_attend(gpu, q.cuda(), table.cuda(), ints(length))
    ro, rl, mag = oc.attend(ref, q, table, [length])
    r = 1.0
    for h in range(q.shape[1]):
        k, _, kinv = oc.read(ref, table, 0, h, length + q.shape[2])
        r = max(r, float((k.norm(dim=-1) * kinv).max()))
    E = (math.sqrt(d) + 4) * 2.0 ** -24 * float(q.double().norm(dim=-1).max()) * r
    near(out, ro, ro.abs() * 2.0 ** -8 + mag * (2 * E + 2.0 ** -13), "out")
    near(lse, rl, E + 2.0 ** -14 + rl.abs() * 2.0 ** -22, "lse")
    return out, lse


# ------------------------------------------------------------------------------ sizes of values
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("n", [1, 12])
@pytest.mark.parametrize("d,page", [(64, 16), (64, 64), (128, 32)])
@pytest.mark.parametrize("up", [12, 20, 30, 60])
@pytest.mark.parametrize("where", [3, 397])
@pytest.mark.parametrize("sharp", [False, True])
def test_attend_one_large_value(sharp, where, up, d, page, n, int8):
    """One value of one token is 2^up times the others, with an ordinary weight, or with a small one
    beside a key that takes nearly all (in whose own zeros the small weights alone are seen): the
    other dimensions do not feel it."""
    L = 400
    x, v = randn(1, 1, L + n, d, seed=1), randn(1, 1, L + n, d, seed=2)
    if sharp:
        u = randn(d, seed=3)
        x[0, 0, L:] = 16 * u + x[0, 0, L:]   # logits of 16 for u, -16 for -u
        x[0, 0, 200], x[0, 0, where] = u, -u
        v[0, 0, 200, :d // 2] = 0.0
    v[0, 0, where, 5] = 2.0 ** up
    x, v = x.bfloat16(), v.bfloat16()
    ref, table, gpu = filled(x, v, page, int8)
    check_attend(ref, table, gpu, x[:, :, L:], L)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("n", [4, 13])
@pytest.mark.parametrize("end", [113, 129])
@pytest.mark.parametrize("up", [0, 20, 40, 90])
def test_attend_a_large_value_behind_the_row(up, end, n, int8):
    """The last drafted token begins a page and has large values: the rows before it, which do not
    see it, are the bits that they are without it."""
    d, page = 64, 16
    L = end - n
    x, v = randn(1, 2, L + n, d, seed=1).bfloat16(), randn(1, 2, L + n, d, seed=2).bfloat16()
    base = None
    for f in (1.0, 2.0 ** up):
        w = v.clone()
        w[:, :, -1] *= f
        ref, table, gpu = filled(x, w, page, int8)
        out, lse = check_attend(ref, table, gpu, x[:, :, L:], L)
        if base is None:
            base = out, lse
        assert torch.equal(out[:, :, :-1], base[0][:, :, :-1]) and torch.equal(lse, base[1])


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("n", [1, 9])
@pytest.mark.parametrize("sizes", [(-110,) * 3, (100,) * 3, (0, 30, -30), (-60, 0, 40), (40, -50, 5)])
def test_attend_values_of_every_size(sizes, n, int8):
    """Pages of values 2^size, one size after the other, tiny, huge and mixed; the large pages'
    keys are opposite to the rows where the sizes differ, so that small ones count too."""
    d, page, L = 64, 32, 500
    x, v = randn(1, 1, L + n, d, seed=1), randn(1, 1, L + n, d, seed=2)
    size = torch.tensor(sizes, dtype=torch.float64)[torch.arange(L + n) // page % 3]
    v = (v.double() * 2.0 ** size[:, None]).bfloat16()
    if len(set(sizes)) > 1:
        u = randn(d, seed=3)
        x[0, 0, L:] += 20 * u
        x[0, 0, :L] += torch.where((size[:L] == max(sizes))[:, None], -2 * u, 0.0)
    x = x.bfloat16()
    ref, table, gpu = filled(x, v, page, int8)
    check_attend(ref, table, gpu, x[:, :, L:], L)


@pytest.mark.parametrize("n", [1, 12])
@pytest.mark.parametrize("d,page", [(64, 16), (64, 128), (128, 32)])
@pytest.mark.parametrize("up", [4, 10, 16, 24, 60])
def test_attend_short_rows_beside_a_long_one(up, d, page, n):
    """int8 rows far shorter than the longest of their page are stored as a few steps of its scale or
    none; their logits are those of what is stored, 0 where that is nothing."""
    L = 300
    x, v = randn(1, 2, L + n, d, seed=1), randn(1, 2, L + n, d, seed=2)
    x[:, :, 5:L:page] *= 2.0 ** up
    x, v = x.bfloat16(), v.bfloat16()
    ref, table, gpu = filled(x, v, page, True)
    check_attend(ref, table, gpu, x[:, :, L:], L)


def test_attend_a_tiny_row_beside_a_huge_one():
    """1/||x|| and the page's scale, both near the ends of fp32: the tiny row is stored as zeros."""
    d, page, L = 64, 16, 100
    x, v = randn(1, 1, L + 1, d, seed=1), randn(1, 1, L + 1, d, seed=2)
    x[0, 0, 20] *= 2.0 ** 90
    x[0, 0, 21] *= 2.0 ** -120
    x, v = x.bfloat16(), v.bfloat16()
    ref, table, gpu = filled(x, v, page, True)
    check_attend(ref, table, gpu, x[:, :, L:], L)


@pytest.mark.parametrize("n", [1, 5, 12])
@pytest.mark.parametrize("d,L", [(64, 40), (64, 5000), (128, 300)])
def test_attend_sees_infinite_values(d, L, n):
    """Infinite values that a row sees, early, in the middle and among the new tokens: its sum is
    infinite with their sign, NaN where signs differ or a value is NaN; other dimensions and rows
    before them are as ever."""
    page = 32
    x, v = randn(1, 2, L + n, d, seed=1).bfloat16(), randn(1, 2, L + n, d, seed=2).bfloat16()
    v[0, 0, 3, 7] = math.inf
    v[0, 0, L // 2, 8] = -math.inf
    v[0, 0, 2, 9], v[0, 0, L // 2, 9] = math.inf, -math.inf
    v[0, 0, 4, 10] = math.nan
    v[0, 1, L, 11] = math.inf
    v[0, 1, L + n - 1, 12] = -math.inf
    ref, table, gpu = filled(x, v, page, False)
    out, _ = lb.lsh_cache_attend(gpu, x[:, :, L:].cuda(), table.cuda(), ints(L))
    clean = torch.where(torch.isfinite(v), v, 0.0)
    ref, _, gpu = filled(x, clean, page, False)
    check_attend(ref, table, gpu, x[:, :, L:], L)
    want, _, mag = oc.attend(ref, x[:, :, L:], table, [L])
    # a token's own weight, exp(-1e5), is 0: 0 times infinity is NaN
    want[0, 0, :, 7], want[0, 0, :, 8] = math.inf, -math.inf
    want[0, 0, :, 9] = want[0, 0, :, 10] = math.nan
    want[0, 1, 0, 11], want[0, 1, 1:, 11] = math.nan, math.inf
    want[0, 1, n - 1, 12] = math.nan
    assert torch.equal(torch.isnan(out.cpu()), torch.isnan(want))
    live = ~torch.isnan(want)
    want, mag = want[live], mag[live]
    # E, with ||x|| < 16, is below 2^-15
    near(out.cpu()[live], want, torch.where(torch.isinf(want), 0.0, want.abs()) * 2.0 ** -8 + mag * 2.0 ** -12, "out")


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("page", [16, 64])
def test_append_of_a_row_that_is_not_finite(page, bad):
    """int8: such a row counts with 1/||x|| = 0, as its logit does, and spoils no other token."""
    d, L = 64, 40
    x, v = randn(1, 2, L + 1, d, seed=1).bfloat16(), randn(1, 2, L + 1, d, seed=2).bfloat16()
    x[0, 1, 11, 6] = bad
    x[0, 0, 23, 0], x[0, 0, 23, 1] = bad, 3.0
    ref, table, _ = filled(x, v, page, True)
    gpu = to_gpu(oc.empty(ref["k"].shape[0], 2, page, d, True))
    lb.lsh_cache_append(gpu, x.cuda(), v.cuda(), table.cuda(), ints(0))
    same_cache(gpu, ref)
    for h, t in ((1, 11), (0, 23)):
        assert float(gpu.key_inv_norm[int(table[0, t // page]), h, t % page]) == 0.0
    check_attend(ref, table, gpu, x[:, :, L:], L)
    assert gpu.get_device_status() == 6
    # a bf16 cache holds the row as it is
    ref, table, gpu = filled(x, v, page, False)
    gpu = to_gpu(oc.empty(ref["k"].shape[0], 2, page, d, False))
    lb.lsh_cache_append(gpu, x.cuda(), v.cuda(), table.cuda(), ints(0))
    same_cache(gpu, ref)


@pytest.mark.parametrize("int8", [False, True])
def test_gather_of_no_rows_looks_at_no_page(int8):
    """A sequence that sits a read-back out: its page numbers do not count, wherever it starts."""
    d, page, H = 64, 16, 2
    ref = oc.empty(3, H, page, d, int8, fill=0.5)
    gpu = to_gpu(ref)
    table = torch.tensor([[1, 2], [-1, -1], [-5, 10 ** 6]], dtype=torch.int32)
    x, v = lb.lsh_cache_gather(gpu, table.cuda(), ints(3, 3, 19), 5, n_valid=ints(5, 0, 0))
    assert gpu.get_device_status() == 0
    assert (x[1:] == 0).all() and (v[1:] == 0).all()
    # nor does a page in front of the rows
    table[1] = torch.tensor([-1, 0])
    lb.lsh_cache_gather(gpu, table.cuda(), ints(3, 17, 16), 5, n_valid=ints(5, 2, 0))
    assert gpu.get_device_status() == 0
    table[1, 1] = -1
    lb.lsh_cache_gather(gpu, table.cuda(), ints(3, 17, 16), 5, n_valid=ints(5, 2, 0))
    assert gpu.get_device_status() == 6


@pytest.mark.parametrize("d,page", [(64, 16), (128, 64)])
@pytest.mark.parametrize("at", [0, 5, 15, 20])
def test_append_again_behind_rejected_rows(at, d, page):
    """Drafted rows, one of them large, appended, rejected and overwritten: a scale does not fall
    while its page holds earlier rows, which stay as they were rounded; with none it starts afresh."""
    H, n = 2, 7
    table = table_of(1, 3, 4)
    ref = oc.empty(4, H, page, d, True)
    gpu = to_gpu(ref)
    x, v = (randn(1, H, at + n, d, seed=s).bfloat16() for s in (1, 2))
    big = [t.clone() for t in (x, v)]
    for t in big:
        t[0, :, at + 2] *= 64.0
    calls = [(x[:, :, :at], v[:, :, :at], 0)] if at else []
    calls += [(t[0][:, :, at:at + m], t[1][:, :, at:at + m], at) for t, m in ((big, n), ((x, v), 3), (big, 2))]
    for a, b, start in calls:
        oc.append(ref, a, b, table, [start])
        lb.lsh_cache_append(gpu, a.cuda(), b.cuda(), table.cuda(), ints(start))
        same_cache(gpu, ref)
    if at % page and (at + 2) // page == at // page:
        stored = oc.read(ref, table, 0, 0, at)[0]
        err = (stored - x[0, 0, :at].double()).abs().amax()
        assert float(err) > 64 * 2.0 ** -7  # the rejected row's scale is what they are rounded to


def test_rope_fp32_sines():
    """Rows (1, 0): the sines and cosines themselves. The angle's fraction of a turn is off by
    2 * 2^-32, 2^-28 in the angle; a sine by a step, at most 2^-24, and by the rounding of a sum, 2^-25.
    Together below 2^-23.3."""
    n, d = 40000, 64
    x = torch.zeros(1, 1, n, d)
    x[..., :32] = 1.0
    pos = torch.arange(n, dtype=torch.int32)[None] * 53
    f = freqs_of((64,))
    out = lb.lsh_rope(x.cuda(), pos.cuda(), f.cuda(), axis_dims=(64,))
    t = pos[0, :, None].double() * f.double()
    want = torch.cat([t.cos(), t.sin()], -1)[None, None]
    near(out, want, 2.0 ** -23.3, "sines")


def test_rope_negative_frequencies_at_far_positions():
    """A frequency and its negative turn to the same angle, as exactly: angles of positions up to
    2^31, whose fraction of a turn is off by 2 * 2^-32, sines to 2^-24 and a rounding each."""
    d, n = 64, 64
    g = torch.Generator().manual_seed(1)
    x = randn(1, 1, n, d)
    pos = torch.randint(2 ** 30, 2 ** 31, (1, n), generator=g).int()
    f = -torch.rand(32, generator=g) * 10.0 ** torch.randint(-5, 0, (32,), generator=g).float()
    for adjacent in (False, True):
        for p in (pos, -pos):
            out = lb.lsh_rope(x.cuda(), p.cuda(), f.cuda(), axis_dims=(64,), adjacent=adjacent)
            size = x.double().abs()
            size = size + (size.unflatten(-1, (-1, 2)).flip(-1).flatten(-2) if adjacent else size.roll(32, -1))
            near(out, oc.rope(x, p, f, (64,), adjacent), size * 2.0 ** -22, "out")


def test_rope_does_not_write_heads_over_one_another():
    x = randn(2, 5, 3, 64).bfloat16().cuda()
    pos, f = torch.arange(3, dtype=torch.int32, device=DEV)[None], freqs_of((64,)).cuda()
    base = torch.zeros_like(x)
    with pytest.raises(lb.LshAttnError):
        lb.lsh_rope(x, pos, f, axis_dims=(64,), out=base[:, :1].expand(-1, 5, -1, -1))
    with pytest.raises(lb.LshAttnError):
        lb.lsh_rope(x, pos, f, axis_dims=(64,), out=base[:1].expand(2, -1, -1, -1))
    torch.cuda.synchronize()
    assert (base == 0).all()
