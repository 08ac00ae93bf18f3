"""Rotary positions, the paged cache and attention over it, through the C ABI, against
oracle/cache.py (float64).

Tolerances. A rounding to bf16 is off by at most 2^-8 of the value, one to fp32 by 2^-24.
* Rotation: the fraction of a turn is rounded to fp32 (below 1/2: off by 2^-26 turns, 2 pi 2^-26 =
  2^-23.3 rad), its sine and cosine are good to two steps (2^-23) for fp32 rows and to 2^-21.1, the
  sine unit's bound, for bf16 ones; two products and a sum add 3 * 2^-24 of |lo| + |hi|. Together
  below 2^-21 (fp32) and 2^-20 (bf16) of |lo| + |hi|, then the result's own rounding.
* 1/||x||: a sum of d <= 128 squares in runs of 8 and a tree (at most 16 roundings), a root, a
  product and a quotient: below 20 * 2^-24 of it.
* Attention: a logit's sum of d products is off by d 2^-24 ||x|| (Cauchy-Schwarz with unit keys),
  over sqrt(d): sqrt(d) 2^-24 ||x||; its scalings by 4 * 2^-24 of it. With ||x|| <= 2 sqrt(d) here
  (rows are N(0, 1), d >= 64) that is at most 2 d 2^-24 + 2^-21 < 2^-15 for d = 128. Weights are
  off by twice that, 2^-14, 2^-20 for the exponential, and the sums of up to n terms of one sign
  by less than 2^-14 for the lengths here; the output by 2^-13 of sum p |v| and its own rounding.
* Over an int8 cache a logit's sum starts from -128 sum x and has d / 16 steps, each rounded at that
  size: 9 * 2^-23 * 128 sum |x| <= 9 * 2^-16 sqrt(d) ||x||, over sqrt(d) and the stored key's norm in
  steps (200 and more for the rows here, N(0, 1) in a page whose largest is about 4): below 2^-15 with
  ||x|| < 23. The weights are rounded to f16, 2^-11, so that all together stays below 2^-10 of
  sum p |v|. They are held 2^8 times larger relative to a reference within 2^7 of the row's largest:
  in steps of 2^-24 below 2^-14, so a weight is off by 2^-25-8+7 = 2^-26 of the row's largest besides,
  and the output by 2^-26 sum |v|.
* lse: the logits' 2^-15 (int8 2^-14), 2^-14 for the sum, and the rounding of the result.
"""
import math

import numpy as np
import pytest
import torch

import oracle
from lsh_attention_b200 import binding as lb
from oracle import cache as oc

pytestmark = pytest.mark.gpu

DEV = "cuda"


def randn(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed))


def freqs_of(dims):
    return torch.tensor([10000.0 ** (-2.0 * i / a) for a in dims for i in range(a // 2)])


def near(got, ref, tol, what):
    got, ref, tol = got.detach().double().cpu(), ref.double(), torch.as_tensor(tol, dtype=torch.float64)
    both_inf = torch.isinf(ref) & (got == ref)
    err = torch.where(both_inf, 0.0, (got - ref).abs())
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} off, worst {float((err / tol.clamp(min=1e-300)).max()):.2f} of the bound"


def rope_tol(x, dims, adjacent, eps):
    """2^-21 or 2^-20 (|lo| + |hi|) and the rounding of the result, per element."""
    size = x.double().abs()
    at = 0
    pair = size.clone()
    for d in dims:
        sec = size[..., at:at + d]
        other = (sec.unflatten(-1, (-1, 2)).flip(-1).flatten(-2) if adjacent
                 else sec.roll(d // 2, -1))
        pair[..., at:at + d] = sec + other
        at += d
    # the result is at most |lo| + |hi|
    return pair * ((2.0 ** -21 if x.dtype == torch.float32 else 2.0 ** -20) + eps)


# ------------------------------------------------------------------------------ rotary positions
AXES64 = [(64,), (24, 24, 16), (40,), (16, 12, 12, 8), (2,), (6, 10)]
AXES128 = [(128,), (44, 42, 42), (64, 32, 32), (96,)]


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,dims", [(64, a) for a in AXES64] + [(128, a) for a in AXES128])
def test_rope(d, dims, dtype, adjacent):
    B, H, n = 2, 3, 13
    x = randn(B, H, n, d).to(dtype)
    pos = torch.randint(-50, 3000, (len(dims), B, n), generator=torch.Generator().manual_seed(1),
                        dtype=torch.int32)
    pos[..., 0], pos[..., 1], pos[..., 2] = 0, 2 ** 24 + 1, -(2 ** 27)
    f = freqs_of(dims)
    out = lb.lsh_rope(x.cuda(), pos.cuda(), f.cuda(), axis_dims=dims, adjacent=adjacent)
    tol = rope_tol(x, dims, adjacent, 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24)
    near(out, oc.rope(x, pos, f, dims, adjacent), tol, "out")
    k = sum(dims)
    assert torch.equal(out[..., k:].cpu(), x[..., k:])  # copied, not computed
    back = lb.lsh_rope(x.cuda(), pos.cuda(), f.cuda(), axis_dims=dims, adjacent=adjacent, inverse=True)
    near(back, oc.rope(x, pos, f, dims, adjacent, inverse=True), tol, "inverse")


@pytest.mark.parametrize("n", [1, 2, 255, 1000])
@pytest.mark.parametrize("heads", [1, 5, 9])
def test_rope_layouts(n, heads):
    """Token-major rows, shared positions, in place, and one head's rows for all: the same bits as
    contiguous rows."""
    B, d, dims = 2, 64, (24, 24, 16)
    x = randn(B, n, heads, d).bfloat16().cuda().permute(0, 2, 1, 3)
    pos = torch.stack([torch.arange(n) // 9, torch.arange(n) // 3 % 3, torch.arange(n) % 3]).int().cuda()
    f = freqs_of(dims).cuda()
    base = lb.lsh_rope(x.contiguous(), pos, f, axis_dims=dims)
    assert torch.equal(lb.lsh_rope(x, pos, f, axis_dims=dims), base)
    per_batch = pos[:, None].expand(-1, B, -1).contiguous()
    assert torch.equal(lb.lsh_rope(x, per_batch, f, axis_dims=dims), base)
    out = torch.full((B, n, heads, d), 7.0, device=DEV, dtype=torch.bfloat16).permute(0, 2, 1, 3)
    assert lb.lsh_rope(x, pos, f, axis_dims=dims, out=out) is out
    assert torch.equal(out, base)
    y = x.clone()
    lb.lsh_rope(y, pos, f, axis_dims=dims, out=y)
    assert torch.equal(y, base)
    one = x[:, :1].expand(-1, heads, -1, -1)
    assert torch.equal(lb.lsh_rope(one, pos, f, axis_dims=dims),
                       base[:, :1].expand(-1, heads, -1, -1))
    with pytest.raises(lb.LshAttnError):
        if heads == 1:
            raise lb.LshAttnError(1, "nothing to refuse with one head")
        lb.lsh_rope(x, pos, f, axis_dims=dims, out=base[:, :1].expand(-1, heads, -1, -1))


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("B,H,n", [(3000, 1, 1), (700, 9, 2), (2, 33, 130), (1, 1, 40000)])
def test_rope_many_and_few_tiles(B, H, n, adjacent):
    """More sequences, heads or tiles than blocks: every row is the one that it is alone."""
    d, dims = 64, (40,)
    x = randn(B, H, n, d).bfloat16().cuda()
    pos = (torch.arange(B * n, dtype=torch.int32).view(1, B, n) % 5000).cuda()
    f = freqs_of(dims).cuda()
    out = lb.lsh_rope(x, pos, f, axis_dims=dims, adjacent=adjacent)
    rows = x.transpose(1, 2).reshape(1, 1, B * n * H, d)
    alone = lb.lsh_rope(rows, pos.view(1, -1, 1).expand(-1, -1, H).reshape(1, -1).contiguous(), f,
                        axis_dims=dims, adjacent=adjacent)
    assert torch.equal(out, alone.view(B, n, H, d).transpose(1, 2))
    few = torch.randint(0, B * n, (20,), generator=torch.Generator().manual_seed(0))
    b, t = few // n, few % n
    got, src = out[b.cuda(), :, t.cuda()].cpu(), x[b.cuda(), :, t.cuda()].cpu()
    want = oc.rope(src[:, :, None], pos[0, b.cuda(), t.cuda()].cpu().view(1, 20, 1), f.cpu(), dims, adjacent)
    near(got, want[:, :, 0], rope_tol(src, dims, adjacent, 2.0 ** -8), "rows")


def test_rope_gradient_against_differences():
    """The map is linear: the difference along any direction is the map of the direction, so the
    gradient of sum(g * rope(x)) along e is <g, rope(e)>."""
    B, H, n, d, dims = 1, 2, 7, 64, (24, 24, 16)
    pos = torch.randint(0, 64, (3, n), dtype=torch.int32).cuda()
    f = freqs_of(dims).cuda()
    g = randn(B, H, n, d, seed=1).cuda()
    grad = lb.lsh_rope(g, pos, f, axis_dims=dims, inverse=True)
    for s in range(8):
        e = randn(B, H, n, d, seed=10 + s).cuda()
        step = lb.lsh_rope(e, pos, f, axis_dims=dims)
        a, b = (g.double() * step.double()).sum(), (grad.double() * e.double()).sum()
        # every element off by 2^-20 of its pair's size at most
        size = 2 * 2.0 ** -20 * (g.double().abs().sum() * e.double().abs().max())
        assert abs(a - b) <= size


def test_rope_infinities_stay_in_their_pair():
    d, dims = 64, (16, 8)
    x = randn(1, 1, 4, d)
    x[0, 0, 1, 3], x[0, 0, 2, 40], x[0, 0, 3, 41] = math.inf, math.nan, -math.inf
    pos = torch.arange(8, dtype=torch.int32).view(2, 4)
    out = lb.lsh_rope(x.cuda(), pos.cuda(), freqs_of(dims).cuda(), axis_dims=dims).cpu()
    clean = torch.isfinite(out)
    assert not clean[0, 0, 1, 3] and not clean[0, 0, 1, 11]
    assert torch.isnan(out[0, 0, 2, 40]) and out[0, 0, 3, 41] == -math.inf
    assert int((~clean).sum()) == 4


# ------------------------------------------------------------------------------ the cache
def table_of(B, per_seq, pages, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randperm(pages, generator=g)[:B * per_seq].view(B, per_seq).int()


def to_gpu(c):
    return lb.LshCache(*[None if t is None else t.cuda()
                         for t in (c["k"], c["v"], c["key_inv_norm"], c["k_scale"], c["v_scale"])])


def bits(t):
    return t.cpu().view(torch.int16 if t.dtype == torch.bfloat16 else
                        torch.int32 if t.dtype == torch.float32 else torch.int8)


def same_cache(gpu, ref, kinv=True):
    """Every slot as the oracle has it, those never written included; 1/||x|| within its bound."""
    assert torch.equal(bits(gpu.k), bits(ref["k"]))
    assert torch.equal(bits(gpu.v), bits(ref["v"]))
    if gpu.int8:
        assert torch.equal(bits(gpu.k_scale), bits(ref["k_scale"]))
        assert torch.equal(bits(gpu.v_scale), bits(ref["v_scale"]))
    got, want = gpu.key_inv_norm.cpu(), ref["key_inv_norm"]
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    live = ~torch.isnan(want)
    near(got[live], want[live].double(), want[live].double().abs() * 20 * 2.0 ** -24, "1/||x||")


PIECES = [  # rows appended one call after the other, and how many of a padded call are valid
    [(1, None)], [(1, None)] * 18, [(16, None), (1, None), (33, None)], [(5, [5, 0, 2]), (9, [1, 9, 7])],
    [(70, [70, 3, 0]), (1, None), (60, None), (2, [0, 2, 1])],
]


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("d,page", [(64, 16), (64, 64), (128, 32), (128, 128)])
@pytest.mark.parametrize("pieces", range(len(PIECES)))
def test_append(d, page, int8, pieces):
    """Rows enter as given; int8 scales grow and earlier rows are rounded again; nothing else in
    the pool changes. Bit for bit."""
    B, H = 3, 2
    total = sum(n for n, _ in PIECES[pieces])
    per_seq = total // page + 1
    table = table_of(B, per_seq, B * per_seq + 2)
    ref = oc.empty(B * per_seq + 2, H, page, d, int8)
    gpu = to_gpu(ref)
    at = [0] * B
    for i, (n, valid) in enumerate(PIECES[pieces]):
        x, v = (randn(B, n, H, d, seed=2 * i + s) * 2.0 ** (i % 5 - 2 * s) for s in (0, 1))
        x, v = (t.bfloat16().permute(0, 2, 1, 3) for t in (x, v))
        x[0, 0, 0] = 0
        oc.append(ref, x, v, table, at, valid)
        seq = torch.tensor(at, dtype=torch.int32).cuda()
        nv = None if valid is None else torch.tensor(valid, dtype=torch.int32).cuda()
        x, v = x.cuda(), v.cuda()
        got = lb.lsh_cache_append(gpu, x, v, table.cuda(), seq, n_valid=nv)
        assert got is x
        at = [a + (n if valid is None else valid[b]) for b, a in enumerate(at)]
        same_cache(gpu, ref)
    assert gpu.get_device_status() == 0


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 64), (64, 128), (128, 128)])
@pytest.mark.parametrize("n", [2, 5, 16, 17, 18])
def test_append_few_rows_across_a_page_end(n, d, page, int8):
    """A handful of rows that begin in one page and end in the next, at every place of it. Bit for
    bit, in the slots behind them too."""
    H = 2
    lens = sorted({page - 1, page - 2, page - n + 1, page - n, page - n - 1, page - 16, 2 * page - 3} -
                  {p for p in range(-32, 0)})
    B = len(lens)
    table = table_of(B, 3, 3 * B + 1)
    ref = oc.empty(3 * B + 1, H, page, d, int8)
    gpu = to_gpu(ref)
    for i, (at, m) in enumerate([([0] * B, max(lens)), (lens, n)]):
        x, v = (randn(B, H, m, d, seed=2 * i + s).bfloat16() * 2.0 ** i for s in (0, 1))
        valid = lens if i == 0 else None
        oc.append(ref, x, v, table, at, valid)
        seq = torch.tensor(at, dtype=torch.int32).cuda()
        nv = None if valid is None else torch.tensor(valid, dtype=torch.int32).cuda()
        lb.lsh_cache_append(gpu, x.cuda(), v.cuda(), table.cuda(), seq, n_valid=nv)
        same_cache(gpu, ref)
    assert gpu.get_device_status() == 0


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("d,dims,adjacent", [(64, (24, 24, 16), False), (64, (40,), True),
                                             (128, (128,), True), (128, (128,), False),
                                             (128, (44, 42, 42), False), (64, (16, 12, 12, 8), False)])
def test_append_rotates(d, dims, adjacent, int8):
    """Appending with a rotation is lsh_rope and appending its rows, bit for bit, but for the norm,
    which is that of the row as given."""
    B, H, n, page = 2, 3, 45, 32
    per_seq = 3
    table = table_of(B, per_seq, 8).cuda()
    x, v = randn(B, H, n, d).bfloat16(), randn(B, H, n, d, seed=1).bfloat16()
    pos = torch.randint(0, 100000, (len(dims), B, n), generator=torch.Generator().manual_seed(3)).int()
    f = freqs_of(dims)
    seq = torch.tensor([7, 30], dtype=torch.int32).cuda()
    nv = torch.tensor([45, 31], dtype=torch.int32)
    a, b = (to_gpu(oc.empty(8, H, page, d, int8, fill=0.5)) for _ in range(2))
    kw = dict(axis_dims=dims, adjacent=adjacent)
    xr = lb.lsh_cache_append(a, x.cuda(), v.cuda(), table, seq, n_valid=nv.cuda(), positions=pos.cuda(),
                             freqs=f.cuda(), **kw)
    rows = lb.lsh_rope(x.cuda(), pos.cuda(), f.cuda(), **kw)
    live = (torch.arange(n) < nv[:, None])[:, None, :, None]
    assert torch.equal(xr, torch.where(live.cuda(), rows, 0.0))
    near(xr, torch.where(live, oc.rope(x, pos, f, dims, adjacent), 0.0),
         rope_tol(x, dims, adjacent, 2.0 ** -8), "rotated rows")
    lb.lsh_cache_append(b, rows, v.cuda(), table, seq, n_valid=nv.cuda())
    assert torch.equal(bits(a.k), bits(b.k)) and torch.equal(bits(a.v), bits(b.v))
    if int8:
        assert torch.equal(a.k_scale, b.k_scale) and torch.equal(a.v_scale, b.v_scale)
    for s in range(B):
        for t in range(int(nv[s])):
            p = int(seq[s]) + t
            got = a.key_inv_norm[int(table[s, p // page]), :, p % page]
            want = 1 / x[s, :, t].double().norm(dim=-1)
            near(got, want, want * 20 * 2.0 ** -24, "1/||x||")
    # the rows may be turned where they lie
    c = to_gpu(oc.empty(8, H, page, d, int8, fill=0.5))
    y = x.cuda()
    assert lb.lsh_cache_append(c, y, v.cuda(), table, seq, n_valid=nv.cuda(), positions=pos.cuda(),
                               freqs=f.cuda(), xr=y, **kw) is y
    assert torch.equal(y, xr) and torch.equal(bits(a.k), bits(c.k))


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("n", [1, 6, 17, 40])
@pytest.mark.parametrize("d,page", [(64, 128), (128, 64)])
def test_append_rotates_across_a_page_end(d, page, n, int8):
    """A few rows behind others, turned on the way or before: the same cache, bit for bit."""
    B, H, dims = 3, 5, (24, 24, 16)
    table = table_of(B, 3, 10).cuda()
    x, v = randn(B, H, n, d).bfloat16().cuda(), randn(B, H, n, d, seed=1).bfloat16().cuda()
    pos = torch.randint(0, 100000, (3, B, n), generator=torch.Generator().manual_seed(3)).int().cuda()
    f = freqs_of(dims).cuda()
    seq = torch.tensor([page - 1, page - 5, 2 * page - 16], dtype=torch.int32).cuda()
    a, b = (to_gpu(oc.empty(10, H, page, d, int8, fill=0.5)) for _ in range(2))
    xr = lb.lsh_cache_append(a, x, v, table, seq, positions=pos, freqs=f, axis_dims=dims)
    rows = lb.lsh_rope(x, pos, f, axis_dims=dims)
    lb.lsh_cache_append(b, rows, v, table, seq)
    assert torch.equal(xr, rows)
    assert torch.equal(bits(a.k), bits(b.k)) and torch.equal(bits(a.v), bits(b.v))
    if int8:
        assert torch.equal(a.k_scale, b.k_scale) and torch.equal(a.v_scale, b.v_scale)


def test_append_extremes():
    """Short and long rows: the norm's squares neither vanish nor overflow; int8 scales reach both
    ends; infinities and NaN are held at the ends of the range and reported."""
    H, d, page = 1, 64, 16
    x = randn(1, H, 6, d)
    scale = [2.0 ** -100, 2.0 ** 100, 2.0 ** -130, 2.0 ** 120, 1.0, 0.0]
    x = (x * torch.tensor(scale)[:, None]).bfloat16()
    for int8 in (False, True):
        for t in range(6):
            ref = oc.empty(2, H, page, d, int8)
            gpu = to_gpu(ref)
            table = torch.tensor([[1]], dtype=torch.int32)
            row = x[:, :, t:t + 1]
            oc.append(ref, row, row, table, [0])
            lb.lsh_cache_append(gpu, row.cuda(), row.cuda(), table.cuda(),
                                torch.zeros(1, dtype=torch.int32, device=DEV))
            same_cache(gpu, ref)
            for got, want in zip(lb.lsh_cache_gather(gpu, table.cuda(), torch.zeros(1, dtype=torch.int32, device=DEV), 1),
                                 oc.read(ref, table, 0, 0, 1)):
                assert torch.equal(got[0, 0].double().cpu(), want)
            assert gpu.get_device_status() == 0
    ref = oc.empty(2, H, page, d, True)
    gpu = to_gpu(ref)
    row = x[:, :, 4:5].clone()
    row[..., 0], row[..., 1], row[..., 2] = math.inf, -math.inf, math.nan
    oc.append(ref, row, row, table, [0], x=x[:, :, 4:5])
    lb.lsh_cache_append(gpu, row.cuda(), row.cuda(), table.cuda(), torch.zeros(1, dtype=torch.int32, device=DEV))
    assert torch.equal(gpu.k.cpu(), ref["k"]) and torch.equal(gpu.v.cpu(), ref["v"])
    assert gpu.k[1, 0, 0, :3].tolist() == [127, -127, 0]
    assert gpu.get_device_status() == 6
    gpu.clear_status()
    assert gpu.get_device_status() == 0


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 64), (64, 128)])
@pytest.mark.parametrize("n", [1, 15, 50])
def test_gather(d, page, int8, n):
    B, H, pages = 3, 2, 40
    c = oc.empty(pages, H, page, d, int8)
    for name in ("k", "v"):
        t = randn(*c[name].shape, seed=ord(name))
        c[name] = (t * 40).round().clamp(-127, 127).to(torch.int8) if int8 else t.bfloat16()
        if int8:
            c[name + "_scale"] = 2.0 ** torch.randint(-20, 20, (pages, H)).float()
    gpu = to_gpu(c)
    per_seq = 160 // page + 1
    table = table_of(B, per_seq, pages)
    start, valid = [0, 77, 13], [n, max(0, n - 3), n // 2]
    x, v = lb.lsh_cache_gather(gpu, table.cuda(), torch.tensor(start, dtype=torch.int32).cuda(), n,
                               n_valid=torch.tensor(valid, dtype=torch.int32).cuda())
    out = torch.empty(B, n, H, d, dtype=torch.bfloat16, device=DEV).permute(0, 2, 1, 3)
    v2 = torch.empty_like(out)
    lb.lsh_cache_gather(gpu, table.cuda(), torch.tensor(start, dtype=torch.int32).cuda(), n,
                        n_valid=torch.tensor(valid, dtype=torch.int32).cuda(), x=out, v=v2)
    assert torch.equal(out, x) and torch.equal(v2, v)
    c["key_inv_norm"].zero_()
    for b in range(B):
        for h in range(H):
            k_ref, v_ref, _ = oc.read(c, table, b, h, start[b] + n)
            for got, ref in ((x, k_ref), (v, v_ref)):
                ref = ref[start[b]:].clone()
                ref[valid[b]:] = 0
                assert torch.equal(got[b, h].double().cpu(), ref)


# ------------------------------------------------------------------------------ attention
def filled(B, H, d, page, int8, lens, n, seed=0, spread=1.0):
    """A cache holding `lens` tokens of each sequence and n more, its table, and the last n rows."""
    total = max(lens) + n
    per_seq = total // page + 1
    pages = B * per_seq + 1
    ref = oc.empty(pages, H, page, d, int8)
    table = table_of(B, per_seq, pages, seed)
    x, v = (randn(B, H, total, d, seed=seed + s) for s in (1, 2))
    if spread != 1.0:  # values of very different sizes, page by page
        v = v * spread ** (torch.arange(total) // page % 3)[:, None]
    x, v = x.bfloat16(), v.bfloat16()
    oc.append(ref, x, v, table, [0] * B, [l + n for l in lens])
    q = torch.stack([x[b, :, l:l + n] for b, l in enumerate(lens)])
    return ref, table, q


def check_attend(gpu, ref, table, q, lens, valid=None, **kw):
    seq = torch.tensor(lens, dtype=torch.int32).cuda()
    nv = None if valid is None else torch.tensor(valid, dtype=torch.int32).cuda()
    out, lse = lb.lsh_cache_attend(gpu, q.cuda(), table.cuda(), seq, n_valid=nv, **kw)
    ro, rl, mag = oc.attend(ref, q, table, lens, valid)
    near(out, ro, ro.abs() * 2.0 ** -8 + mag * (2.0 ** -13 if ref["k_scale"] is None else 2.0 ** -10), "out")
    near(lse, rl, 2.0 ** -13 + torch.where(torch.isinf(rl), 0.0, rl.abs()) * 2.0 ** -23, "lse")
    return out, lse


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("d,page", [(64, 16), (64, 128), (128, 32), (128, 64)])
@pytest.mark.parametrize("lens,n,valid", [
    ([0], 1, None),                          # alone: its own value, lse -1e5
    ([1, 15, 16], 1, None), ([127, 128, 300], 1, None),
    ([0, 5, 63], 3, None), ([200, 0, 31], 8, [8, 0, 5]), ([10, 129, 64], 9, [9, 1, 8]),
    ([33, 100], 17, None), ([5, 120], 11, [11, 4]), ([0, 77], 33, [20, 33]), ([128, 250], 16, None),
])
def test_attend(d, page, int8, lens, n, valid):
    ref, table, q = filled(len(lens), 2, d, page, int8, lens, n)
    gpu = to_gpu(ref)
    out, lse = check_attend(gpu, ref, table, q, lens, valid)
    again = lb.lsh_cache_attend(gpu, q.cuda(), table.cuda(), torch.tensor(lens).int().cuda(),
                                n_valid=None if valid is None else torch.tensor(valid).int().cuda())
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    assert gpu.get_device_status() == 0


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("B,H,d,page,lens,n", [
    (1, 1, 128, 64, [4999], 1), (1, 3, 64, 16, [2601], 5), (5, 2, 64, 32, [1, 2000, 640, 3, 1029], 2),
    (40, 1, 64, 16, [(37 * i) % 90 for i in range(40)], 1), (1, 2, 128, 128, [1500], 16),
])
def test_attend_long_and_many(B, H, d, page, lens, n, int8):
    """Keys shared out over the card and joined; sequences far more than blocks' worth of work and
    far less."""
    ref, table, q = filled(B, H, d, page, int8, lens, n, seed=5)
    check_attend(to_gpu(ref), ref, table, q, lens)


def random_cache(B, H, d, page, int8, lens, n, seed=3):
    """A cache filled at random (as tensors, quickly), its table, and n rows of x."""
    total = max(lens) + n
    per_seq = total // page + 1
    pages = B * per_seq + 1
    c = {"k": randn(pages, H, page, d, seed=seed), "v": randn(pages, H, page // 16, d, 16, seed=seed + 1),
         "k_scale": None, "v_scale": None}
    c["key_inv_norm"] = 1.0 / c["k"].norm(dim=-1)
    for name in ("k", "v"):
        if int8:
            c[name] = (c[name] * 25).round().clamp(-127, 127).to(torch.int8)
            c[name + "_scale"] = 2.0 ** torch.randint(-6, -3, (pages, H)).float()
        else:
            c[name] = c[name].bfloat16()
    return c, table_of(B, per_seq, pages, seed), randn(B, H, n, d, seed=seed + 2).bfloat16()


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("B,H,d,page,lens,n", [
    (3, 16, 128, 64, [3000, 2500, 3100], 1),              # the ring turns over many times in a block
    (4, 16, 64, 32, [9000, 11, 7000, 8999], 3),
    (64, 16, 64, 16, [(53 * i) % 130 for i in range(64)], 2),  # segments of one to a few units
    (64, 16, 128, 128, [(29 * i) % 200 for i in range(64)], 9),
    (2, 2, 64, 64, [40000, 33333], 1),
])
def test_attend_work_of_every_shape(B, H, d, page, lens, n, int8):
    ref, table, q = random_cache(B, H, d, page, int8, lens, n)
    valid = None if n == 1 else [(n + b) % (n + 1) for b in range(B)]
    check_attend(to_gpu(ref), ref, table, q, lens, valid)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("B,n,lens,valid", [
    (3, 4, [5, 0, 90], [0, 0, 0]),                                   # no row at all
    (70, 2, [7 * i for i in range(70)], [0] * 40 + [2] + [0] * 28 + [1]),  # long runs of none
    (1, 300, [50], [290]),                                           # many row groups
    (2, 16, [0, 3], [16, 15]),
])
def test_attend_few_rows_of_many(B, n, lens, valid, int8):
    ref, table, q = random_cache(B, 2, 64, 32, int8, lens, n, seed=9)
    out, lse = check_attend(to_gpu(ref), ref, table, q, lens, valid)
    for b in range(B):
        assert (out[b, :, valid[b]:] == 0).all() and torch.isneginf(lse[b, :, valid[b]:]).all()


@pytest.mark.parametrize("int8", [False, True])
def test_attend_values_of_different_sizes(int8):
    """Pages whose scales differ by 2^12 and 2^24."""
    lens = [150, 40]
    ref, table, q = filled(2, 2, 64, 16, int8, lens, 2, spread=4096.0)
    check_attend(to_gpu(ref), ref, table, q, lens)


def test_attend_sharp_and_flat_rows():
    """Logits far apart (one key takes all the weight, late or early) and all alike."""
    H, d, page, L = 1, 64, 16, 300
    x = randn(1, H, L + 2, d)
    x[0, 0, L] *= 60.0       # logits up to hundreds
    x[0, 0, 7] = x[0, 0, L]  # its best key comes early
    x[0, 0, L + 1] = 0.0     # a zero row: every logit 0
    x[0, 0, 11] = 0.0        # a zero key: logit 0
    x = x.bfloat16()
    v = randn(1, H, L + 2, d, seed=1).bfloat16()
    for int8 in (False, True):
        ref = oc.empty(20, H, page, d, int8)
        table = table_of(1, 19, 20)
        oc.append(ref, x, v, table, [0])
        gpu = to_gpu(ref)
        q = x[:, :, L:]
        out, lse = lb.lsh_cache_attend(gpu, q.cuda(), table.cuda(), torch.tensor([L]).int().cuda())
        ro, rl, mag = oc.attend(ref, q, table, [L])
        # the derived bound with ||x|| = 60 * 2 sqrt(d): 60 times the logits' share
        small = 2.0 ** -26 * oc.read(ref, table, 0, 0, L + 2)[1].abs().sum(0) if int8 else 0.0
        near(out, ro, ro.abs() * 2.0 ** -8 + mag * (60 * 2.0 ** -13 + 2.0 ** -11) + small, "out")
        near(lse, rl, 60 * 2.0 ** -13 + rl.abs() * 2.0 ** -23, "lse")


@pytest.mark.parametrize("n", [5, 12])
def test_attend_does_not_see_what_is_masked(n):
    """Slots past the sequence hold NaN, a later token's value and key infinities: a row sees
    neither; a NaN query spoils its own row only."""
    lens = [45]
    ref, table, q = filled(1, 2, 64, 16, False, lens, n)
    page, slot = int(table[0, 48 // 16]), 48 % 16
    ref["v"][page, :, 0, :, slot] = math.inf
    ref["k"][page, :, slot, 3] = -math.inf
    ref["v"][page, :, 0, 5, slot] = math.nan
    gpu = to_gpu(ref)
    q[0, 1, 1] = math.nan
    out, lse = lb.lsh_cache_attend(gpu, q.cuda(), table.cuda(), torch.tensor(lens).int().cuda())
    ro, rl, mag = oc.attend(ref, q, table, lens)
    for h, t in ((0, 0), (0, 1), (0, 2), (1, 0), (1, 2)):
        near(out[0, h, t], ro[0, h, t], ro[0, h, t].abs() * 2.0 ** -8 + mag[0, h, t] * 2.0 ** -13, "out")
        near(lse[0, h, t], rl[0, h, t], 2.0 ** -12, "lse")
    assert torch.isnan(out[0, 1, 1]).all()
    assert not torch.isfinite(out[0, :, 4:]).any()  # see the infinite key and value


def test_bad_tables_are_reported_and_skipped():
    lens, n = [40, 20, 33, 5], 2
    ref, table, q = filled(4, 2, 64, 16, False, lens, n)
    bad = table.clone()
    bad[0, 1] = 10 ** 6      # a middle page of sequence 0
    bad[1, :] = -3           # every page of sequence 1
    seq, nv = torch.tensor([40, 20, -1, 5]).int().cuda(), torch.tensor([2, 2, 2, 3]).int().cuda()
    gpu = to_gpu(ref)
    out, lse = lb.lsh_cache_attend(gpu, q.cuda(), bad.cuda(), seq, n_valid=nv)
    assert gpu.get_device_status() == 6
    # sequence 0 without the tokens of its bad page
    for h in range(2):
        k, v, kinv = oc.read(ref, table, 0, h, 42)
        for t in range(2):
            l = (k[:41 + t] @ q[0, h, t].double()) * kinv[:41 + t] / 8
            l[40 + t], l[16:32] = oc.SELF_LOGIT, -math.inf
            w = torch.softmax(l, 0)
            o = w @ v[:41 + t]
            near(out[0, h, t], o, o.abs() * 2.0 ** -8 + (w @ v[:41 + t].abs()) * 2.0 ** -13, "out")
    assert (out[1:] == 0).all() and (lse[1:] == -math.inf).all()
    gpu.clear_status()
    before = bits(gpu.k).clone(), bits(gpu.v).clone()
    x = randn(4, 2, n, 64, seed=9).bfloat16().cuda()
    bad[0, 2], bad[3, 0] = -1, 10 ** 6
    xr = lb.lsh_cache_append(gpu, x, x, bad.cuda(), seq, n_valid=nv, xr=torch.empty_like(x))
    assert gpu.get_device_status() == 6
    assert torch.equal(before[0], bits(gpu.k)) and torch.equal(before[1], bits(gpu.v))
    assert torch.equal(xr[:2], x[:2]) and (xr[2:] == 0).all()
    gpu.clear_status()
    a, b = lb.lsh_cache_gather(gpu, bad.cuda(), torch.tensor([8, 0, 0, 1000]).int().cuda(), 12)
    assert gpu.get_device_status() == 6
    k0 = oc.read(ref, table, 0, 0, 16)[0]
    assert torch.equal(a[0, 0, :8].double().cpu(), k0[8:]) and (a[0, :, 8:] == 0).all()
    assert (a[1] == 0).all() and (b[1] == 0).all() and (a[3] == 0).all()


@pytest.mark.parametrize("int8", [False, True])
def test_far_pages(int8):
    """Page numbers whose offsets pass 2^31 elements."""
    H, page, d = 8, 128, 128
    pages = 17000 if int8 else 16500
    cache = lb.LshCache.empty(pages, H, page, d, int8=int8)
    assert cache.k.numel() > 2 ** 31
    table = torch.tensor([[pages - 1, pages - 7]], dtype=torch.int32)
    x, v = randn(1, H, 140, d).bfloat16(), randn(1, H, 140, d, seed=1).bfloat16()
    zero = torch.zeros(1, dtype=torch.int32, device=DEV)
    lb.lsh_cache_append(cache, x.cuda(), v.cuda(), table.cuda(), zero)
    ref = oc.empty(2, H, page, d, int8, fill=0.0)
    oc.append(ref, x, v, torch.tensor([[0, 1]]), [0])
    ids = table[0].long().cuda()
    assert torch.equal(cache.k[ids[0]].cpu(), ref["k"][0]) and torch.equal(cache.v[ids[0]].cpu(), ref["v"][0])
    q = x[:, :, 139:]
    out, lse = lb.lsh_cache_attend(cache, q.cuda(), table.cuda(), zero + 139)
    ro, rl, mag = oc.attend(ref, q, torch.tensor([[0, 1]]), [139])
    near(out, ro, ro.abs() * 2.0 ** -8 + mag * (2.0 ** -10 if int8 else 2.0 ** -13), "out")
    a, b = lb.lsh_cache_gather(cache, table.cuda(), zero, 140)
    k0, v0, _ = oc.read(ref, torch.tensor([[0, 1]]), 0, 3, 140)
    assert torch.equal(a[0, 3].double().cpu(), k0) and torch.equal(b[0, 3].double().cpu(), v0)


# ------------------------------------------------------------------------------ together
@pytest.mark.parametrize("int8", [False, True])
def test_generating_is_the_dense_attention_of_the_whole(int8):
    """A prompt rotated, attended densely and appended; then tokens one by one and a few at a time:
    every row is that of dense causal attention over the whole rotated sequence."""
    H, d, page, dims = 2, 64, 32, (24, 24, 16)
    n0, steps = 77, [1, 1, 4, 1, 3]
    n = n0 + sum(steps)
    x, v = randn(1, H, n, d).bfloat16(), randn(1, H, n, d, seed=1).bfloat16()
    t = torch.arange(n)
    pos = torch.stack([t // 12, t // 3 % 4, t % 3]).int()
    f = freqs_of(dims)
    rows = lb.lsh_rope(x.cuda(), pos.cuda(), f.cuda(), axis_dims=dims)
    cache = lb.LshCache.empty(6, H, page, d, int8=int8)
    table = torch.tensor([[4, 1, 5, 0]], dtype=torch.int32).cuda()
    seq = torch.zeros(1, dtype=torch.int32, device=DEV)
    dense, dense_lse = lb.lsh_attn_dense_forward(rows, v.cuda(), causal=True)
    at = 0
    for m in [n0] + steps:
        sl = slice(at, at + m)
        xr = lb.lsh_cache_append(cache, x[:, :, sl].cuda(), v[:, :, sl].cuda(), table, seq,
                                 positions=pos[:, sl].contiguous().cuda(), freqs=f.cuda(), axis_dims=dims)
        assert torch.equal(xr, rows[:, :, sl])
        out, lse = lb.lsh_cache_attend(cache, xr, table, seq)
        if int8:
            # a stored value is within a step s <= 2 max / 127 < 0.08 of the row; a key's steps
            # move its logit by at most ||x|| s sqrt(d) / (||x_j|| sqrt(d)) < 0.08 * 1.25 = 0.1, the
            # lse by as much and the weights by twice that, the output by 0.2 of sum p |v| < 1.5
            # and by the values' own 0.08
            tol, tol_lse = 0.38, 0.1
        else:
            # both round P V's result to bf16, the dense kernel its weights too
            tol, tol_lse = 4 * 2.0 ** -8 * 1.5 + 2.0 ** -7, 2.0 ** -7
        err = (out.float() - dense[:, :, sl].float()).abs()
        assert float(err.max()) <= tol
        assert float((lse - dense_lse[:, :, sl]).abs().max()) <= tol_lse
        seq += m
        at += m
    assert cache.get_device_status() == 0
    xs, vs = lb.lsh_cache_gather(cache, table, torch.zeros_like(seq), 64)
    if not int8:
        assert torch.equal(xs, rows[:, :, :64]) and torch.equal(vs, v[:, :, :64].cuda())
        buckets = torch.zeros(1, H, 1, 64, dtype=torch.int32, device=DEV)
        a, _ = lb.lsh_attn_forward(xs, vs, n_buckets=2, chunk=64, causal=True, buckets=buckets)
        # one bucket, one chunk: dense attention over the cached rows
        assert float((a.float() - dense[:, :, :64].float()).abs().max()) <= 4 * 2.0 ** -8 * 1.5 + 2.0 ** -7


@pytest.mark.parametrize("int8", [False, True])
def test_captured_step_follows_its_tables(int8):
    """One captured step, append and attend, replayed as lengths, pages and rows change; an eager
    call between the replays leaves it alone."""
    H, d, page, dims = 2, 64, 16, (64,)
    B = 2
    n = 40
    x, v = randn(B, H, n, d).bfloat16(), randn(B, H, n, d, seed=1).bfloat16()
    f = freqs_of(dims).cuda()
    table = table_of(B, 3, 7).cuda()
    ref, cache = (lb.LshCache.empty(7, H, page, d, int8=int8) for _ in range(2))
    xs, vs = (torch.empty(B, H, 1, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    pos, seq = torch.zeros(1, 1, dtype=torch.int32, device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV)

    def step(c):
        xr = lb.lsh_cache_append(c, xs, vs, table, seq, positions=pos, freqs=f, axis_dims=dims)
        return lb.lsh_cache_attend(c, xr, table, seq)

    xs.copy_(x[:, :, :1])
    vs.copy_(v[:, :, :1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(cache)
    torch.cuda.current_stream().wait_stream(s)
    g, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = step(cache)
    with torch.cuda.graph(g2):  # a second graph beside it
        out2, lse2 = step(cache)
    for t in range(n):
        xs.copy_(x[:, :, t:t + 1])
        vs.copy_(v[:, :, t:t + 1])
        pos.fill_(t)
        seq.fill_(t)
        g.replay()
        a, b = step(ref)
        assert torch.equal(out, a) and torch.equal(lse, b), t
        g2.replay()
        assert torch.equal(out2, a) and torch.equal(lse2, b), t
    for a, b in zip(*(lb.lsh_cache_gather(c, table, torch.zeros_like(seq), n) for c in (cache, ref))):
        assert torch.equal(a, b)


def test_on_another_stream():
    """With `stream`, everything runs there: results are right once it is waited for."""
    lens = [500]
    ref, table, q = filled(1, 2, 64, 16, False, lens, 1)
    gpu = to_gpu(ref)
    x, tab, seq = q.cuda(), table.cuda(), torch.tensor(lens).int().cuda()
    want = lb.lsh_cache_attend(gpu, x, tab, seq)
    f = freqs_of((64,)).cuda()
    pos = torch.tensor([[5]], dtype=torch.int32).cuda()
    want_r = lb.lsh_rope(x, pos, f, axis_dims=(64,))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = lb.lsh_cache_attend(gpu, x, tab, seq, stream=s)
    got_r = lb.lsh_rope(x, pos, f, axis_dims=(64,), stream=s)
    back = lb.lsh_cache_gather(gpu, tab, seq, 1, stream=s)
    lb.lsh_cache_append(gpu, x, x, tab, seq, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(got_r, want_r)
    assert torch.equal(back[0], x)
    assert torch.equal(lb.lsh_cache_gather(gpu, tab, seq, 1)[1], x)
