"""The rotary, cache and cached-attention operators: cases, inputs and plain forms.

Four kinds of case, one for each entry point:

* ``rope``   -- rotary positions of one to four axes on the rows of x, or their gradient;
* ``append`` -- new rows of x and v into a paged cache (bf16, or 8 bits with a scale for
  each page and head), rotated on the way;
* ``gather`` -- rows of the cache back as [B, H, n, d];
* ``attend`` -- shared-QK attention of new tokens over the cache.

A cache holds, for each page and head, the rows of x as [page_size, d], the rows of v as
[page_size / 16, d, 16] (groups of 16 tokens, dimension-major), 1/||x|| of every row and,
in 8 bits, one power-of-two scale each for x and v.
"""
import math

import torch

own = False

SELF = -1.0e5  # logit of a token against itself


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # the image workload's whole batch before its attention: row, column and channel axes
        {"name": "rope-image-12k", "kind": "rope", "batch": 8, "heads": 8, "n": 12288, "d": 64,
         "axes": "24,24,16", "adjacent": False, "inverse": False, "dtype": "bf16",
         "tokens_first": False, "offset": 0},
        # the gradient of the long text's rotation, handed on in the projections' token-major layout
        {"name": "rope-text-gradient", "kind": "rope", "batch": 1, "heads": 8, "n": 65536, "d": 128,
         "axes": "128", "adjacent": True, "inverse": True, "dtype": "bf16", "tokens_first": True,
         "offset": 0},
        # one short fp32 sequence at far positions, part of the dimensions rotated: latency
        {"name": "rope-small-far", "kind": "rope", "batch": 1, "heads": 1, "n": 1023, "d": 64,
         "axes": "40", "adjacent": False, "inverse": False, "dtype": "f32", "tokens_first": False,
         "offset": 5000000},
        # four prompts enter an empty bf16 cache
        {"name": "append-prompt", "kind": "append", "batch": 4, "heads": 8, "d": 128, "page": 64,
         "format": "bf16", "new": 8192, "ragged": False, "lo": 0, "hi": 0, "axes": "128",
         "adjacent": True, "tokens_first": True},
        # a padded batch of prompts continues sequences of an 8-bit cache, pages half full
        {"name": "append-chunk-i8", "kind": "append", "batch": 8, "heads": 8, "d": 64, "page": 32,
         "format": "i8", "new": 2000, "ragged": True, "lo": 500, "hi": 4001, "axes": "24,24,16",
         "adjacent": False, "tokens_first": True},
        # the generating step of 64 sequences: one token each
        {"name": "append-token-i8", "kind": "append", "batch": 64, "heads": 8, "d": 64, "page": 64,
         "format": "i8", "new": 1, "ragged": False, "lo": 1, "hi": 12287, "axes": "24,24,16",
         "adjacent": False, "tokens_first": True},
        # a long cached sequence read back for a forward pass over all of it
        {"name": "gather-long-i8", "kind": "gather", "batch": 1, "heads": 8, "d": 128, "page": 128,
         "format": "i8", "new": 65536, "ragged": False, "lo": 0, "hi": 0},
        # ragged spans of several sequences on the smallest pages
        {"name": "gather-spans", "kind": "gather", "batch": 16, "heads": 8, "d": 64, "page": 16,
         "format": "bf16", "new": 1001, "ragged": True, "lo": 3, "hi": 3001},
        # one token of the long text against its bf16 cache
        {"name": "attend-token-64k", "kind": "attend", "batch": 1, "heads": 8, "d": 128, "page": 64,
         "format": "bf16", "new": 1, "ragged": False, "lo": 65535, "hi": 65535},
        # 64 images in progress, each at its own pixel, over an 8-bit cache
        {"name": "attend-images-i8", "kind": "attend", "batch": 64, "heads": 8, "d": 64, "page": 64,
         "format": "i8", "new": 1, "ragged": False, "lo": 1, "hi": 12287},
        # five drafted tokens each of 16 sequences, a padded batch
        {"name": "attend-drafts", "kind": "attend", "batch": 16, "heads": 8, "d": 128, "page": 32,
         "format": "bf16", "new": 5, "ragged": True, "lo": 100, "hi": 8192},
        # the start of one sequence: latency
        {"name": "attend-start", "kind": "attend", "batch": 1, "heads": 8, "d": 64, "page": 16,
         "format": "i8", "new": 1, "ragged": False, "lo": 199, "hi": 199},
    ]


def draw(rng):
    def log(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    kind = rng.choice(["rope", "append", "gather", "attend", "attend"])
    d = rng.choice([64, 128])
    heads = rng.choice([1, 2, 4, 8, 12, 16])
    axes = rng.choice(["24,24,16", "64", "40", "32,32", "16,12,12,8"] if d == 64
                      else ["128", "64", "44,42,42", "64,32,32", "96"])
    adjacent = rng.choice([False, True])
    first = rng.choice([False, True])
    if kind == "rope":
        batch = log(1, 16)
        most = 50_000_000 // (batch * heads * d)
        n = log(1, min(131072, most))
        return {"kind": kind, "batch": batch, "heads": heads, "n": n, "d": d, "axes": axes,
                "adjacent": adjacent, "inverse": rng.choice([False, True]),
                "dtype": rng.choice(["bf16", "bf16", "f32"]) if n * batch * heads * d < 25_000_000
                else "bf16", "tokens_first": first, "offset": rng.choice([0, 0, 100003, 16777217])}
    page = rng.choice([16, 32, 64, 128])
    fmt = rng.choice(["bf16", "i8"])
    batch = log(1, 96)
    ragged = batch > 1 and rng.random() < 0.4
    if kind == "attend":
        new = rng.choice([1, 1, 1, 2, 3, 5, 8, 11, 16])
        hi = log(1, max(2, min(65536, 400_000_000 // (batch * heads * d * 2))))
        return {"kind": kind, "batch": batch, "heads": heads, "d": d, "page": page, "format": fmt,
                "new": new, "ragged": ragged and new > 1, "lo": rng.randint(0, hi), "hi": hi}
    most = 60_000_000 // (batch * heads * d)
    if kind == "append" and rng.random() < 0.5:
        new = rng.choice([1, 1, 2, 4, 7])
    else:
        new = log(1, max(2, min(65536, most // 2)))
    hi = log(1, max(2, min(65536, most // 2)))
    case = {"kind": kind, "batch": batch, "heads": heads, "d": d, "page": page, "format": fmt,
            "new": new, "ragged": ragged, "lo": rng.randint(0, hi), "hi": hi}
    if kind == "append":
        case.update(axes=axes, adjacent=adjacent, tokens_first=first)
    return case


def lengths(case):
    """Tokens each sequence holds before the call, lo to hi, and how many rows of `new` it has (in a
    padded batch down to none: a sequence that sits a step out)."""
    B, lo, hi, new = case["batch"], case["lo"], case["hi"], case["new"]
    at = [(7 * b + 3) % B if B % 7 else (5 * b + 3) % B if B % 5 else b for b in range(B)]
    before = [lo + (hi - lo) * a // max(1, B - 1) if B > 1 else hi for a in at]
    valid = [new - (new + 1) * a // B if case["ragged"] else new for a in at]
    return before, valid


def axes_of(case):
    return [int(a) for a in case["axes"].split(",")]


def work(case):
    B, H, d = case["batch"], case["heads"], case["d"]
    if case["kind"] == "rope":
        E = 4 if case["dtype"] == "f32" else 2
        n, A = case["n"], len(axes_of(case))
        x = B * H * n * d
        return {"bytes": 2 * x * E + 4 * A * B * n, "flops": 3 * x}
    before, valid = lengths(case)
    E = 1 if case["format"] == "i8" else 2
    P, T = case["page"], case["new"]
    rows = sum(valid) * H
    if case["kind"] == "append":
        # x, v in; rotated rows, cached rows and norms out; the positions and page numbers
        w = rows * d * (2 + 2 + 2 + 2 * E) + rows * 4
        w += len(axes_of(case)) * 4 * B * T + 4 * sum((v + P - 1) // P for v in valid)
        if E == 1:  # the rows of the pages that were written, read back as values
            back = H * sum(b % P + v for b, v in zip(before, valid))
            w += back * d * 2 * (1 + 2)
        return {"bytes": w, "flops": 3 * rows * d}
    if case["kind"] == "gather":
        # the cached rows in, all rows of the padded batch out
        return {"bytes": 2 * rows * d * E + 2 * B * H * T * d * 2, "flops": 0}
    seen = [b + v if v else 0 for b, v in zip(before, valid)]
    w = H * sum(seen) * (2 * d * E + 4) + 4 * sum((s + P - 1) // P for s in seen)
    w += rows * (2 * d) + B * H * T * (2 * d + 4)
    return {"bytes": w, "flops": 4 * d * H * sum(v * b + v * (v + 1) // 2
                                                 for b, v in zip(before, valid))}


# ------------------------------------------------------------------------------ inputs
def frequencies(axes, device):
    """The usual frequencies of every axis: 10000^(-2 i / dims)."""
    f = [10000.0 ** (-2.0 * i / a) for a in axes for i in range(a // 2)]
    return torch.tensor(f, dtype=torch.float64, device=device).float()


def image_positions(at, axes):
    """Positions of the tokens numbered `at`, one row for each axis: the channel, column and row of
    a raster of 64 columns and 3 channels (the last axes run fastest), or the number itself."""
    if axes == 1:
        return at[None]
    p, rows = at, []
    for size in (3, 64, 64)[:axes - 1]:
        rows.append(p % size)
        p = p // size
    return torch.stack([p] + rows[::-1])


def pairs(axes, adjacent, device):
    """Of every rotated pair: its two dimensions and its axis."""
    lo, hi, axis, at = [], [], [], 0
    for a, dims in enumerate(axes):
        i = torch.arange(dims // 2)
        lo.append(at + (2 * i if adjacent else i))
        hi.append(at + (2 * i + 1 if adjacent else i + dims // 2))
        axis.append(torch.full_like(i, a))
        at += dims
    return [torch.cat(t).to(device) for t in (lo, hi, axis)]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    B, H, d = case["batch"], case["heads"], case["d"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev)

    def heads_of(T, dtype):
        """Rows [B, H, T, d]; token-major in memory where the case says so, as projections are."""
        if case.get("tokens_first"):
            return normal(B, T, H, d).to(dtype).permute(0, 2, 1, 3)
        return normal(B, H, T, d).to(dtype)

    s = {"case": dict(case)}
    if "axes" in case:
        s["pairs"] = pairs(axes_of(case), case["adjacent"], dev)
    if case["kind"] == "rope":
        axes, n = axes_of(case), case["n"]
        dtype = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        # a gradient comes head by head from the attention, and its result may be asked for token-major
        s["x"] = normal(B, H, n, d).to(dtype) if case["inverse"] else heads_of(n, dtype)
        at = case["offset"] + torch.arange(n, device=dev) + 17 * torch.arange(B, device=dev)[:, None]
        s["positions"] = image_positions(at, len(axes)).to(torch.int32).contiguous()
        s["freqs"] = frequencies(axes, dev)
        return s
    P, T = case["page"], case["new"]
    before, valid = lengths(case)
    # every sequence has pages for all its rows and two more
    per_seq = max(before) // P + (T + P - 1) // P + 2
    pages = B * per_seq + 3
    order = torch.randperm(pages, generator=g, device=dev)
    s["table"] = order[:B * per_seq].view(B, per_seq).to(torch.int32).contiguous()
    s["before"] = torch.tensor(before, dtype=torch.int32, device=dev)
    s["valid"] = torch.tensor(valid, dtype=torch.int32, device=dev) if case["ragged"] else None
    if case["format"] == "i8":
        # rows of scale 2^-5: values of about 0.9 in steps of 1/32
        s["k"] = normal(pages, H, P, d).mul_(28).round_().clamp_(-127, 127).to(torch.int8)
        s["v"] = normal(pages, H, P // 16, d, 16).mul_(28).round_().clamp_(-127, 127).to(torch.int8)
        s["k_scale"] = torch.exp2(torch.randint(-6, -3, (pages, H), generator=g, device=dev).float())
        s["v_scale"] = torch.exp2(torch.randint(-6, -3, (pages, H), generator=g, device=dev).float())
        # summed head by head: the squares of a large cache need not be held at once
        sq = torch.stack([s["k"][:, h].float().square_().sum(-1) for h in range(H)], 1)
        norm = sq.sqrt_() * s["k_scale"][:, :, None]
    else:
        s["k"] = normal(pages, H, P, d).bfloat16()
        s["v"] = normal(pages, H, P // 16, d, 16).bfloat16()
        s["k_scale"] = s["v_scale"] = None
        sq = torch.stack([s["k"][:, h].float().square_().sum(-1) for h in range(H)], 1)
        norm = sq.sqrt_()
    s["kinv"] = 1.0 / norm.clamp_(min=1e-30)
    if case["kind"] == "gather":
        return s
    s["x"] = heads_of(T, torch.bfloat16)
    if case["kind"] == "attend":
        # as after the step's append: the new tokens' own rows are in the cache already
        return s
    s["v_new"] = heads_of(T, torch.bfloat16)
    axes = axes_of(case)
    at = s["before"][:, None].long() + torch.arange(T, device=dev)
    s["positions"] = image_positions(at, len(axes)).to(torch.int32).contiguous()
    s["freqs"] = frequencies(axes, dev)
    if case["format"] == "i8":
        # the rows read back: from the start of the first page written
        s["start"] = s["before"] // P * P
        s["span"] = T + P - 1
        s["back"] = s["before"] - s["start"] + (T if s["valid"] is None else s["valid"])
    return s


# ------------------------------------------------------------------------------ plain forms
def plain_rope(x, positions, freqs, dims, inverse):
    lo, hi, axis = dims
    angle = positions.double()[axis].permute(1, 2, 0) * freqs.double()  # [B, n, pairs]
    c, s = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if inverse:
        s = -s
    out = x.float()
    a, b = out[..., lo], out[..., hi]
    out = out.clone(memory_format=torch.contiguous_format)
    out[..., lo] = a * c - b * s
    out[..., hi] = a * s + b * c
    return out.to(x.dtype)


def rows_of_v(v):
    """[..., page_size / 16, d, 16] -> [..., page_size, d]"""
    return v.transpose(-1, -2).flatten(-3, -2)


def groups_of_v(v):
    """[..., page_size, d] -> [..., page_size / 16, d, 16]"""
    return v.unflatten(-2, (-1, 16)).transpose(-1, -2)


def plain_append(s):
    case = s["case"]
    P, T = case["page"], case["new"]
    x, v = s["x"], s["v_new"]
    xr = plain_rope(x, s["positions"], s["freqs"], s["pairs"], False)
    norm = x.float().square().sum(-1).sqrt()
    kinv = torch.where(norm < 2.0 ** -126, 0.0, 1.0 / norm)
    # the pages that the new rows touch, and which new row each of their slots takes
    B, H, d = case["batch"], case["heads"], case["d"]
    first = s["before"].long() // P
    window = (T + P - 2) // P + 1
    page = s["table"].long().gather(1, first[:, None] + torch.arange(window, device=x.device))
    pos = (first * P)[:, None] + torch.arange(window * P, device=x.device)
    t = pos - s["before"][:, None]
    count = s["valid"][:, None] if s["valid"] is not None else T
    fresh = (t >= 0) & (t < count)
    src = t.clamp(0, T - 1)[:, None, :, None].expand(B, H, -1, d)
    fresh_rows = fresh[:, None].expand(B, H, -1)

    def paged(rows):  # [B, H, window * P, ...] -> [B, window, H, P, ...]
        return rows.unflatten(2, (window, P)).transpose(1, 2)

    new = paged(fresh_rows)
    s["kinv"][page] = torch.where(new, paged(kinv.gather(2, src[..., 0])), s["kinv"][page])
    for rows, name, is_v in ((xr, "k", False), (v, "v", True)):
        store = s[name]
        r = paged(rows.gather(2, src)).float()
        old = store[page].float()
        old = rows_of_v(old) if is_v else old
        if case["format"] == "i8":
            scales = s[name + "_scale"]
            amax = torch.where(new[..., None], r.abs(), 0.0).amax((-1, -2))
            m, e = torch.frexp(amax)
            need = torch.ldexp(torch.ones_like(m), (e - 7 + (m > 127 / 128).int()).clamp(min=-126))
            # a page without earlier rows starts with the scale that its new rows need
            has_old = (first[:, None] + torch.arange(window, device=x.device)) * P < s["before"][:, None]
            was = torch.where(has_old[..., None], scales[page], 0.0)
            touched = new.any(-1)
            scale = torch.where(touched, torch.maximum(was, need), scales[page])
            kept = torch.round(old * (was / scale)[..., None, None])
            q = torch.round(r / scale[..., None, None]).clamp(-127, 127)
            earlier = paged((pos < s["before"][:, None])[:, None].expand(B, H, -1))
            kept = torch.where((earlier & touched[..., None])[..., None], kept, old)
            r, old = q, kept
            scales[page] = scale
        r = torch.where(new[..., None], r, old)
        store[page] = (groups_of_v(r) if is_v else r).to(store.dtype)
    if s["valid"] is not None:
        live = torch.arange(T, device=x.device) < s["valid"][:, None]
        xr = torch.where(live[:, None, :, None], xr, 0.0)
    return xr


def plain_gather(s, start, n, valid):
    P = s["case"]["page"]
    B = s["table"].shape[0]
    i = torch.arange(n, device=start.device)
    pos = start.long()[:, None] + i
    page = s["table"].long().gather(1, (pos // P).clamp(max=s["table"].shape[1] - 1))
    slot = pos % P
    k = s["k"][page, :, slot].float()  # [B, n, H, d]
    v = s["v"][page, :, slot // 16, :, slot % 16].float()
    if s["k_scale"] is not None:
        k = k * s["k_scale"][page][..., None]
        v = v * s["v_scale"][page][..., None]
    if valid is not None:
        live = (i < valid[:, None])[:, :, None, None]
        k, v = torch.where(live, k, 0.0), torch.where(live, v, 0.0)
    return k.transpose(1, 2).to(torch.bfloat16), v.transpose(1, 2).to(torch.bfloat16)


def plain_attend(s):
    x, P = s["x"], s["case"]["page"]
    B, H, T, d = x.shape
    page = s["table"].long()
    k = s["k"][page].float()  # [B, pages, H, P, d]
    v = rows_of_v(s["v"][page]).float()
    if s["k_scale"] is not None:
        k = k * s["k_scale"][page][..., None, None]
        v = v * s["v_scale"][page][..., None, None]
    k, v = k.transpose(1, 2).flatten(2, 3), v.transpose(1, 2).flatten(2, 3)
    kinv = s["kinv"][page].transpose(1, 2).flatten(2, 3)
    logit = x.float() @ k.transpose(-1, -2) * (kinv / math.sqrt(d))[:, :, None]
    at = s["before"].long()[:, None] + torch.arange(T, device=x.device)
    at = at[:, None, :, None]
    j = torch.arange(k.shape[2], device=x.device)
    logit = torch.where(j == at, SELF, torch.where(j < at, logit, -math.inf))
    top = logit.amax(-1, keepdim=True)
    p = (logit - top).exp()
    total = p.sum(-1, keepdim=True)
    out = (p @ v / total).to(x.dtype)
    lse = (top + total.log())[..., 0]
    if s["valid"] is not None:
        live = (torch.arange(T, device=x.device) < s["valid"][:, None])[:, None]
        out, lse = torch.where(live[..., None], out, 0.0), torch.where(live, lse, -math.inf)
    return out, lse


def cache_of(s):
    """The cache object that a program makes once and keeps."""
    from lsh_attention_b200 import binding as lb
    if "cache" not in s:
        s["cache"] = lb.LshCache(s["k"], s["v"], s["kinv"], s["k_scale"], s["v_scale"])
    return lb, s["cache"]


def run(s):
    case = s["case"]
    kind = case["kind"]
    if kind == "rope":
        if own:
            from lsh_attention_b200 import binding as lb
            out = None
            if case["inverse"] and case["tokens_first"]:
                B, H, n, d = s["x"].shape
                out = s["x"].new_empty(B, n, H, d).permute(0, 2, 1, 3)
            return lb.lsh_rope(s["x"], s["positions"], s["freqs"], axis_dims=axes_of(case),
                               adjacent=case["adjacent"], inverse=case["inverse"], out=out)
        return plain_rope(s["x"], s["positions"], s["freqs"], s["pairs"], case["inverse"])
    if kind == "append":
        if own:
            lb, cache = cache_of(s)
            xr = lb.lsh_cache_append(cache, s["x"], s["v_new"], s["table"], s["before"],
                                     n_valid=s["valid"], positions=s["positions"],
                                     freqs=s["freqs"], axis_dims=axes_of(case),
                                     adjacent=case["adjacent"])
        else:
            xr = plain_append(s)
        if case["format"] == "bf16":
            return {"xr": xr, "k": s["k"], "v": s["v"], "kinv": s["kinv"]}
        if own:
            k, v = lb.lsh_cache_gather(cache, s["table"], s["start"], s["span"], n_valid=s["back"])
        else:
            k, v = plain_gather(s, s["start"], s["span"], s["back"])
        return {"xr": xr, "k": k, "v": v, "kinv": s["kinv"]}
    if kind == "gather":
        if own:
            lb, cache = cache_of(s)
            return lb.lsh_cache_gather(cache, s["table"], s["before"], case["new"],
                                       n_valid=s["valid"])
        return plain_gather(s, s["before"], case["new"], s["valid"])
    if own:
        lb, cache = cache_of(s)
        return lb.lsh_cache_attend(cache, s["x"], s["table"], s["before"], n_valid=s["valid"])
    return plain_attend(s)


# ------------------------------------------------------------------------------ in 64 bits
def exact_rotation(x, positions, freqs, axes, adjacent, inverse):
    """Rows x [B, H, n, d] turned pair by pair, as complex numbers in 64 bits."""
    y = x.double()
    parts, at, f = [], 0, 0
    for a, dims in enumerate(axes):
        sec = y[..., at:at + dims]
        turn = positions[a].double()[:, None, :, None] * freqs[f:f + dims // 2].double()
        turn = torch.polar(torch.ones_like(turn), -turn if inverse else turn)
        if adjacent:
            z = torch.view_as_complex(sec.unflatten(-1, (-1, 2)).contiguous()) * turn
            sec = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(sec[..., :dims // 2], sec[..., dims // 2:]) * turn
            sec = torch.cat([z.real, z.imag], -1)
        parts.append(sec)
        at, f = at + dims, f + dims // 2
    parts.append(y[..., at:])
    return torch.cat(parts, -1)


def exact_page(s, h, ids):
    """Rows of x and v and the norms' reciprocals of head h on the pages `ids`, in 64 bits."""
    P, d = s["case"]["page"], s["case"]["d"]
    k = s["k"][ids, h].double()
    v = s["v"][ids, h].double().movedim(-1, -2).reshape(len(ids), P, d)
    if s["k_scale"] is not None:
        k = k * s["k_scale"][ids, h].double()[:, None, None]
        v = v * s["v_scale"][ids, h].double()[:, None, None]
    return k.reshape(-1, d), v.reshape(-1, d), s["kinv"][ids, h].double().reshape(-1)


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "rope":
        return exact_rotation(s["x"], s["positions"], s["freqs"], axes_of(case), case["adjacent"],
                              case["inverse"])
    B, H, d, T, P = case["batch"], case["heads"], case["d"], case["new"], case["page"]
    if B * H > 2000:
        return None
    before, valid = lengths(case)
    if kind == "attend":
        out = torch.zeros(B, H, T, d, dtype=torch.float64, device="cuda")
        lse = torch.full((B, H, T), -math.inf, dtype=torch.float64, device="cuda")
        for b in range(B):
            n = before[b] + valid[b]
            if not valid[b]:
                continue
            ids = s["table"][b, :(n + P - 1) // P].long()
            for h in range(H):
                k, v, kinv = exact_page(s, h, ids)
                k = k[:n] * kinv[:n, None]
                l = (s["x"][b, h, :valid[b]].double() @ k.T) / d ** 0.5
                at = torch.arange(before[b], n, device="cuda")
                l[torch.arange(valid[b], device="cuda"), at] = SELF
                l.masked_fill_(torch.arange(n, device="cuda") > at[:, None], -math.inf)
                lse[b, h, :valid[b]] = torch.logsumexp(l, -1)
                out[b, h, :valid[b]] = torch.softmax(l, -1) @ v[:n]
        return out, lse
    if kind == "gather":
        k_out = torch.zeros(B, H, T, d, dtype=torch.float64, device="cuda")
        v_out = torch.zeros_like(k_out)
        for b in range(B):
            first, last = before[b] // P, (before[b] + valid[b] + P - 1) // P
            ids = s["table"][b, first:last].long()
            for h in range(H):
                k, v, _ = exact_page(s, h, ids)
                at = before[b] - first * P
                k_out[b, h, :valid[b]] = k[at:at + valid[b]]
                v_out[b, h, :valid[b]] = v[at:at + valid[b]]
        return k_out, v_out
    xr = exact_rotation(s["x"], s["positions"], s["freqs"], axes_of(case), case["adjacent"], False)
    norm = torch.linalg.vector_norm(s["x"].double(), dim=-1)
    kinv = s["kinv"].double()
    k, v = (None, None) if case["format"] == "i8" else (s["k"].double(), s["v"].double())
    for b in range(B):
        xr[b, :, valid[b]:] = 0
        t = torch.arange(valid[b], device="cuda")
        page, slot = s["table"][b].long()[(before[b] + t) // P], (before[b] + t) % P
        kinv[page, :, slot] = 1.0 / norm[b, :, :valid[b]].T
        if k is not None:
            k[page, :, slot] = xr[b, :, :valid[b]].transpose(0, 1)
            v[page, :, slot // 16, :, slot % 16] = s["v_new"][b, :, :valid[b]].transpose(0, 1).double()
    # the rows of an 8-bit cache are what the rounding decides, not computed numbers
    return {"xr": xr, "k": k, "v": v, "kinv": kinv}
