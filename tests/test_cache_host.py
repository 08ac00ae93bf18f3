"""Host checks of the rotary and cache entry points: every refusal comes before anything is
launched or dereferenced. CPU only."""
import ctypes

import pytest
import torch

from lsh_attention_b200 import binding as lb
from lsh_attention_b200 import build as lbuild

from test_binding_host import FakeCudaTensor, FakeStream, device0  # noqa: F401

P = ctypes.c_void_p(4096)  # aligned, never dereferenced
ODD = ctypes.c_void_p(4096 + 8)
B, H, N, D = 2, 3, 5, 64
HEADS_FIRST = (H * N * D, N * D, D)
TOKENS_FIRST = (N * H * D, D, H * D)


@pytest.fixture(scope="module")
def lib():
    lbuild.build()
    return lb.load()


def three(s):
    return (ctypes.c_int64 * 3)(*s)


def axes(*dims, adjacent=0, count=None):
    return lb.LshRopeAxes(len(dims) if count is None else count, (ctypes.c_int32 * 4)(*dims), adjacent)


def rope(lib, x=P, pos=P, freqs=P, out=P, rot=None, xs=HEADS_FIRST, os_=HEADS_FIRST, **kw):
    f = dict(batch=B, heads=H, n=N, d=D, dtype=lb.LSH_BF16, inverse=0, pos_batched=1)
    f.update(kw)
    desc = lb.LshRopeDesc(*f.values(), rot or axes(32, 16), three(xs), three(os_))
    return lib.lsh_rope(ctypes.byref(desc), x, pos, freqs, out, None)


@pytest.mark.parametrize("kw,status", [
    ({"batch": 0}, 1), ({"heads": -1}, 1), ({"n": 0}, 1), ({"d": 0}, 1), ({"d": 96}, 2),
    ({"n": (1 << 24) + 1}, 2), ({"heads": 65536}, 2), ({"batch": (1 << 24) + 1}, 2),
    ({"inverse": 2}, 1), ({"pos_batched": 3}, 1), ({"dtype": 7}, 1),
    ({"x": None}, 1), ({"pos": None}, 1), ({"freqs": None}, 1), ({"out": None}, 1),
    ({"x": ODD}, 1), ({"out": ODD}, 1),
    ({"rot": axes(count=0)}, 1), ({"rot": axes(16, count=5)}, 1), ({"rot": axes(15)}, 1),
    ({"rot": axes(0)}, 1), ({"rot": axes(64, 2)}, 1), ({"rot": axes(32, -2)}, 1),
    ({"rot": axes(32, adjacent=2)}, 1),
    ({"xs": (H * N * D, N * D, -D)}, 1), ({"xs": (H * N * D, N * D, D + 4)}, 1),
    ({"os_": (H * N * D, 0, D)}, 1),                # heads written over one another
    ({"os_": (H * N * D, N * D, D - 8)}, 1),        # rows that overlap
    ({"os_": (N * D, N * D, D)}, 1),                # batches over heads
])
def test_rope_refusals(lib, kw, status):
    assert rope(lib, **kw) == status
    assert lib.lsh_rope(None, P, P, P, P, None) == 1


CACHE = dict(pages=4, heads=H, page_size=16, d=D, format=lb.LSH_CACHE_I8)
MEM = dict(k=4096, v=4096, key_inv_norm=4096, k_scale=4096, v_scale=4096, status=0)
ROWS = dict(batch=B, n=N, max_pages=3, pos_batched=1, x=TOKENS_FIRST, v=TOKENS_FIRST, out=HEADS_FIRST)


def parts(kw):
    pick = lambda base: {k: kw.get(k2, base[k]) for k, k2 in ((k, k) for k in base)}  # noqa: E731
    c, r = pick(CACHE), dict(ROWS)
    m = {k: kw.get("m_" + k, v) for k, v in MEM.items()}
    for k in ROWS:
        r[k] = kw.get("r_" + k, r[k])
    rows = lb.LshCacheRows(r["batch"], r["n"], r["max_pages"], r["pos_batched"], three(r["x"]),
                           three(r["v"]), three(r["out"]))
    return [ctypes.byref(lb.LshCacheDesc(*c.values())), ctypes.byref(lb.LshCacheMemory(*m.values())),
            ctypes.byref(rows)]


def append(lib, kw):
    a = lambda k, default=P: kw.get(k, default)  # noqa: E731
    rot = kw.get("rot", axes(32, 16))
    return lib.lsh_cache_append(*parts(kw), ctypes.byref(rot), a("x"), a("v"), a("pos"), a("freqs"),
                                a("table"), a("len"), None, a("xr"), None)


def gather(lib, kw):
    a = lambda k, default=P: kw.get(k, default)  # noqa: E731
    return lib.lsh_cache_gather(*parts(kw), a("table"), a("len"), None, a("x"), a("v"), None)


def attend(lib, kw):
    a = lambda k, default=P: kw.get(k, default)  # noqa: E731
    return lib.lsh_cache_attend(*parts(kw), a("x"), a("table"), a("len"), None, a("xr"), a("lse"),
                                a("ws"), kw.get("bytes", 1 << 40), None)


@pytest.mark.parametrize("call", [append, gather, attend])
@pytest.mark.parametrize("kw,status", [
    ({"pages": 0}, 1), ({"heads": 0}, 1), ({"page_size": 0}, 1), ({"format": 2}, 1),
    ({"page_size": 48}, 2), ({"page_size": 256}, 2), ({"d": 32}, 2), ({"heads": 70000}, 2),
    ({"m_k": 0}, 1), ({"m_v": 0}, 1), ({"m_key_inv_norm": 0}, 1), ({"m_k_scale": 0}, 1),
    ({"m_v_scale": 0}, 1), ({"m_k": 4100}, 1), ({"m_status": 4}, 1),
    ({"r_batch": 0}, 1), ({"r_n": 0}, 1), ({"r_max_pages": 0}, 1), ({"r_batch": 65536}, 2),
    ({"r_n": (1 << 24) + 1}, 2), ({"r_max_pages": (1 << 27) - (1 << 20)}, 2), ({"r_x": (0, 0, 12)}, 1), ({"r_x": (0, -8, 8)}, 1),
    ({"x": None}, 1), ({"x": ODD}, 1), ({"table": None}, 1), ({"len": None}, 1),
])
def test_cache_refusals(lib, call, kw, status):
    assert call(lib, kw) == status


@pytest.mark.parametrize("call,kw,status", [
    (append, {"v": None}, 1), (append, {"v": ODD}, 1), (append, {"xr": ODD}, 1),
    (append, {"pos": None}, 1), (append, {"freqs": None}, 1), (append, {"rot": axes(64, 64)}, 1),
    (append, {"rot": axes(count=-1)}, 1), (append, {"r_pos_batched": 2}, 1),
    (append, {"r_v": (8, 8, 4)}, 1), (append, {"r_out": (0, N * D, D)}, 1),
    (gather, {"v": None}, 1), (gather, {"r_x": (0, N * D, D)}, 1), (gather, {"r_v": (0, 0, D)}, 1),
    (attend, {"xr": None}, 1), (attend, {"lse": None}, 1), (attend, {"r_out": (0, 0, D)}, 1),
    (attend, {"ws": None}, 3), (attend, {"ws": ctypes.c_void_p(4096 + 64)}, 3),
    (attend, {"bytes": 16}, 3),
])
def test_cache_refusals_of_one_call(lib, call, kw, status):
    assert call(lib, kw) == status


def test_attend_workspace_size(lib):
    size = ctypes.c_size_t(0)
    c, _, r = parts({})
    assert lib.lsh_cache_attend_workspace_size(c, r, ctypes.byref(size)) == 0
    assert size.value > 0 and size.value % 256 == 0
    assert lib.lsh_cache_attend_workspace_size(c, r, None) == 1
    assert lib.lsh_cache_attend_workspace_size(None, r, ctypes.byref(size)) == 1
    c, _, r = parts({"d": 96})
    assert lib.lsh_cache_attend_workspace_size(c, r, ctypes.byref(size)) == 2


# ------------------------------------------------------------------------------ the binding
class Tensor(FakeCudaTensor):
    def __init__(self, shape, dtype=torch.bfloat16, index=0, strides=None):
        super().__init__(shape, dtype, index)
        self._t = torch.empty(self.shape, dtype=dtype, device="meta") if strides is None else \
            torch.empty_strided(self.shape, strides, dtype=dtype, device="meta")

    def stride(self):
        return self._t.stride()

    def is_contiguous(self):
        return self._t.is_contiguous()

    def dim(self):
        return len(self.shape)


class Cache:
    heads, d, page_size, int8 = H, D, 16, False

    def __init__(self, index=0):
        self.k = Tensor((4, H, 16, D), index=index)
        self.kind = index


def ints(*shape, index=0):
    return Tensor(shape, torch.int32, index)


def test_binding_rejects_other_devices(device0):  # noqa: F811
    x, v, tab, ln = Tensor((B, H, N, D)), Tensor((B, H, N, D)), ints(B, 3), ints(B)
    f = Tensor((24,), torch.float32)
    with pytest.raises(ValueError, match="positions is on cuda:1"):
        lb.lsh_rope(x, ints(2, N, index=1), f, axis_dims=(32, 16))
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        lb.lsh_rope(x, ints(2, N), f, axis_dims=(32, 16), stream=FakeStream(1))
    with pytest.raises(ValueError, match="cache is on cuda:1"):
        lb.lsh_cache_append(Cache(1), x, v, tab, ln)
    with pytest.raises(ValueError, match="seq_len is on cuda:1"):
        lb.lsh_cache_attend(Cache(), x, tab, ints(B, index=1))
    with pytest.raises(ValueError, match="start is on cuda:1"):
        lb.lsh_cache_gather(Cache(), tab, ints(B, index=1), N)
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        lb.lsh_rope(torch.zeros(B, H, N, D), ints(2, N), f, axis_dims=(32, 16))


def test_binding_rejects_shapes_and_types(device0):  # noqa: F811
    x, v, tab, ln = Tensor((B, H, N, D)), Tensor((B, H, N, D)), ints(B, 3), ints(B)
    f = Tensor((24,), torch.float32)
    with pytest.raises(ValueError, match="positions must have shape"):
        lb.lsh_rope(x, ints(1, N), f, axis_dims=(32, 16))
    with pytest.raises(ValueError, match="freqs must have shape"):
        lb.lsh_rope(x, ints(2, N), Tensor((23,), torch.float32), axis_dims=(32, 16))
    with pytest.raises(TypeError, match="positions must be torch.int32"):
        lb.lsh_rope(x, Tensor((2, N), torch.int64), f, axis_dims=(32, 16))
    with pytest.raises(ValueError, match="last dimension must be contiguous"):
        lb.lsh_rope(Tensor((B, H, N, D), strides=(H * N * D, N * D, 1, N)), ints(2, N), f,
                    axis_dims=(32, 16))
    with pytest.raises(TypeError, match="unsupported dtype"):
        lb.lsh_rope(Tensor((B, H, N, D), torch.float16), ints(2, N), f, axis_dims=(32, 16))
    with pytest.raises(ValueError, match="at most 4 axes"):
        lb.lsh_rope(x, ints(5, N), Tensor((5,), torch.float32), axis_dims=(2,) * 5)
    with pytest.raises(ValueError, match="needs positions and freqs"):
        lb.lsh_cache_append(Cache(), x, v, tab, ln, axis_dims=(64,))
    with pytest.raises(ValueError, match="the cache 3 of 64"):
        lb.lsh_cache_append(Cache(), Tensor((B, H + 1, N, D)), v, tab, ln)
    with pytest.raises(ValueError, match="the cache 3 of 64"):
        lb.lsh_cache_attend(Cache(), Tensor((B, H, N, 128)), tab, ln)
    with pytest.raises(TypeError, match="v must be torch.bfloat16"):
        lb.lsh_cache_append(Cache(), x, Tensor((B, H, N, D), torch.float32), tab, ln)
    with pytest.raises(ValueError, match="page_table must have shape"):
        lb.lsh_cache_append(Cache(), x, v, ints(B + 1, 3), ln)
    with pytest.raises(ValueError, match="n_valid must have shape"):
        lb.lsh_cache_attend(Cache(), x, tab, ln, n_valid=ints(B + 1))


def test_cache_object_checks_its_arrays():
    mk = lambda shape, dt=torch.bfloat16: Tensor(shape, dt)  # noqa: E731
    good = [mk((4, H, 16, D)), mk((4, H, 1, D, 16)), mk((4, H, 16), torch.float32)]
    status = ints(64)
    for i, bad in ((0, mk((4, H, 16, D), torch.float16)), (1, mk((4, H, 16, D))),
                   (2, mk((4, H, 16))), (1, mk((4, H, 1, D, 16), torch.int8))):
        args = list(good)
        args[i] = bad
        with pytest.raises((TypeError, ValueError)):
            lb.LshCache(*args, status=status)
    with pytest.raises(ValueError, match="k_scale belongs to an int8 cache"):
        lb.LshCache(*good, k_scale=mk((4, H), torch.float32), v_scale=mk((4, H), torch.float32),
                    status=status)
    with pytest.raises(ValueError, match="k_scale belongs to an int8 cache"):
        lb.LshCache(mk((4, H, 16, D), torch.int8), mk((4, H, 1, D, 16), torch.int8), good[2],
                    status=status)
    with pytest.raises(ValueError, match="status must have shape"):
        lb.LshCache(*good, status=ints(63))
