"""What the paged-cache and mixture-of-experts entry points refuse, before anything
reaches a GPU: the C functions by status, the binding by exception."""
import ctypes as C

import pytest
import torch

from int4_weight_kv_w4a16_gb300 import build, futr
from int4_weight_kv_w4a16_gb300.inputs import LLAMA8B, TOY

PAGED_MAGIC, PAGED_WS_MAGIC = 0x3850564B52545546, 0x3857534B52545546
MOE_WS_MAGIC = 0x5745304D52545546
ARG, UNSUPPORTED = futr.FUTR_ERR_INVALID_ARG, futr.FUTR_ERR_UNSUPPORTED
MEM = 1 << 20   # an address that is passed on and never read


@pytest.fixture(scope="module")
def L():
    build.build()
    return futr.lib()


# ------------------------------------------------------------------- sizes --

@pytest.mark.parametrize("layers,pages,page,max_pos,want", [
    (0, 8, 16, 64, ARG), (-1, 8, 16, 64, ARG), (1, 0, 16, 64, ARG), (1, 8, 16, 0, ARG),
    (1, 8, 0, 64, UNSUPPORTED), (1, 8, 8, 64, UNSUPPORTED), (1, 8, 48, 64, UNSUPPORTED),
    (1, 8, 256, 64, UNSUPPORTED), (1, 8, -16, 64, UNSUPPORTED),
    (1, 8, 16, (1 << 20) + 1, UNSUPPORTED),
    (1 << 15, 1 << 15, 16, 64, UNSUPPORTED), (2 ** 31 - 1, 2 ** 31 - 1, 16, 64, UNSUPPORTED),
])
def test_paged_size_refuses(L, layers, pages, page, max_pos, want):
    n = C.c_size_t(7)
    s = futr.make_shape(TOY)
    assert L.futr_paged_size(C.byref(s), layers, pages, page, max_pos, C.byref(n)) == want
    assert n.value == 7
    with pytest.raises(futr.FutrError):
        futr.futr_paged_size(s, layers, pages, page, max_pos)


@pytest.mark.parametrize("block,layers,pages,page", [(TOY, 1, 1, 16), (TOY, 2, 5, 32), (LLAMA8B, 3, 70, 128),
                                                     (LLAMA8B, 80, 10000, 64)])
def test_paged_size_holds_codes_scales_and_table(L, block, layers, pages, page):
    got = futr.futr_paged_size(futr.make_shape(block), layers, pages, page, 4096)
    blocks = layers * pages * block.n_kv_heads * 2
    need = blocks * page * block.head_dim + blocks * 4 + 4096 * block.head_dim // 2 * 8
    assert need <= got <= need + 8192


def test_paged_size_null_and_bad_shape(L):
    n = C.c_size_t()
    s = futr.make_shape(TOY)
    assert L.futr_paged_size(C.byref(s), 1, 8, 16, 64, None) == ARG
    assert L.futr_paged_size(None, 1, 8, 16, 64, C.byref(n)) == UNSUPPORTED
    s.head_dim = 96
    assert L.futr_paged_size(C.byref(s), 1, 8, 16, 64, C.byref(n)) == UNSUPPORTED
    assert L.futr_paged_workspace_size(C.byref(s), C.byref(n)) == UNSUPPORTED
    assert L.futr_paged_workspace_size(None, C.byref(n)) == UNSUPPORTED
    assert L.futr_paged_workspace_size(C.byref(s), None) == ARG


def test_paged_init_refuses_memory(L):
    s, cache = futr.make_shape(TOY), futr.futr_paged()
    need = futr.futr_paged_size(s, 1, 8, 16, 64)
    for mem, n, desc in ((None, need, cache), (MEM, need - 1, cache), (MEM + 16, need, cache), (MEM, 0, cache),
                         (MEM, need, None)):
        d = None if desc is None else C.byref(desc)
        assert L.futr_paged_init(C.byref(s), 1, 8, 16, 64, 1, mem, n, d, None) == ARG
    assert cache.magic == 0
    assert L.futr_paged_init(C.byref(s), 1, 8, 24, 64, 1, MEM, need, C.byref(cache), None) == UNSUPPORTED
    assert L.futr_paged_workspace_init(C.byref(s), None, 1 << 30, C.byref(futr.futr_paged_ws()), None) == ARG
    assert L.futr_paged_workspace_init(C.byref(s), MEM, 1 << 30, None, None) == ARG


# ------------------------------------------------------------------- calls --

def a_cache(block=TOY, layers=2):
    c = futr.futr_paged()
    c.shape = futr.make_shape(block)
    c.n_layers, c.n_pages, c.page, c.max_pos, c.rope = layers, 8, 16, 64, 1
    c.base, c.magic = MEM, PAGED_MAGIC
    return c


def a_paged_ws(block=TOY):
    w = futr.futr_paged_ws()
    w.head_dim, w.ctas, w.base, w.magic = block.head_dim, 1 << 20, MEM, PAGED_WS_MAGIC
    return w


ROWS = dict(layer=0, batch=2, pos=MEM, start=MEM, n_rows=3, table=MEM, table_ld=4, dtype=0)
BAD_ROWS = [("layer", -1, ARG), ("layer", 2, ARG), ("batch", 0, ARG), ("batch", -1, ARG), ("pos", None, ARG),
            ("start", None, ARG), ("n_rows", -1, ARG), ("table", None, ARG), ("table_ld", 0, ARG),
            ("dtype", 2, UNSUPPORTED), ("dtype", -1, UNSUPPORTED)]


def call_append(L, cache, k=MEM, ld_k=256, v=MEM, ld_v=256, **kw):
    a = dict(ROWS, **kw)
    return L.futr_paged_append(C.addressof(cache) if cache else None, a["layer"], a["batch"], a["pos"], a["start"],
                               a["n_rows"], a["table"], a["table_ld"], k, ld_k, v, ld_v, a["dtype"], None)


def call_attention(L, cache, ws, q=MEM, ld_q=256, out=MEM + 4096, ld_out=256, scale=0.0, window=0, **kw):
    a = dict(ROWS, **kw)
    return L.futr_paged_attention(C.addressof(cache) if cache else None, a["layer"], a["batch"], a["pos"], a["start"],
                                  a["n_rows"], a["table"], a["table_ld"], q, ld_q, out, ld_out, a["dtype"], scale,
                                  window, C.addressof(ws) if ws else None, None)


@pytest.mark.parametrize("name,value,want", BAD_ROWS)
def test_paged_calls_refuse_rows(L, name, value, want):
    c, w = a_cache(), a_paged_ws()
    assert call_append(L, c, **{name: value}) == want
    assert call_attention(L, c, w, **{name: value}) == want


def test_paged_calls_refuse_descriptors(L):
    c, w = a_cache(), a_paged_ws()
    fresh = futr.futr_paged()
    assert call_append(L, None) == ARG and call_append(L, fresh) == ARG
    assert call_attention(L, None, w) == ARG and call_attention(L, fresh, w) == ARG
    assert call_attention(L, c, None) == ARG and call_attention(L, c, futr.futr_paged_ws()) == ARG
    assert call_attention(L, c, a_paged_ws(LLAMA8B)) == ARG   # a workspace of another head size
    assert L.futr_paged_check(None, None, None) == ARG
    assert L.futr_paged_check(C.byref(fresh), None, None) == ARG
    assert L.futr_paged_check(C.byref(c), C.byref(futr.futr_paged_ws()), None) == ARG


@pytest.mark.parametrize("kw", [{"k": None}, {"v": None}, {"k": MEM + 2}, {"v": MEM + 8}, {"ld_k": 120}, {"ld_v": 124},
                                {"ld_k": 132}, {"ld_k": -128}, {"ld_v": 0}])
def test_append_refuses_row_tensors(L, kw):
    assert call_append(L, a_cache(), **kw) == ARG


@pytest.mark.parametrize("kw", [{"q": None}, {"out": None}, {"q": MEM + 2}, {"out": MEM + 8}, {"ld_q": 248},
                                {"ld_out": 260}, {"ld_q": -256}, {"out": MEM}, {"window": -1}, {"scale": -1.0},
                                {"scale": float("nan")}, {"scale": float("inf")}, {"scale": 3e38}])
def test_attention_refuses_row_tensors_and_scalars(L, kw):
    assert call_attention(L, a_cache(), a_paged_ws(), **kw) == ARG


def test_no_rows_is_no_work(L):
    c, w = a_cache(), a_paged_ws()
    assert call_append(L, c, n_rows=0, k=None, v=None) == futr.FUTR_OK
    assert call_attention(L, c, w, n_rows=0, q=None, out=None) == futr.FUTR_OK


# --------------------------------------------------------- mixture of experts --

@pytest.mark.parametrize("kw", [
    {"hidden": 0}, {"hidden": 192}, {"hidden": -128}, {"hidden": 1 << 21}, {"inter": 0}, {"inter": 200},
    {"n_experts": 0}, {"n_experts": 257}, {"top_k": 0}, {"top_k": 9}, {"top_k": 17, "n_experts": 64}, {"group": 64},
    {"rms_eps": -1e-5}, {"rms_eps": float("nan")}, {"rms_eps": float("inf")},
])
def test_moe_shape_refuses(L, kw):
    a = dict(hidden=256, inter=128, n_experts=8, top_k=2)
    a.update(kw)
    ms, n = futr.make_moe_shape(**a), C.c_size_t(7)
    assert L.futr_moe_weights_size(C.byref(ms), C.byref(n)) == UNSUPPORTED
    assert L.futr_moe_workspace_size(C.byref(ms), 4, C.byref(n)) == UNSUPPORTED
    assert L.futr_moe_pack(C.byref(ms), 0, MEM, MEM, MEM, None, MEM, 1 << 40, None) == UNSUPPORTED
    assert L.futr_moe_unpack(C.byref(ms), MEM, 0, futr.FUTR_PROJ_GATE, MEM, MEM, None) == UNSUPPORTED
    assert n.value == 7


def test_moe_sizes(L):
    ms = futr.make_moe_shape(256, 384, 8, 2)
    got = futr.futr_moe_weights_size(ms)
    need = 8 * 3 * 256 * 384 // 128 * (64 + 2)      # 4-bit codes and one fp16 scale of each 128
    assert need <= got <= need + 8192
    n = C.c_size_t()
    assert L.futr_moe_weights_size(C.byref(ms), None) == ARG
    assert L.futr_moe_weights_size(None, C.byref(n)) == UNSUPPORTED
    for b in (0, -1, 33):
        assert L.futr_moe_workspace_size(C.byref(ms), b, C.byref(n)) == ARG
    assert L.futr_moe_workspace_size(C.byref(ms), 4, None) == ARG
    assert L.futr_moe_workspace_init(C.byref(ms), 4, None, 1 << 30, C.byref(futr.futr_moe_ws()), None) == ARG
    assert L.futr_moe_workspace_init(C.byref(ms), 4, MEM, 1 << 30, None, None) == ARG


def test_moe_pack_and_unpack_refuse(L):
    ms = futr.make_moe_shape(256, 384, 8, 2)
    need = futr.futr_moe_weights_size(ms)
    ok = dict(expert=0, g=MEM, u=MEM, d=MEM, blob=MEM, n=need)
    for kw in ({"expert": -1}, {"expert": 8}, {"g": None}, {"u": None}, {"d": None}, {"blob": None}, {"n": need - 1},
               {"blob": MEM + 128}):
        a = dict(ok, **kw)
        assert L.futr_moe_pack(C.byref(ms), a["expert"], a["g"], a["u"], a["d"], None, a["blob"], a["n"], None) == ARG
    for blob, e, which, codes, scales in ((None, 0, 1, MEM, MEM), (MEM, 8, 1, MEM, MEM), (MEM, -1, 1, MEM, MEM),
                                          (MEM, 0, 99, MEM, MEM), (MEM, 0, 1, None, MEM), (MEM, 0, 1, MEM, None)):
        which = futr.FUTR_PROJ_GATE if which == 1 else which
        assert L.futr_moe_unpack(C.byref(ms), blob, e, which, codes, scales, None) == ARG


def a_moe_ws(max_batch=8):
    w = futr.futr_moe_ws()
    w.shape = futr.make_moe_shape(256, 384, 8, 2)
    w.max_batch, w.ctas, w.base, w.magic = max_batch, 1 << 20, MEM, MOE_WS_MAGIC
    return w


@pytest.mark.parametrize("kw,want", [
    ({"batch": 0}, UNSUPPORTED), ({"batch": 33}, UNSUPPORTED), ({"batch": 9}, ARG), ({"x": None}, ARG),
    ({"router": None}, ARG), ({"blob": None}, ARG), ({"y": None}, ARG), ({"x": MEM + 2}, ARG), ({"y": MEM + 8}, ARG),
    ({"resid": MEM + 4}, ARG), ({"router": MEM + 2}, ARG), ({"gain": MEM + 4}, ARG), ({"ids": MEM + 2}, ARG),
    ({"weights": MEM + 1}, ARG), ({"blob": MEM + 8}, ARG),
])
def test_moe_layer_refuses(L, kw, want):
    a = dict(x=MEM, gain=None, router=MEM, blob=MEM, batch=4, resid=None, y=MEM, ids=None, weights=None)
    a.update(kw)
    w = a_moe_ws()
    assert L.futr_moe_layer(*a.values(), C.addressof(w), None) == want


def test_moe_layer_refuses_descriptors(L):
    fresh = futr.futr_moe_ws()
    assert L.futr_moe_layer(MEM, None, MEM, MEM, 4, None, MEM, None, None, C.addressof(fresh), None) == ARG
    assert L.futr_moe_layer(MEM, None, MEM, MEM, 4, None, MEM, None, None, None, None) == ARG
    assert L.futr_moe_check(C.byref(fresh), None) == ARG and L.futr_moe_check(None, None) == ARG


# ------------------------------------------------------------------- binding --
# The tensor checks, on CPU tensors: the binding is told that the current device is
# theirs, and the library that every call is a failure of the test.

class _Never:
    def __getattr__(self, name):
        def called(*_):
            raise AssertionError(f"{name} was called")
        return called


class _Elsewhere:
    """A tensor, but on another device."""

    def __init__(self, t):
        self._t = t

    def __getattr__(self, name):
        return getattr(self._t, name)

    def get_device(self):
        return 1


@pytest.fixture
def binding(L, monkeypatch):
    t = futr._Torch()
    t.device, t.stream = (lambda: -1), (lambda device: 0)
    monkeypatch.setattr(futr, "_T", t)
    sizes = {"futr_moe_weights_size": futr.lib().futr_moe_weights_size}

    class Only(_Never):
        futr_moe_weights_size = staticmethod(sizes["futr_moe_weights_size"])

    monkeypatch.setattr(futr, "lib", lambda: Only())
    return t


BF, F16, F32, I32 = torch.bfloat16, torch.float16, torch.float32, torch.int32


def paged_tensors(**kw):
    t = dict(pos=torch.zeros(2, dtype=I32), start=torch.zeros(3, dtype=I32), table=torch.zeros((2, 4), dtype=I32),
             k=torch.zeros((3, 2, 64), dtype=BF), v=torch.zeros((3, 2, 64), dtype=BF),
             q=torch.zeros((3, 4, 64), dtype=BF), out=torch.zeros((3, 4, 64), dtype=BF))
    t.update(kw)
    return t


def append(t, cache=None):
    c = cache or a_cache()
    c._mem = getattr(c, "_mem", torch.zeros(1))
    futr.futr_paged_append(c, 0, 2, t["pos"], t["start"], t["table"], t["k"], t["v"])


def attention(t, ws=None):
    c, w = a_cache(), a_paged_ws()
    c._mem = w._mem = torch.zeros(1)
    futr.futr_paged_attention(c, 0, 2, t["pos"], t["start"], t["table"], t["q"], t["out"], w)


@pytest.mark.parametrize("kw,error", [
    ({"pos": torch.zeros(2, dtype=torch.int64)}, ValueError), ({"pos": torch.zeros(3, dtype=I32)}, ValueError),
    ({"pos": torch.zeros(4, dtype=I32)[::2]}, ValueError), ({"start": torch.zeros(2, dtype=I32)}, ValueError),
    ({"start": torch.zeros(3)}, ValueError), ({"table": torch.zeros(2, dtype=I32)}, ValueError),
    ({"table": torch.zeros((3, 4), dtype=I32)}, ValueError), ({"table": torch.zeros((2, 8), dtype=I32)[:, ::2]}, ValueError),
    ({"table": torch.zeros((2, 4), dtype=torch.int64)}, ValueError), ({"pos": _Elsewhere(torch.zeros(2, dtype=I32))}, ValueError),
])
def test_binding_refuses_rows(binding, kw, error):
    for call in (append, attention):
        with pytest.raises(error):
            call(paged_tensors(**kw))


@pytest.mark.parametrize("kw,error", [
    ({"k": torch.zeros((3, 2, 64), dtype=F16)}, TypeError), ({"k": torch.zeros((3, 2, 64)), "v": torch.zeros((3, 2, 64))}, TypeError),
    ({"v": torch.zeros((4, 2, 64), dtype=BF)}, ValueError), ({"v": torch.zeros((3, 4, 64), dtype=BF)}, ValueError),
    ({"k": torch.zeros((3, 64, 2), dtype=BF).transpose(1, 2)}, ValueError),
    ({"k": torch.zeros((3, 4, 64), dtype=BF)[:, ::2]}, ValueError),
    ({"k": torch.zeros((3, 2, 128), dtype=BF)[..., :64]}, ValueError),
    ({"k": _Elsewhere(torch.zeros((3, 2, 64), dtype=BF))}, ValueError),
])
def test_binding_refuses_keys_and_values(binding, kw, error):
    with pytest.raises(error):
        append(paged_tensors(**kw))


@pytest.mark.parametrize("kw,error", [
    ({"out": torch.zeros((3, 4, 64), dtype=F16)}, TypeError), ({"out": torch.zeros((3, 2, 64), dtype=BF)}, ValueError),
    ({"q": torch.zeros((3, 4, 32), dtype=BF)}, ValueError), ({"q": torch.zeros((3, 8, 64), dtype=BF)[:, ::2]}, ValueError),
])
def test_binding_refuses_queries_and_output(binding, kw, error):
    with pytest.raises(error):
        attention(paged_tensors(**kw))


def test_binding_refuses_a_cache_of_another_device(binding):
    c = a_cache()
    c._mem = _Elsewhere(torch.zeros(1))
    with pytest.raises(ValueError, match="the cache"):
        append(paged_tensors(), c)


def moe_layer(**kw):
    w = a_moe_ws()
    w._mem, w.blob_bytes = torch.zeros(1), 4096
    a = dict(x=torch.zeros((4, 256), dtype=BF), gain=None, router=torch.zeros((8, 256), dtype=BF),
             blob=torch.zeros(4096, dtype=torch.uint8), resid=None, y=torch.zeros((4, 256), dtype=BF), ids=None,
             weights=None)
    a.update(kw)
    futr.futr_moe_layer(a["x"], a["gain"], a["router"], a["blob"], a["resid"], a["y"], w, ids=a["ids"],
                        weights=a["weights"])


@pytest.mark.parametrize("kw", [
    {"x": torch.zeros((4, 128), dtype=BF)}, {"x": torch.zeros((4, 256), dtype=F16)},
    {"x": torch.zeros((4, 512), dtype=BF)[:, ::2]}, {"y": torch.zeros((3, 256), dtype=BF)},
    {"resid": torch.zeros((5, 256), dtype=BF)}, {"resid": torch.zeros((4, 256))},
    {"router": torch.zeros((7, 256), dtype=BF)}, {"router": torch.zeros((8, 256))},
    {"gain": torch.zeros(256, dtype=BF)}, {"gain": torch.zeros(128)}, {"blob": torch.zeros(4095, dtype=torch.uint8)},
    {"blob": torch.zeros(8192, dtype=torch.uint8)[::2]}, {"ids": torch.zeros((4, 2), dtype=torch.int64)},
    {"ids": torch.zeros((4, 3), dtype=I32)}, {"weights": torch.zeros((4, 2), dtype=BF)},
    {"weights": torch.zeros((3, 2))},
])
def test_binding_refuses_moe_layer(binding, kw):
    with pytest.raises(ValueError):
        moe_layer(**kw)


def test_binding_refuses_moe_weights(binding):
    ms = futr.make_moe_shape(256, 384, 8, 2)
    blob = torch.zeros(8 * 3 * 256 * 384, dtype=torch.uint8)
    w = [torch.zeros((384, 256)), torch.zeros((384, 256)), torch.zeros((256, 384))]
    codes, scales = torch.zeros((384, 256), dtype=torch.int8), torch.zeros((384, 2), dtype=F16)
    for i, bad in ((0, torch.zeros((256, 384))), (1, torch.zeros((384, 256), dtype=BF)), (2, torch.zeros((384, 256)))):
        with pytest.raises(ValueError):
            futr.futr_moe_pack(ms, 0, *[bad if j == i else w[j] for j in range(3)], None, blob)
    with pytest.raises(ValueError):
        futr.futr_moe_pack(ms, 0, *w, torch.zeros(384), blob)
    with pytest.raises(ValueError):
        futr.futr_moe_pack(ms, 0, *w, None, blob[:1000])
    for c, s in ((codes[:128], scales), (codes, scales.float()), (codes.to(torch.uint8), scales)):
        with pytest.raises(ValueError):
            futr.futr_moe_unpack(ms, blob, 0, futr.FUTR_PROJ_GATE, c, s)
    with pytest.raises(ValueError):
        futr.futr_moe_unpack(ms, blob, 0, futr.FUTR_PROJ_DOWN, codes, scales)
