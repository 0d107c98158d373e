"""What the calls for beams, cache slots, pages and sinks refuse, before anything reaches a GPU: the C functions by
status, the binding by exception; and the restatement of the page calls against cases worked by hand."""
import ctypes as C

import pytest
import torch

from int4_weight_kv_w4a16_gb300 import build, futr
from int4_weight_kv_w4a16_gb300.inputs import TOY
from tests._gen_ref import Pool, beam_best, beam_values

PAGED_MAGIC, PAGED_WS_MAGIC, KV_MAGIC = 0x3850564B52545546, 0x3857534B52545546, 0x31564B3452545546
BEAM_MAGIC, PAGES_MAGIC = 0x3142575452545546, 0x3147504752545546
ARG, UNSUPPORTED = futr.FUTR_ERR_INVALID_ARG, futr.FUTR_ERR_UNSUPPORTED
MEM = 1 << 20   # an address that is passed on and never read
F32, I32 = torch.float32, torch.int32


@pytest.fixture(scope="module")
def L():
    build.build()
    return futr.lib()


def a_cache(n_pages=8):
    c = futr.futr_paged()
    c.shape = futr.make_shape(TOY)
    c.n_layers, c.n_pages, c.page, c.max_pos, c.rope = 2, n_pages, 16, 64, 1
    c.base, c.magic, c._mem = MEM, PAGED_MAGIC, torch.zeros(1)
    return c


def a_paged_ws():
    w = futr.futr_paged_ws()
    w.head_dim, w.ctas, w.base, w.magic, w._mem = TOY.head_dim, 1 << 20, MEM, PAGED_WS_MAGIC, torch.zeros(1)
    return w


def a_pool(n_pages=8, max_seqs=4):
    p = futr.futr_pages()
    p.n_pages, p.max_seqs, p.base, p.magic, p._mem = n_pages, max_seqs, MEM, PAGES_MAGIC, torch.zeros(1)
    return p


def a_beam_ws(rows=8, keep=8):
    w = futr.futr_beam_ws()
    w.rows, w.keep, w.ctas, w.base, w.magic, w._mem = rows, keep, 1 << 20, MEM, BEAM_MAGIC, torch.zeros(1)
    return w


def a_kv(max_batch=40):
    k = futr.futr_kv()
    k.shape = futr.make_shape(TOY)
    k.n_layers, k.max_batch, k.capacity, k.base, k.magic, k._mem = 1, max_batch, 64, MEM, KV_MAGIC, torch.zeros(1)
    return k


def ref(d):
    return C.addressof(d) if d is not None else None


def test_status_strings(L):
    assert "free pages" in futr.futr_status_string(futr.FUTR_ERR_NO_PAGES)
    assert "free" in futr.futr_status_string(futr.FUTR_ERR_NOT_HELD)


# ------------------------------------------------------------------- sinks --

@pytest.mark.parametrize("window,sinks", [(5, -1), (-1, 5), (0, -1), (0, -2 ** 31)])
def test_attention_refuses_sinks(L, window, sinks):
    c, w = a_cache(), a_paged_ws()
    assert L.futr_paged_attention_sinks(ref(c), 0, 2, MEM, MEM, 3, MEM, 4, MEM, 256, MEM + 4096, 256, 0, 0.0, window, sinks,
                                        ref(w), None) == ARG
    # no rows: no work, but the arguments still have to be right
    assert L.futr_paged_attention_sinks(ref(c), 0, 2, MEM, MEM, 0, MEM, 4, MEM, 256, MEM + 4096, 256, 0, 0.0, window, sinks,
                                        ref(w), None) == ARG
    assert L.futr_paged_attention_sinks(ref(c), 0, 2, MEM, MEM, 0, MEM, 4, MEM, 256, MEM + 4096, 256, 0, 0.0, 7, 3, ref(w),
                                        None) == futr.FUTR_OK


# ------------------------------------------------------------------- beams --

@pytest.mark.parametrize("rows,keep", [(0, 4), (-1, 4), (65537, 4), (4, 0), (4, 65), (4, -1)])
def test_beam_workspace_refuses(L, rows, keep):
    n = C.c_size_t(7)
    assert L.futr_beam_workspace_size(rows, keep, C.byref(n)) == UNSUPPORTED and n.value == 7
    assert L.futr_beam_workspace_init(rows, keep, MEM, 1 << 30, C.byref(futr.futr_beam_ws()), None) == UNSUPPORTED
    with pytest.raises(futr.FutrError):
        futr.futr_beam_workspace_size(rows, keep)


def test_beam_workspace_refuses_null(L):
    assert L.futr_beam_workspace_size(4, 4, None) == ARG
    assert L.futr_beam_workspace_init(4, 4, None, 1 << 30, C.byref(futr.futr_beam_ws()), None) == ARG
    assert L.futr_beam_workspace_init(4, 4, MEM, 1 << 30, None, None) == ARG
    assert L.futr_beam_check(None, None) == ARG
    assert L.futr_beam_check(C.byref(futr.futr_beam_ws()), None) == ARG


SELECT = dict(logits=MEM, ld=1000, dtype=2, batch=2, beams=4, vocab=1000, scores=MEM, done=MEM, end=3, keep=4, stay=0,
              score_out=MEM + 64, parent=MEM, token=MEM, done_out=MEM + 64, ws=0)


@pytest.mark.parametrize("kw,want", [
    ({"logits": None}, ARG), ({"scores": None}, ARG), ({"score_out": None}, ARG), ({"parent": None}, ARG),
    ({"token": None}, ARG), ({"ws": None}, ARG), ({"ld": 999}, ARG), ({"ld": -1000}, ARG), ({"dtype": 3}, UNSUPPORTED),
    ({"dtype": -1}, UNSUPPORTED), ({"batch": 0}, ARG), ({"batch": 3}, ARG), ({"beams": 0}, UNSUPPORTED),
    ({"beams": 33}, UNSUPPORTED), ({"beams": -1}, UNSUPPORTED), ({"vocab": 0}, ARG), ({"vocab": -5}, ARG),
    ({"keep": 0}, UNSUPPORTED), ({"keep": 65}, UNSUPPORTED), ({"keep": 9}, ARG), ({"end": -1}, ARG), ({"end": -2}, ARG),
    ({"end": 1000}, ARG), ({"stay": 1, "keep": 5}, ARG), ({"logits": MEM + 2}, ARG), ({"logits": MEM + 1, "dtype": 0}, ARG),
    ({"score_out": MEM, "keep": 8}, ARG), ({"done_out": MEM, "keep": 8}, ARG),
    ({"batch": 2 ** 31 - 1, "beams": 32}, ARG),
])
def test_select_refuses(L, kw, want):
    a = dict(SELECT, **kw)
    w = a_beam_ws() if a["ws"] == 0 else None
    assert L.futr_beam_select(a["logits"], a["ld"], a["dtype"], a["batch"], a["beams"], a["vocab"], a["scores"], a["done"],
                              a["end"], a["keep"], a["stay"], a["score_out"], a["parent"], a["token"], a["done_out"],
                              ref(w), None) == want


@pytest.mark.parametrize("kw,want", [({"parent": None}, ARG), ({"pos": None}, ARG), ({"pos": MEM}, ARG), ({"batch": 0}, ARG),
                                     ({"batch": 41}, ARG), ({"batch": 33}, UNSUPPORTED), ({"kv": None}, ARG)])
def test_reorder_refuses(L, kw, want):
    a = dict(dict(kv=a_kv(), batch=4, parent=MEM, pos=MEM + 64), **kw)
    assert L.futr_kv_reorder(ref(a["kv"]), a["batch"], a["parent"], a["pos"], None) == want
    assert L.futr_kv_reorder(ref(futr.futr_kv()), 4, MEM, MEM + 64, None) == ARG


# ------------------------------------------------------------------- pages --

@pytest.mark.parametrize("n_pages,max_seqs,want", [(0, 4, ARG), (-1, 4, ARG), (8, 0, ARG), (8, -1, ARG),
                                                   (8, 1025, UNSUPPORTED)])
def test_pool_size_refuses(L, n_pages, max_seqs, want):
    n = C.c_size_t(7)
    assert L.futr_pages_size(n_pages, max_seqs, C.byref(n)) == want and n.value == 7
    assert L.futr_pages_init(n_pages, max_seqs, MEM, 1 << 40, C.byref(futr.futr_pages()), None) == want


def test_pool_init_refuses_memory(L):
    need, p = futr.futr_pages_size(100, 5), futr.futr_pages()
    assert L.futr_pages_size(100, 5, None) == ARG
    for mem, n, desc in ((None, need, p), (MEM, need - 1, p), (MEM + 16, need, p), (MEM, need, None)):
        assert L.futr_pages_init(100, 5, mem, n, None if desc is None else C.byref(desc), None) == ARG
    assert p.magic == 0
    assert futr.futr_pages_size(2 ** 31 - 1, 1024) > 4 * (2 ** 31 - 1) * 4    # counts and lists beyond 32 bits


def page_calls(L, c, p, batch=3, table=MEM, ld=4, pos=MEM, parent=MEM + 64, window=0, sinks=0, lo=0, hi=8):
    c, p = ref(c), ref(p)
    return {"hold": L.futr_pages_hold(c, p, batch, table, ld, None) if not (pos is None or parent is None) else ARG,
            "grow": L.futr_pages_grow(c, p, batch, pos, None, table, ld, None),
            "free": L.futr_pages_free(c, p, batch, pos, table, ld, window, sinks, None),
            "fork": L.futr_pages_fork(c, p, batch, parent, pos, table, ld, None),
            "compact": L.futr_pages_compact(c, p, batch, table, ld, lo, hi, None)}


@pytest.mark.parametrize("kw", [{"batch": 0}, {"batch": -1}, {"batch": 5}, {"table": None}, {"ld": 0}, {"ld": -4}])
def test_page_calls_refuse(L, kw):
    assert set(page_calls(L, a_cache(), a_pool(), **kw).values()) == {ARG}


def test_page_calls_refuse_descriptors(L):
    for c, p in ((None, a_pool()), (futr.futr_paged(), a_pool()), (a_cache(), None), (a_cache(), futr.futr_pages()),
                 (a_cache(9), a_pool(8))):
        assert set(page_calls(L, c, p).values()) == {ARG}
    assert L.futr_pages_check(None, None, None) == ARG
    assert L.futr_pages_check(C.byref(futr.futr_pages()), None, None) == ARG


def test_page_calls_refuse_their_own(L):
    c, p = ref(a_cache()), ref(a_pool())
    assert L.futr_pages_grow(c, p, 3, None, None, MEM, 4, None) == ARG
    assert L.futr_pages_free(c, p, 3, None, MEM, 4, 0, 0, None) == ARG
    assert L.futr_pages_free(c, p, 3, MEM, MEM, 4, -1, 0, None) == ARG
    assert L.futr_pages_free(c, p, 3, MEM, MEM, 4, 5, -1, None) == ARG
    assert L.futr_pages_fork(c, p, 3, None, MEM, MEM, 4, None) == ARG
    assert L.futr_pages_fork(c, p, 3, MEM, None, MEM, 4, None) == ARG
    assert L.futr_pages_fork(c, p, 3, MEM, MEM, MEM, 4, None) == ARG
    for lo, hi in ((-1, 8), (0, 9), (5, 4), (9, 9)):
        assert L.futr_pages_compact(c, p, 3, MEM, 4, lo, hi, None) == ARG


# ----------------------------------------------------------------- binding --

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
    """The binding is told that the current device is the tensors', and that every call of the library is a failure."""
    t = futr._Torch()
    t.device, t.stream = (lambda: -1), (lambda device: 0)

    class Never:
        def __getattr__(self, name):
            def called(*_):
                raise AssertionError(f"{name} was called")
            return called

    monkeypatch.setattr(futr, "_T", t)
    monkeypatch.setattr(futr, "lib", Never)
    return t


def select(**kw):
    a = dict(logits=torch.zeros((6, 50)), scores=torch.zeros((2, 3)), score_out=torch.zeros((2, 4)),
             parent=torch.zeros((2, 4), dtype=I32), token=torch.zeros((2, 4), dtype=I32), done=torch.zeros((2, 3), dtype=I32),
             done_out=torch.zeros((2, 4), dtype=I32), ws=a_beam_ws())
    a.update(kw)
    futr.futr_beam_select(a["logits"], a["scores"], a["score_out"], a["parent"], a["token"], a["ws"], done=a["done"],
                          done_out=a["done_out"], end=4)


@pytest.mark.parametrize("kw,error", [
    ({"logits": torch.zeros((6, 50), dtype=torch.float64)}, TypeError), ({"logits": torch.zeros((5, 50))}, ValueError),
    ({"logits": torch.zeros((50, 6)).t()}, ValueError), ({"logits": torch.zeros(300)}, ValueError),
    ({"logits": torch.zeros((2, 3, 50))}, ValueError), ({"logits": torch.zeros((6, 100))[:, ::2]}, ValueError),
    ({"logits": _Elsewhere(torch.zeros((6, 50)))}, ValueError), ({"scores": torch.zeros(6)}, ValueError),
    ({"scores": torch.zeros((2, 3), dtype=torch.float64)}, ValueError), ({"scores": torch.zeros((2, 6))[:, ::2]}, ValueError),
    ({"score_out": torch.zeros((3, 4))}, ValueError), ({"score_out": torch.zeros(8)}, ValueError),
    ({"parent": torch.zeros((2, 3), dtype=I32)}, ValueError), ({"parent": torch.zeros((2, 4))}, ValueError),
    ({"token": torch.zeros((2, 4), dtype=torch.int64)}, ValueError), ({"done": torch.zeros((2, 4), dtype=I32)}, ValueError),
    ({"done_out": torch.zeros((2, 3), dtype=I32)}, ValueError), ({"done": torch.zeros((2, 3), dtype=torch.bool)}, ValueError),
])
def test_binding_refuses_select(binding, kw, error):
    with pytest.raises(error):
        select(**kw)


def test_binding_refuses_handles_of_another_device(binding):
    far = _Elsewhere(torch.zeros(1))
    w, kv, c, p = a_beam_ws(), a_kv(), a_cache(), a_pool()
    table, pos = torch.zeros((3, 4), dtype=I32), torch.zeros(3, dtype=I32)
    w._mem = kv._mem = far
    with pytest.raises(ValueError, match="workspace"):
        select(ws=w)
    with pytest.raises(ValueError, match="cache"):
        futr.futr_kv_reorder(kv, pos, pos.clone())
    c._mem = far
    with pytest.raises(ValueError, match="cache"):
        futr.futr_pages_hold(c, p, table)
    c._mem, p._mem = torch.zeros(1), far
    with pytest.raises(ValueError, match="pool"):
        futr.futr_pages_free(c, p, pos, table)


@pytest.mark.parametrize("bad", [torch.zeros(3), torch.zeros(3, dtype=torch.int64), torch.zeros(4, dtype=I32),
                                 torch.zeros(6, dtype=I32)[::2], torch.zeros((3, 1), dtype=I32),
                                 _Elsewhere(torch.zeros(3, dtype=I32))])
def test_binding_refuses_positions_and_parents(binding, bad):
    c, p, table, good = a_cache(), a_pool(), torch.zeros((3, 4), dtype=I32), torch.zeros(3, dtype=I32)
    for call in (lambda: futr.futr_pages_grow(c, p, bad, None, table), lambda: futr.futr_pages_free(c, p, bad, table),
                 lambda: futr.futr_pages_fork(c, p, bad, good, table), lambda: futr.futr_pages_fork(c, p, good, bad, table),
                 lambda: futr.futr_pages_grow(c, p, good, bad if bad.shape != (4,) else good, table),
                 lambda: futr.futr_kv_reorder(a_kv(), good, bad)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("bad", [torch.zeros(12, dtype=I32), torch.zeros((3, 4), dtype=torch.int64),
                                 torch.zeros((3, 8), dtype=I32)[:, ::2], _Elsewhere(torch.zeros((3, 4), dtype=I32))])
def test_binding_refuses_tables(binding, bad):
    c, p, good = a_cache(), a_pool(), torch.zeros(3, dtype=I32)
    for call in (lambda: futr.futr_pages_hold(c, p, bad), lambda: futr.futr_pages_grow(c, p, good, None, bad),
                 lambda: futr.futr_pages_free(c, p, good, bad), lambda: futr.futr_pages_fork(c, p, good, good.clone(), bad),
                 lambda: futr.futr_pages_compact(c, p, bad, 0)):
        with pytest.raises(ValueError):
            call()


# -------------------------------------------------------- the restatements --

def test_pool_by_hand():
    p = Pool(10, 16, 3, 4)
    assert p.grow([0, 0, 0], [33, 16, 0]) and p.table == [[0, 1, 2, -1], [3, -1, -1, -1], [-1] * 4]
    copies, pos = p.fork([0, 0, 1], [33, 16, 0])
    assert copies == [(2, 4, 1)] and pos == [33, 33, 16]
    assert p.table == [[0, 1, 2, -1], [0, 1, 4, -1], [3, -1, -1, -1]] and p.refs()[:5] == [2, 2, 1, 1, 1]
    p.give([33, 30, 0])
    assert p.table == [[0, 1, 2, -1], [0, 1, -1, -1], [-1] * 4] and p.free() == [3, 4, 5, 6, 7, 8, 9]
    p.give([33, 30, 0], window=2, sinks=1)       # rows from 33 on see 32, 33, .. and 0; from 30 on 29, .. and 0
    assert p.table == [[0, -1, 2, -1], [0, 1, -1, -1], [-1] * 4]
    assert p.compact(0, 2) == {0: 3, 1: 4} and p.table == [[3, -1, 2, -1], [3, 4, -1, -1], [-1] * 4]
    assert p.compact(0, 5) == {2: 5, 3: 6, 4: 7} and p.compact(1, 10) is None
    assert not p.grow([0, 0, 0], [64, 64, 64])


def test_beams_by_hand():
    x = torch.log(torch.tensor([[0.5, 0.25, 0.25], [0.1, 0.1, 0.8]], dtype=torch.float64)) + 7.0
    v, bad = beam_values(x, torch.zeros((1, 2)))
    assert torch.allclose(v.exp(), torch.tensor([[0.5, 0.25, 0.25, 0.1, 0.1, 0.8]], dtype=torch.float64)) and not bad.any()
    best, at = beam_best(torch.tensor([[1.0, 3.0, 3.0, -float("inf")]], dtype=torch.float64), 5)
    assert at.tolist() == [[1, 2, 0, -1, -1]]
    v, _ = beam_values(x, torch.tensor([[-1.0, -2.0]]), torch.tensor([[0, 1]]), end=1)
    assert v[0, 3:].tolist() == [-float("inf"), -2.0, -float("inf")]
