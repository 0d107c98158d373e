"""Attention over the paged cache with a window and first tokens that stay visible, against 64 bits."""
import ctypes as C
import math

import pytest
import torch

from int4_weight_kv_w4a16_gb300 import futr
from tests._gpu_helpers import ensure_lib
from tests._paged_ref import F64, Paged, ints, rotate, starts

pytestmark = pytest.mark.gpu
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def rows(n, heads, d, dtype, seed, fused=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((n, heads + (3 if fused else 0), d), generator=g, device="cuda")
    return x.to(dtype)[:, 1:1 + heads] if fused else x.to(dtype)


def visible(p, j, window, sinks):
    return (j <= p) & ((j > p - window) | (j < sinks)) if window else j <= p


def exact(c, q, pos, counts, window, sinks, layer=0):
    """Outputs in 64 bits, and what the kernels' roundings may add: a weight's 2^-11, and a query's 2^-11 in a
    score (twice, above and below the fraction) times the mean magnitude of the values."""
    out = torch.zeros(q.shape, dtype=F64, device="cuda")
    bound = torch.zeros_like(out)
    G, r, scale = c.heads // c.kv_heads, 0, c.d ** -0.5
    for b, n in enumerate(counts):
        if n:
            at = torch.arange(pos[b], pos[b] + n, device="cuda")
            x = q[r:r + n].to(F64)
            x = (rotate(x, at, c.shape.rope_theta) if c.rope else x).transpose(0, 1)
            k, v = (t.repeat_interleave(G, 0) for t in c.values(b, pos[b] + n, layer))
            s = x @ k.transpose(1, 2) * scale
            see = visible(at[:, None], torch.arange(pos[b] + n, device="cuda"), window, sinks)
            s[:, ~see] = -math.inf
            w = torch.softmax(s, -1)
            out[r:r + n] = (w @ v).transpose(0, 1)
            spread = (w @ v.abs()).transpose(0, 1)
            mag = (x.abs() @ k.abs().transpose(1, 2) * scale).masked_fill(s == -math.inf, 0).amax(-1)
            moved = (2.0 ** -11 + 2.0 ** -18) * mag.transpose(0, 1)[..., None]
            bound[r:r + n] = (2.0 ** -11 + 2.0 ** -16 + 2 * moved) * spread
        r += n
    return out, bound


def run(c, q, pos, counts, window, sinks, start=True, layer=0):
    out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
    futr.futr_paged_attention(c.cache, layer, len(pos), ints(pos), starts(counts) if start else None, c.table, q, out,
                              c.ws, window=window, sinks=sinks)
    assert futr.futr_paged_check(c.cache, c.ws) == futr.FUTR_OK
    return out


def check(c, q, got, pos, counts, window, sinks, layer=0):
    want, bound = exact(c, q, pos, counts, window, sinks, layer)
    err = (got.to(F64) - want).abs()
    tol = HALF_STEP[q.dtype] * want.abs() + bound + 2.0 ** -24
    assert bool((err <= tol).all()), float((err / tol).max())
    assert float(err.norm() / want.norm()) <= 2 * HALF_STEP[q.dtype] + 2.0 ** -9


def give_back(c, pos, counts, window, sinks):
    """The table without the pages that no row sees."""
    i = torch.arange(c.table.shape[1], device="cuda")
    p = ints(pos)[:, None]
    gone = (i * c.page >= sinks) & ((i + 1) * c.page <= p - window + 1)
    c.table[gone] = -1


CASES = [
    # heads, kv-heads, d, page, type, fused, window, sinks, positions, rows of each sequence
    (32, 8, 128, 64, torch.bfloat16, True, 300, 4, [2000, 299, 300, 0, 3000], [1] * 5),
    (8, 2, 64, 16, torch.float16, False, 17, 1, [5, 16, 17, 18, 1000, 127, 128, 129, 145, 146, 272], [1] * 11),
    (8, 8, 128, 32, torch.bfloat16, False, 128, 128, [127, 128, 255, 256, 257, 1111], [1] * 6),
    (16, 1, 128, 128, torch.float16, False, 1, 129, [0, 1, 128, 129, 130, 2047], [1] * 6),
    (4, 4, 64, 64, torch.bfloat16, True, 1000, 700, [500, 1700, 1701, 5000], [3, 1, 4, 8]),
    (5, 1, 128, 16, torch.bfloat16, False, 100, 5000, [300, 4000], [2, 5]),            # sinks that hold everything
    (32, 8, 128, 64, torch.bfloat16, True, 500, 4, [3000, 40, 700], [300, 200, 0]),    # chunks
    (8, 2, 128, 32, torch.float16, False, 129, 100, [0, 1000, 256], [700, 130, 257]),
    (16, 4, 64, 16, torch.bfloat16, False, 64, 300, [2000, 100], [400, 600]),
    (16, 2, 64, 128, torch.float16, True, 1, 1, [1500], [350]),
    (32, 2, 128, 64, torch.bfloat16, False, 700, 33, [1 + 97 * i for i in range(40)], [1] * 39 + [400]),   # both kernels
    (8, 2, 64, 32, torch.float16, False, 40, 20, [i * 31 for i in range(70)], [1 + i % 3 for i in range(70)]),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_sinks(case):
    heads, hkv, d, page, dtype, fused, window, sinks, pos, counts = CASES[case]
    width = -(-max(p + n for p, n in zip(pos, counts)) // page) + 1
    c = Paged(heads, hkv, d, page, len(pos), width, layers=2)
    c.fill(case, layer=1)
    q = rows(sum(counts), heads, d, dtype, case + 50, fused)
    got = run(c, q, pos, counts, window, sinks, layer=1)
    check(c, q, got, pos, counts, window, sinks, layer=1)
    assert torch.equal(run(c, q, pos, counts, window, sinks, layer=1), got)   # no sum depends on timing
    if all(n == 1 for n in counts):
        assert torch.equal(run(c, q, pos, counts, window, sinks, start=False, layer=1), got)
    # the pages in between may be gone, and what they hold may be anything
    give_back(c, pos, counts, window, sinks)
    held = c.table[c.table >= 0].unique()
    rest = torch.ones(c.n_pages, dtype=torch.bool, device="cuda")
    rest[held.long()] = False
    c.codes.view(torch.uint8)[1, rest] = 0x7F
    c.scales[1, rest] = math.nan
    assert torch.equal(run(c, q, pos, counts, window, sinks, layer=1), got)


@pytest.mark.parametrize("n", [1, 150], ids=["token", "chunk"])
def test_sinks_without_effect(n):
    """No sinks, no window, and windows of everything give what futr_paged_attention gives."""
    c = Paged(4, 2, 128, 64, 1, 8)
    c.fill(8)
    q = rows(n, 4, 128, torch.bfloat16, 12)
    plain = run(c, q, [300], [n], 0, 0)
    for window, sinks in ((0, 5), (0, 2 ** 31 - 1), (300 + n, 3), (2 ** 31 - 1, 2 ** 31 - 1), (5, 2 ** 31 - 1), (1, 300 + n)):
        got = run(c, q, [300], [n], window, sinks)
        check(c, q, got, [300], [n], 0, 0)
        if window in (0, 2 ** 31 - 1):
            assert torch.equal(got, plain)
    windowed = run(c, q, [300], [n], 40, 0)
    assert torch.equal(run(c, q, [300], [n], 40, 0), windowed)
    check(c, q, windowed, [300], [n], 40, 0)


def test_a_sink_takes_the_weight():
    """Nearly all of the weight on the first token, far behind the window: the other rows' sums start low and
    rescale, or start high and vanish."""
    for where, sinks in ((0, 1), (3, 4), (130, 131)):
        for n in (1, 140):
            c = Paged(4, 1, 128, 16, 1, 200, rope=False)
            c.fill(2, gain=1.0)
            q = rows(n, 4, 128, torch.bfloat16, 9)
            q = q[:, :1].expand(-1, 4, -1).contiguous()
            line = torch.sign(q[0, 0].float())
            page, slot = int(c.table[0, where // 16]), where % 16
            c.codes[0, page, 0, 0, slot] = (448 * line).to(torch.float8_e4m3fn)
            check(c, q, run(c, q, [3000], [n], 50, sinks), [3000], [n], 50, sinks)


@pytest.mark.parametrize("n", [1, 100], ids=["token", "chunk"])
def test_missing_sinks_are_not_visible(n):
    """A page of sinks that the table does not have is reported and counts as not visible; with nothing left: zeros."""
    c = Paged(8, 2, 64, 16, 1, 80)
    c.fill(1)
    q = rows(n, 8, 64, torch.bfloat16, 2)
    want = run(c, q, [1000], [n], 60, 0)
    c.table[0, :2] = -1
    out = torch.empty_like(q)
    futr.futr_paged_attention(c.cache, 0, 1, ints([1000]), starts([n]), c.table, q, out, c.ws, window=60, sinks=20)
    assert futr.futr_paged_check(c.cache, c.ws) == futr.FUTR_ERR_OUT_OF_RANGE
    assert float((out.double() - want.double()).norm() / want.double().norm()) <= 2.0 ** -8
    c.table.fill_(-1)
    futr.futr_paged_attention(c.cache, 0, 1, ints([1000]), starts([n]), c.table, q, out, c.ws, window=60, sinks=20)
    assert futr.futr_paged_check(c.cache, c.ws) == futr.FUTR_ERR_OUT_OF_RANGE
    assert bool((out == 0).all())


def test_a_long_answer_in_few_pages():
    """A graph that takes pages, appends, attends and gives back, over many times the pool's positions."""
    heads, hkv, d, page, window, sinks, B = 8, 2, 64, 16, 40, 5, 3
    c = Paged(heads, hkv, d, page, B, 200)                       # every position kept: the comparison
    cs = c.cs
    n_pages = B * 6
    size = futr.futr_paged_size(cs, 1, n_pages, page, 200 * page)
    cache = futr.futr_paged_init(cs, 1, n_pages, page, 200 * page, True, futr.alloc_bytes(size))
    pool = futr.futr_pages_init(n_pages, B, futr.alloc_bytes(futr.futr_pages_size(n_pages, B)))
    ws = futr.futr_paged_workspace_init(cs, futr.alloc_bytes(futr.futr_paged_workspace_size(cs)))
    table = torch.full((B, 200), -1, dtype=torch.int32, device="cuda")
    pos = ints([0] * B)
    q, k, v = (rows(B, h, d, torch.bfloat16, h) for h in (heads, hkv, hkv))
    out, want = torch.empty_like(q), torch.empty_like(q)

    def step():
        futr.futr_pages_free(cache, pool, pos, table, window=window, sinks=sinks)
        futr.futr_pages_grow(cache, pool, pos, None, table)
        futr.futr_paged_append(cache, 0, B, pos, None, table, k, v)
        futr.futr_paged_attention(cache, 0, B, pos, None, table, q, out, ws, window=window, sinks=sinks)
        pos.add_(1)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    pos.zero_()
    for i in range(600):
        for t, s in ((q, 1), (k, 2), (v, 3)):
            t.copy_(rows(B, t.shape[1], d, torch.bfloat16, 10 * i + s))
        graph.replay()
        p = ints([i] * B)
        futr.futr_paged_append(c.cache, 0, B, p, None, c.table, k, v)
        futr.futr_paged_attention(c.cache, 0, B, p, None, c.table, q, want, c.ws, window=window, sinks=sinks)
        assert torch.equal(out, want), i
    assert futr.futr_pages_check(pool)[0] == futr.FUTR_OK and futr.futr_paged_check(cache, ws) == futr.FUTR_OK


@pytest.mark.parametrize("n", [1, 3, 150], ids=["token", "draft", "chunk"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_the_entry_point_without_sinks(n, dtype):
    """futr_paged_attention by its own name, with windows and scales: what the one with sinks gives for none, bit for
    bit, and right."""
    c = Paged(8, 2, 64, 32, 2, 30)
    c.fill(4)
    pos, counts = [700, 64], [n, n]
    q = rows(2 * n, 8, 64, dtype, 30 + n)
    p, s, stream = ints(pos), starts(counts), torch.cuda.current_stream().cuda_stream
    kind = futr.FUTR_DTYPE_F16 if dtype == torch.float16 else futr.FUTR_DTYPE_BF16
    for window in (0, 1, 40, 300, 2 ** 31 - 1):
        for scale in (0.0, 0.05, 0.5):
            args = [C.addressof(c.cache), 0, 2, p.data_ptr(), s.data_ptr(), 2 * n, c.table.data_ptr(), c.table.shape[1],
                    q.data_ptr(), q.stride(0)]
            outs = [torch.full_like(q, 7.0) for _ in range(2)]
            assert futr.lib().futr_paged_attention(*args, outs[0].data_ptr(), q.stride(0), kind, scale, window,
                                                   C.addressof(c.ws), stream) == futr.FUTR_OK
            assert futr.lib().futr_paged_attention_sinks(*args, outs[1].data_ptr(), q.stride(0), kind, scale, window, 0,
                                                         C.addressof(c.ws), stream) == futr.FUTR_OK
            assert futr.futr_paged_check(c.cache, c.ws) == futr.FUTR_OK
            assert torch.equal(outs[0], outs[1])
            if scale == 0.0:
                check(c, q, outs[0], pos, counts, window, 0)
                default = outs[0]
            else:
                assert not torch.equal(outs[0], default) or window == 1
