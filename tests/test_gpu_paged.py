"""Paged 8-bit cache: append and attention against plain 64-bit forms."""
import math

import pytest
import torch

from int4_weight_kv_w4a16_gb300 import futr
from tests._gpu_helpers import ensure_lib
from tests._paged_ref import F64, Paged, ints, page_scale, rotate, starts

pytestmark = pytest.mark.gpu

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def rows(n, heads, d, dtype, seed, fused=False, gain=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((n, heads + (3 if fused else 0), d), generator=g, device="cuda") * gain
    return x.to(dtype)[:, 1:1 + heads] if fused else x.to(dtype)


# ----------------------------------------------------------------- append --

def check_append(c, before, k, v, pos, counts, layer=0):
    """Codes and scales of the touched pages against the definition in 64 bits.

    A code is e4m3's rounding of x / s: off by half a step, 2^-4 |x| + 2^-10 s, and x
    itself by the rotation's three fp32 roundings, 3 * 2^-24 (|x1| + |x2|)."""
    codes0, scales0 = before
    x = torch.stack([k.to(F64), v.to(F64)], 2)                                       # [rows, kv-heads, 2, d]
    at = torch.tensor([pos[b] + i for b, n in enumerate(counts) for i in range(n)], device="cuda")
    seq = [b for b, n in enumerate(counts) for _ in range(n)]
    slack = torch.zeros_like(x)
    if c.rope:
        x[:, :, 0] = rotate(x[:, :, 0], at, c.shape.rope_theta)
        d = c.d
        mag = k.to(F64).abs()
        slack[:, :, 0] = 3 * 2.0 ** -24 * torch.cat([mag[..., :d // 2] + mag[..., d // 2:]] * 2, -1)
    touched = {}
    for i, (b, p) in enumerate(zip(seq, at.tolist())):
        touched.setdefault(int(c.table[b, p // c.page]), []).append((i, p % c.page))
    for page in range(c.n_pages):
        new, old = c.codes[layer, page].to(F64), codes0[page].to(F64)
        if page not in touched:
            assert torch.equal(new, old) and torch.equal(c.scales[layer, page], scales0[page]), page
            continue
        idx, slots = [t[0] for t in touched[page]], [t[1] for t in touched[page]]
        amax = x[idx].abs().amax((0, 3))
        for h in range(c.kv_heads):
            for w in range(2):
                s_old = 0.0 if 0 in slots else float(scales0[page, h, w])
                s = max(s_old, page_scale(float(amax[h, w])))
                assert float(c.scales[layer, page, h, w]) == s, (page, h, w)
                err = (new[h, w, slots] * s - x[idx, h, w]).abs()
                tol = 2.0 ** -4 * x[idx, h, w].abs() + 2.0 ** -10 * s + slack[idx, h, w]
                assert bool((err <= tol).all()), (page, h, w, float((err - tol).max()))
                keep = [j for j in range(c.page) if j not in slots]
                want = old[h, w, keep]
                if s_old > 0 and s > s_old:
                    want = (want * (s_old / s)).float().to(torch.float8_e4m3fn).to(F64)
                assert torch.equal(new[h, w, keep], want), (page, h, w)


APPEND = [
    # page, d, kv-heads, rope, dtype, fused, positions, rows of each sequence
    (16, 128, 8, True, torch.bfloat16, False, [0], [1]),
    (16, 64, 2, True, torch.float16, False, [15, 16, 17], [1, 1, 1]),
    (32, 128, 2, True, torch.bfloat16, True, [5, 0, 63], [3, 0, 66]),
    (64, 64, 4, True, torch.float16, True, [0, 1], [257, 63]),
    (64, 128, 1, False, torch.bfloat16, False, [60, 7], [9, 1]),
    (128, 128, 4, True, torch.float16, False, [127, 255, 3], [2, 1, 300]),
    (16, 128, 2, True, torch.bfloat16, False, list(range(3, 40)), [1 + i % 3 for i in range(37)]),
]


@pytest.mark.parametrize("case", range(len(APPEND)))
@pytest.mark.parametrize("gain", [1.0, 37.0], ids=["same", "grown"])
def test_append(case, gain):
    page, d, hkv, rope, dtype, fused, pos, counts = APPEND[case]
    width = -(-max(p + n for p, n in zip(pos, counts)) // page) + 1
    c = Paged(2 * hkv, hkv, d, page, len(pos), width, layers=2, rope=rope)
    c.fill(1, layer=1)
    other = c.codes[0].clone()
    before = c.codes[1].clone(), c.scales[1].clone()
    n = sum(counts)
    k, v = rows(n, hkv, d, dtype, 2, fused, gain), rows(n, hkv, d, dtype, 3, fused, gain)
    futr.futr_paged_append(c.cache, 1, len(pos), ints(pos), starts(counts), c.table, k, v)
    assert futr.futr_paged_check(c.cache) == futr.FUTR_OK
    check_append(c, before, k, v, pos, counts, layer=1)
    assert torch.equal(c.codes[0].view(torch.uint8), other.view(torch.uint8))
    # the same rows again change nothing
    once = c.codes[1].clone(), c.scales[1].clone()
    futr.futr_paged_append(c.cache, 1, len(pos), ints(pos), starts(counts), c.table, k, v)
    assert torch.equal(c.codes[1].view(torch.uint8), once[0].view(torch.uint8)) and torch.equal(c.scales[1], once[1])


def test_append_grows_a_page_token_by_token():
    """A page whose every token is twice the last: each growth halves the old codes, and
    a value keeps its first rounding until it reaches e4m3's subnormals."""
    c = Paged(2, 1, 128, 16, 1, 1, rope=False)
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((16, 1, 128), generator=g, device="cuda") * 2.0 ** torch.arange(16, device="cuda")[:, None, None]
    x = x.to(torch.bfloat16)
    for i in range(16):
        futr.futr_paged_append(c.cache, 0, 1, ints([i]), None, c.table, x[i:i + 1], x[i:i + 1])
    assert futr.futr_paged_check(c.cache) == futr.FUTR_OK
    k, v = c.values(0, 16)
    s = page_scale(float(x.abs().max()))
    assert float(c.scales[0, int(c.table[0, 0]), 0, 0]) == s
    for t in (k, v):
        err = (t[0] - x[:, 0].to(F64)).abs()
        # half a step at first; each of the 15 growths may cost a subnormal half its step, at scales
        # that double: in all less than 2 * 2^-10 s
        assert bool((err <= 2.0 ** -4 * x[:, 0].to(F64).abs() + 2 * 2.0 ** -10 * s).all())


def test_append_values_of_every_size():
    """Zeros, subnormals, the largest bf16 values and ties."""
    c = Paged(2, 1, 64, 16, 6, 1, rope=False)
    x = torch.zeros((6, 1, 64), dtype=torch.bfloat16, device="cuda")
    x[1] = 1e-40
    x[2] = 3.38e38
    x[3, 0, :32], x[3, 0, 32:] = 448.0, 0.0009765625   # 2^-10: half of e4m3's smallest, a tie to zero
    x[4, 0] = 1.0625                                     # between 1 and 1.125: a tie to 1
    x[4, 0, 0] = 448.0
    x[5, 0] = -449.0                                     # bf16 rounds it to 448 or 450: the scale follows
    futr.futr_paged_append(c.cache, 0, 6, ints([0] * 6), None, c.table, x, x)
    assert futr.futr_paged_check(c.cache) == futr.FUTR_OK
    for b in range(6):
        k, v = c.values(b, 1)
        s = page_scale(float(x[b].abs().max()))
        assert float(c.scales[0, int(c.table[b, 0]), 0, 0]) == s
        want = (x[b, 0].to(F64) / s).float().to(torch.float8_e4m3fn).to(F64) * s
        assert torch.equal(k[0, 0], want) and torch.equal(v[0, 0], want), b


def test_append_reports_what_is_not_finite():
    c = Paged(2, 1, 64, 16, 2, 1)
    x = rows(2, 1, 64, torch.bfloat16, 3)
    y = x.clone()
    y[0, 0, 5], y[1, 0, 9] = math.inf, math.nan
    futr.futr_paged_append(c.cache, 0, 2, ints([0, 3]), None, c.table, x, y)
    assert futr.futr_paged_check(c.cache) == futr.FUTR_ERR_NOT_FINITE
    assert futr.futr_paged_check(c.cache) == futr.FUTR_OK
    z = x.clone()
    z[0, 0, 5], z[1, 0, 9] = 0.0, 0.0
    assert bool(torch.isfinite(c.codes.to(torch.float32)).all())
    for b, p in ((0, 0), (1, 3)):
        v = c.values(b, p + 1)[1][0, p]
        s = page_scale(float(z[b].abs().max()))
        assert torch.equal(v, (z[b, 0].to(F64) / s).float().to(torch.float8_e4m3fn).to(F64) * s)


# -------------------------------------------------------------- attention --

ATTN = [
    # heads, kv-heads, d, page, dtype, fused, window, positions, rows of each sequence
    (32, 8, 128, 16, torch.bfloat16, False, 0, [0], [1]),
    (32, 8, 128, 16, torch.bfloat16, False, 0, [1023], [1]),
    (32, 8, 128, 64, torch.bfloat16, True, 0, [3, 64, 1000, 127, 15], [1, 1, 1, 1, 1]),
    (8, 1, 128, 128, torch.float16, False, 0, [5000, 40], [1, 1]),
    (10, 2, 64, 32, torch.float16, True, 0, [77, 200], [1, 1]),
    (28, 4, 128, 32, torch.bfloat16, False, 100, [90, 99, 100, 101, 700], [1, 1, 1, 1, 1]),
    (32, 2, 64, 16, torch.bfloat16, False, 0, [333, 12], [1, 1]),
    (16, 1, 128, 64, torch.float16, False, 0, [2000], [1]),
    (32, 8, 128, 64, torch.bfloat16, True, 0, [0, 5, 300], [37, 0, 4]),
    (16, 4, 64, 16, torch.float16, False, 33, [0, 250], [70, 5]),
    (4, 4, 128, 128, torch.bfloat16, False, 0, [100, 0, 1], [130, 1, 0]),
    (64, 8, 128, 64, torch.bfloat16, False, 1, [70, 0], [3, 2]),
    (16, 16, 64, 64, torch.bfloat16, True, 0, [i * 37 % 400 for i in range(45)], [1 + (i % 5 == 0) for i in range(45)]),
]


# many rows a sequence: heads, kv-heads, d, page, dtype, fused, window, positions, rows
CHUNKS = [
    (4, 4, 128, 64, torch.bfloat16, False, 0, [0], [128]),
    (4, 4, 128, 64, torch.bfloat16, False, 0, [1], [129]),
    (8, 2, 128, 16, torch.bfloat16, True, 0, [0], [64]),
    (32, 8, 128, 64, torch.bfloat16, True, 0, [700, 0, 130], [130, 65, 1]),
    (8, 2, 128, 128, torch.float16, False, 0, [250], [257]),
    (16, 2, 128, 32, torch.bfloat16, False, 200, [1000, 0], [90, 300]),
    (16, 1, 128, 32, torch.bfloat16, False, 0, [77], [100]),
    (10, 2, 64, 16, torch.float16, True, 0, [33, 500, 4], [60, 200, 0]),
    (8, 8, 64, 128, torch.bfloat16, False, 50, [0, 10], [256, 255]),
    (28, 4, 128, 64, torch.float16, False, 0, [2000, 1], [3, 150]),
    (4, 1, 64, 64, torch.bfloat16, False, 0, [3000], [500]),
    (16, 1, 64, 32, torch.bfloat16, False, 0, [i * 53 % 300 for i in range(40)], [5 + i % 7 for i in range(40)]),
    (16, 2, 128, 16, torch.bfloat16, True, 40, [2 * i for i in range(35)], [20 * (i % 3) for i in range(35)]),
]


@pytest.mark.parametrize("case", range(len(CHUNKS)))
def test_attention_chunks(case):
    heads, hkv, d, page, dtype, fused, window, pos, counts = CHUNKS[case]
    width = -(-max(p + n for p, n in zip(pos, counts)) // page) + 1
    c = Paged(heads, hkv, d, page, len(pos), width)
    c.fill(case)
    q = rows(sum(counts), heads, d, dtype, case + 70, fused)
    got = run_attention(c, q, pos, counts, window)
    check_attention(c, q, got, pos, counts, window)
    for _ in range(3):
        assert torch.equal(run_attention(c, q, pos, counts, window), got)   # no sum depends on timing


def run_attention(c, q, pos, counts, window=0, start=True, scale=0.0, layer=0):
    out = torch.full((q.shape[0] + 2, c.heads, c.d), 7.0, dtype=q.dtype, device="cuda")
    futr.futr_paged_attention(c.cache, layer, len(pos), ints(pos), starts(counts) if start else None, c.table, q,
                              out[1:-1], c.ws, scale=scale, window=window)
    assert futr.futr_paged_check(c.cache, c.ws) == futr.FUTR_OK
    assert bool((out[0] == 7).all()) and bool((out[-1] == 7).all())
    return out[1:-1]


def check_attention(c, q, got, pos, counts, window=0, scale=None, layer=0):
    """The output's rounding, half a step, and what the operands' fp16 roundings
    can move it by: 2^-11 of each weight, and of the query, whose score error
    moves a weight by as much relatively."""
    want, bound = c.attention(q, pos, counts, window, scale, layer)
    err = (got.to(F64) - want).abs()
    tol = HALF_STEP[q.dtype] * want.abs() + bound + 2.0 ** -24
    assert bool((err <= tol).all()), float((err / tol).max())
    assert float(err.norm() / want.norm()) <= 2 * HALF_STEP[q.dtype] + 2.0 ** -9


@pytest.mark.parametrize("case", range(len(ATTN)))
def test_attention(case):
    heads, hkv, d, page, dtype, fused, window, pos, counts = ATTN[case]
    width = -(-max(p + n for p, n in zip(pos, counts)) // page) + 1
    c = Paged(heads, hkv, d, page, len(pos), width, layers=2)
    c.fill(case, layer=1)
    q = rows(sum(counts), heads, d, dtype, case + 50, fused)
    got = run_attention(c, q, pos, counts, window, layer=1)
    check_attention(c, q, got, pos, counts, window, layer=1)
    again = run_attention(c, q, pos, counts, window, layer=1)
    assert torch.equal(again, got)   # no sum depends on timing
    if all(n == 1 for n in counts):
        assert torch.equal(run_attention(c, q, pos, counts, window, start=False, layer=1), got)


def test_pages_before_the_window_are_not_read():
    """A program may give pages back that no row can see any more."""
    c = Paged(8, 2, 128, 16, 2, 40)
    c.fill(2)
    for counts in ([1, 1], [100, 90]):
        pos, window = [400, 371], 60
        q = rows(sum(counts), 8, 128, torch.bfloat16, 8)
        got = run_attention(c, q, pos, counts, window)
        table = c.table.clone()
        for b in range(2):
            c.table[b, :(pos[b] - window + 1) // 16] = -1
        assert torch.equal(run_attention(c, q, pos, counts, window), got)
        c.table = table


def test_attention_scale_and_large_scores():
    """A scale of its own, and scores so far apart that one key takes the whole weight."""
    c = Paged(8, 2, 128, 32, 2, 20)
    c.fill(3)
    q = rows(2, 8, 128, torch.float16, 4)
    check_attention(c, q, run_attention(c, q, [600, 31], [1, 1], scale=0.01), [600, 31], [1, 1], scale=0.01)
    q = (q * 300).to(torch.float16)
    got = run_attention(c, q, [600, 31], [1, 1]).to(F64)
    want, _ = c.attention(q, [600, 31], [1, 1])
    assert bool(torch.isfinite(got).all())
    # a score can move by more than 1 here: the output is still a mean of the values
    assert float(got.abs().max()) <= float(c.values(0, 601)[1].abs().max()) * (1 + 2.0 ** -10)
    assert float((got - want).norm() / want.norm()) < 0.2


def test_attention_pages_of_very_different_value_scales():
    """Value scales 2^40 apart: the page that holds the weight decides, large or small."""
    c = Paged(4, 1, 128, 16, 1, 8, rope=False)
    c.fill(2, gain=1.0)
    ids = c.table[0].long()
    c.scales[0, ids[1], 0, 1] *= 2.0 ** 40
    c.scales[0, ids[3], 0, 1] *= 2.0 ** -40
    c.codes[0, ids[5], 0, 1] = torch.zeros((16, 128), device="cuda").to(torch.float8_e4m3fn)
    c.scales[0, ids[5], 0, 1] = 2.0 ** -60
    q = rows(1, 4, 128, torch.bfloat16, 9)
    check_attention(c, q, run_attention(c, q, [127], [1]), [127], [1])
    # all weight on one page: its keys along the query, the others against it
    for hot in (3, 5, 0):
        c.fill(2, gain=1.0)
        c.scales[0, ids[1], 0, 1] *= 2.0 ** 40
        c.scales[0, ids[3], 0, 1] *= 2.0 ** -40
        c.scales[0, ids[5], 0, 1] *= 2.0 ** -20
        line = torch.sign(q[0, 0].float())
        for j in range(8):
            sign = 1.0 if j == hot else -1.0
            c.codes[0, ids[j], 0, 0] = (sign * 448 * line).expand(16, -1).to(torch.float8_e4m3fn)
            c.scales[0, ids[j], 0, 0] = 2.0 ** -6
        one = q[:, :1].expand(-1, 4, -1).contiguous()
        check_attention(c, one, run_attention(c, one, [127], [1]), [127], [1])


def test_attention_ignores_what_unwritten_slots_hold():
    """NaN codes and any scale behind the last token, and in pages of no one, change nothing."""
    c = Paged(8, 2, 64, 32, 2, 4)
    c.fill(1)
    pos, counts = [40, 3], [2, 1]
    q = rows(3, 8, 64, torch.bfloat16, 2)
    got = run_attention(c, q, pos, counts)
    bits = c.codes.view(torch.uint8)
    used = {int(c.table[0, 0]): 32, int(c.table[0, 1]): 10, int(c.table[1, 0]): 4}
    for p in range(c.n_pages):
        bits[0, p, :, :, used.get(p, 0):] = 0x7F
        if p not in used:
            c.scales[0, p] = math.nan
    c.table[0, 2:] = -5
    c.table[1, 1:] = 1 << 30
    assert torch.equal(run_attention(c, q, pos, counts), got)


def test_bad_rows_and_pages_are_reported_and_skipped():
    c = Paged(8, 2, 64, 16, 3, 4)
    c.fill(1)
    q, k = rows(3, 8, 64, torch.bfloat16, 2), rows(3, 2, 64, torch.bfloat16, 3)
    good = run_attention(c, q, [20, 30, 40], [1, 1, 1])
    for pos in ([20, 64, 40], [20, -1, 40], [20, 2 ** 31 - 1, 40]):
        out = torch.zeros_like(good)
        futr.futr_paged_attention(c.cache, 0, 3, ints(pos), None, c.table, q, out, c.ws)
        assert futr.futr_paged_check(c.cache, c.ws) == futr.FUTR_ERR_OUT_OF_RANGE
        assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2]) and bool((out[1] == 0).all())
        before = c.codes.clone().view(torch.uint8)
        futr.futr_paged_append(c.cache, 0, 3, ints(pos), None, c.table, k, k)
        assert futr.futr_paged_check(c.cache) == futr.FUTR_ERR_OUT_OF_RANGE
        changed = (c.codes.view(torch.uint8) != before).flatten(2).any(-1)[0].nonzero().flatten().tolist()
        assert sorted(changed) == sorted([int(c.table[0, 1]), int(c.table[2, 2])])
        c.fill(1)
    # rows that are not in order, and rows past the end
    for start in ([0, 2, 1, 3], [0, 1, 2, 4], [-1, 0, 1, 3]):
        out = torch.zeros_like(good)
        futr.futr_paged_attention(c.cache, 0, 3, ints([20, 30, 40]), ints(start), c.table, q, out, c.ws)
        assert futr.futr_paged_check(c.cache, c.ws) == futr.FUTR_ERR_OUT_OF_RANGE
        futr.futr_paged_append(c.cache, 0, 3, ints([20, 30, 40]), ints(start), c.table, k, k)
        assert futr.futr_paged_check(c.cache) == futr.FUTR_ERR_OUT_OF_RANGE
    # page ids outside the pool: not visible, not written
    c.fill(1)
    tab = c.table.clone()
    tab[1, 0], tab[1, 1] = -1, c.n_pages
    out = torch.full_like(good, 7.0)
    futr.futr_paged_attention(c.cache, 0, 3, ints([20, 30, 40]), None, tab, q, out, c.ws)
    assert futr.futr_paged_check(c.cache, c.ws) == futr.FUTR_ERR_OUT_OF_RANGE
    assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2]) and bool((out[1] == 0).all())
    before = c.codes.clone().view(torch.uint8)
    futr.futr_paged_append(c.cache, 0, 3, ints([20, 30, 40]), None, tab, k, k)
    assert futr.futr_paged_check(c.cache) == futr.FUTR_ERR_OUT_OF_RANGE
    assert int((c.codes.view(torch.uint8) != before).flatten(2).any(-1).sum()) == 2


def test_append_then_attention_in_a_graph_and_on_another_stream():
    """One captured append + attention follows tables, positions and rows that change between replays."""
    c = Paged(32, 8, 128, 16, 3, 40)
    c.fill(4)
    pos, counts = ints([5, 100, 31]), [1, 1, 1]
    q, k, v = (rows(3, h, 128, torch.bfloat16, 20 + h) for h in (32, 8, 8))
    out = torch.empty_like(q)

    def step():
        futr.futr_paged_append(c.cache, 0, 3, pos, None, c.table, k, v)
        futr.futr_paged_attention(c.cache, 0, 3, pos, None, c.table, q, out, c.ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        lens = [5 + 150 * i, 100 + i, 31 + i]
        pos.copy_(ints(lens))
        for t, s in ((q, 1), (k, 2), (v, 3)):
            t.copy_(rows(3, t.shape[1], 128, torch.bfloat16, 100 * i + s))
        before = c.codes[0].clone(), c.scales[0].clone()
        graph.replay()
        assert futr.futr_paged_check(c.cache, c.ws) == futr.FUTR_OK
        check_append(c, before, k, v, lens, counts)
        check_attention(c, q, out, lens, counts)


def test_shared_pages_and_prompts_in_pieces():
    """Two sequences that read the same first pages; a prompt in one call and in pieces gives
    the same output where the pages' scales are the same (values of one size)."""
    c = Paged(8, 2, 128, 32, 2, 8)
    g = torch.Generator(device="cuda").manual_seed(1)
    n = 200
    k = torch.where(torch.rand((n, 2, 128), generator=g, device="cuda") < 0.5, -1.0, 1.0).to(torch.bfloat16)
    q = rows(n, 8, 128, torch.bfloat16, 6)
    futr.futr_paged_append(c.cache, 0, 1, ints([0]), ints([0, n]), c.table[:1], k, k)
    whole = torch.empty_like(q)
    futr.futr_paged_attention(c.cache, 0, 1, ints([0]), ints([0, n]), c.table[:1], q, whole, c.ws)
    check_attention(c, q, whole, [0], [n])
    table = c.table.clone()
    table[1, :3] = table[0, :3]          # 96 positions shared
    m = n - 96
    futr.futr_paged_append(c.cache, 0, 1, ints([96]), ints([0, m]), table[1:].contiguous(), k[96:], k[96:])
    part = torch.empty_like(q[96:])
    futr.futr_paged_attention(c.cache, 0, 1, ints([96]), ints([0, m]), table[1:].contiguous(), q[96:], part, c.ws)
    c.table = table[1:].contiguous()
    check_attention(c, q[96:], part, [96], [m])
    assert futr.futr_paged_check(c.cache, c.ws) == futr.FUTR_OK


@pytest.mark.parametrize("n", [1, 150], ids=["token", "chunk"])
def test_window_of_everything_is_none(n):
    """Windows up to the largest int32 give what no window gives."""
    c = Paged(4, 2, 128, 64, 1, 6)
    c.fill(8)
    q = rows(n, 4, 128, torch.bfloat16, 12)
    want = run_attention(c, q, [130], [n], 0)
    for window in (130 + n, c.max_pos - 1, c.max_pos, 2 ** 31 - 1):
        assert torch.equal(run_attention(c, q, [130], [n], window), want)


def test_query_that_is_not_finite_stays_its_own():
    """An infinity or NaN in one row's query leaves the other rows as they were."""
    for counts in ([3], [100]):
        c = Paged(4, 2, 128, 64, 1, 6)
        c.fill(9)
        q = rows(counts[0], 4, 128, torch.bfloat16, 13)
        want = run_attention(c, q, [200], counts)
        bad = q.clone()
        bad[1, 2, 5], bad[2, 0, 100] = float("nan"), float("inf")
        got = run_attention(c, bad, [200], counts)
        keep = torch.ones(q.shape[:2], dtype=torch.bool, device="cuda")
        keep[1, 2] = keep[2, 0] = False
        assert torch.equal(got[keep], want[keep])
        assert bool(torch.isnan(got[1, 2]).all())


@pytest.mark.parametrize("counts", [[2, 0, 1], [70, 0, 41]], ids=["few", "many"])
def test_rows_behind_the_last_sequence_stay(counts):
    """Row tensors longer than start says: the rows behind are not read (NaN), nor written."""
    c = Paged(8, 2, 64, 32, 3, 6)
    c.fill(3)
    n, pos = sum(counts), [33, 7, 64]
    q, k, v = (rows(n + 5, h, 64, torch.bfloat16, 40 + h) for h in (8, 2, 2))
    for t in (q, k, v):
        t[n:] = float("nan")
    before = c.codes[0].clone(), c.scales[0].clone()
    futr.futr_paged_append(c.cache, 0, 3, ints(pos), starts(counts), c.table, k, v)
    out = torch.full_like(q, 7.0)
    futr.futr_paged_attention(c.cache, 0, 3, ints(pos), starts(counts), c.table, q, out, c.ws)
    assert futr.futr_paged_check(c.cache, c.ws) == futr.FUTR_OK
    check_append(c, before, k[:n], v[:n], pos, counts)
    check_attention(c, q[:n], out[:n], pos, counts)
    assert bool((out[n:] == 7).all())


@pytest.mark.parametrize("heads,hkv,d,dtype,window", [(32, 8, 128, torch.bfloat16, 0), (8, 2, 64, torch.float16, 150)])
def test_chunks_among_single_tokens(heads, hkv, d, dtype, window):
    """Batches whose sequences differ much: single tokens, drafts, chunks and idle ones in one call."""
    counts = [1, 300, 1, 0, 5, 19, 20, 21, 1, 1, 90, 0] + [1] * 25
    pos = [(i * 97) % 500 for i in range(len(counts))]
    c = Paged(heads, hkv, d, 32, len(counts), 26)
    c.fill(2)
    q = rows(sum(counts), heads, d, dtype, 21)
    got = run_attention(c, q, pos, counts, window)
    check_attention(c, q, got, pos, counts, window)
    assert torch.equal(run_attention(c, q, pos, counts, window), got)


@pytest.mark.parametrize("n", [1, 90], ids=["few", "many"])
def test_a_timeout_stays_with_its_workspace(n):
    """What a call that gave up leaves in its workspace (error and abort words, counters mid-count)
    reaches no other workspace of the cache, and stays until a check with that workspace."""
    c = Paged(8, 2, 128, 32, 2, 100)
    c.fill(6)
    pos, counts = [3000, 2000], [n, n]
    q = rows(2 * n, 8, 128, torch.bfloat16, 31)
    good = run_attention(c, q, pos, counts)
    mine = c.ws
    other = futr.futr_paged_workspace_init(c.cs, futr.alloc_bytes(futr.futr_paged_workspace_size(c.cs)))
    words = mine._mem[mine.err_offset:mine.err_offset + 8].view(torch.int32)
    words[0], words[1] = futr.FUTR_ERR_TIMEOUT, 1
    mine._mem[:4 * mine.ctas].view(torch.int32).fill_(1)
    c.ws = other
    assert torch.equal(run_attention(c, q, pos, counts), good)
    assert futr.futr_paged_check(c.cache) == futr.FUTR_OK
    assert words.tolist() == [futr.FUTR_ERR_TIMEOUT, 1]
    c.ws = mine
    assert futr.futr_paged_check(c.cache, mine) == futr.FUTR_ERR_TIMEOUT
    assert futr.futr_paged_check(c.cache, mine) == futr.FUTR_OK
    assert torch.equal(run_attention(c, q, pos, counts), good)


@pytest.mark.parametrize("gain", [2.0 ** -5, 64.0], ids=["kept", "grown"])
@pytest.mark.parametrize("n", [1, 9])
def test_append_onto_scales_between_powers_of_two(n, gain):
    """A page whose scale a program wrote by its own rule: new codes are e4m3(x / s), x / s in fp32, and
    where s grows old ones e4m3(c * (s_old / s))."""
    c = Paged(4, 2, 128, 16, 3, 2, rope=False)
    c.fill(6, gain=1.0)
    factor = torch.tensor([1.0, 1.5, 1.3, 1.9990234375], device="cuda")
    c.scales[0] *= factor[torch.arange(c.scales[0].numel(), device="cuda") % 4].view_as(c.scales[0])
    old_codes, old_scales = c.codes[0].clone(), c.scales[0].clone()
    pos = [3, 5, 6]
    k, v = (rows(3 * n, 2, 128, torch.bfloat16, s) * gain for s in (4, 5))
    futr.futr_paged_append(c.cache, 0, 3, ints(pos), starts([n] * 3), c.table, k, v)
    assert futr.futr_paged_check(c.cache) == futr.FUTR_OK
    grown = 0
    for b in range(3):
        page = int(c.table[b, 0])
        for h in range(2):
            for w, t in enumerate((k, v)):
                x = t[b * n:(b + 1) * n, h].float()
                s_old = old_scales[page, h, w]
                s = torch.clamp(s_old, min=page_scale(float(x.abs().max())))
                assert torch.equal(c.scales[0, page, h, w], s), (b, h, w)
                want = old_codes[page, h, w].clone()
                if s > s_old:
                    grown += 1
                    want = (want.float() * (s_old / s)).to(torch.float8_e4m3fn)
                want[pos[b]:pos[b] + n] = (x / s).to(torch.float8_e4m3fn)
                assert torch.equal(c.codes[0, page, h, w].view(torch.uint8), want.view(torch.uint8)), (b, h, w)
    assert grown == (0 if gain < 1 else 12)


@pytest.mark.parametrize("nats", [17.0, 17.5, 18.0])
@pytest.mark.parametrize("n,batch", [(1, 304), (32, 160)], ids=["few", "many"])
def test_faint_keys_behind_one_that_carries_nothing(n, batch, nats):
    """One key takes nearly all of the weight and has the value 0: the output is what 2^11 others carry, of
    2^-24.5, 2^-25.2 or 2^-26 of its weight each, below fp16's smallest number next to 1.  As many sequences
    as there are CTAs, so that one has a sequence to itself."""
    N = 1 << 11
    c = Paged(4, 1, 64, 128, 1, N // 128, rope=False)
    c.codes[0, :, :, 0] = torch.tensor(-1.0, device="cuda").to(torch.float8_e4m3fn)
    c.codes[0, :, :, 1] = torch.tensor(1.0, device="cuda").to(torch.float8_e4m3fn)
    c.scales.fill_(1.0)
    first = int(c.table[0, 0])
    c.codes[0, first, :, 0, 5] = torch.tensor(1.0, device="cuda").to(torch.float8_e4m3fn)
    c.codes[0, first, :, 1, 5] = torch.tensor(0.0, device="cuda").to(torch.float8_e4m3fn)
    c.table = c.table.expand(batch, -1).contiguous()     # all read the same pages
    q = torch.full((n * batch, 4, 64), nats / 16, device="cuda").to(torch.bfloat16)    # q.k / 8 = +- nats / 2
    assert float(q[0, 0, 0]) * 16 == nats
    got = run_attention(c, q, [N - n] * batch, [n] * batch).to(F64)
    others = torch.arange(N - n, N, dtype=F64, device="cuda").repeat(batch)[:, None, None] * math.exp(-nats)
    want = (others / (1 + others)).expand_as(got)
    # the query, the keys and the values are exact: the output's half step, a weight's in fp16 (2^-25 at the
    # most where the largest is 2^11, 2^-10 of these), and fp32 sums of 2^11 terms, 2^-24 each
    assert float((got / want - 1).abs().max()) <= 2.0 ** -8 + 2.0 ** -10 + 2.0 ** -12


@pytest.mark.parametrize("power", [118, -118])
@pytest.mark.parametrize("n,rope", [(1, False), (1, True), (40, False), (40, True)])
def test_queries_of_any_size(n, rope, power):
    """Queries near either end of bf16's range, with a scale that brings the scores back.  Without a
    rotation (whose small products may be subnormal) a power of two changes no bit."""
    c = Paged(8, 2, 128, 32, 1, 8, rope=rope)
    c.fill(3)
    g = torch.Generator(device="cuda").manual_seed(2)
    q = (1 + torch.rand((n, 8, 128), generator=g, device="cuda")).to(torch.bfloat16)
    q = torch.where(torch.rand(q.shape, generator=g, device="cuda") < 0.5, -q, q)
    scale = 2.0 ** -5
    want = run_attention(c, q, [100], [n], scale=scale)
    check_attention(c, q, want, [100], [n], scale=scale)
    q, scale = q * 2.0 ** power, scale * 2.0 ** -power
    got = run_attention(c, q, [100], [n], scale=scale)
    check_attention(c, q, got, [100], [n], scale=scale)
    assert rope or torch.equal(got, want)


@pytest.mark.parametrize("heads,kv_heads,d,counts", [
    (8, 2, 64, [1] * 40), (8, 2, 128, [1] * 40), (8, 2, 64, [100, 70]), (8, 2, 128, [100, 70]), (8, 8, 128, [300]),
], ids=["tokens64", "tokens128", "chunks64", "chunks128", "prompt128"])
def test_fp16_rows_keep_their_bits(heads, kv_heads, d, counts):
    """fp16 rows whatever the kernel: the output's rounding and the weights'.  Over values spread evenly
    in their logarithm a rounding to 11 bits is 2^-11 / sqrt(3) / 1.47 = 1.92e-4 of the norm; both
    together sqrt(2) times that, 2.7e-4.  A query of 11 bits would add 2^-12 of each score."""
    pos = [700 + 13 * i for i in range(len(counts))]
    c = Paged(heads, kv_heads, d, 32, len(counts), 60)
    c.fill(5)
    q = rows(sum(counts), heads, d, torch.float16, 17)
    got = run_attention(c, q, pos, counts).to(F64)
    want, _ = c.attention(q, pos, counts)
    e = float((got - want).norm() / want.norm())
    assert e <= 3e-4


@pytest.mark.parametrize("n", [1, 90], ids=["few", "many"])
def test_a_copy_that_never_comes(monkeypatch, n):
    """The last CTA's waits run out (test hook): the call ends, the cache and the workspace report it,
    another workspace is not affected, and after a check with its own the call is exact again."""
    c = Paged(8, 2, 128, 32, 2, 100)
    c.fill(6)
    pos, counts = [3000, 2000], [n, n]
    q = rows(2 * n, 8, 128, torch.bfloat16, 31)
    good = run_attention(c, q, pos, counts)
    mine = c.ws
    other = futr.futr_paged_workspace_init(c.cs, futr.alloc_bytes(futr.futr_paged_workspace_size(c.cs)))
    for _ in range(2):
        monkeypatch.setenv("FUTR_TEST_WITHHOLD_COPY", "1")
        futr.futr_paged_attention(c.cache, 0, 2, ints(pos), starts(counts), c.table, q, torch.empty_like(q), mine)
        monkeypatch.delenv("FUTR_TEST_WITHHOLD_COPY")
        assert futr.futr_paged_check(c.cache) == futr.FUTR_ERR_TIMEOUT
        c.ws = other
        assert torch.equal(run_attention(c, q, pos, counts), good)
        c.ws = mine
        assert futr.futr_paged_check(c.cache, mine) == futr.FUTR_ERR_TIMEOUT
        assert torch.equal(run_attention(c, q, pos, counts), good)
