"""Choice of beams against 64 bits, and the order of the INT4 cache's slots."""
import math

import numpy as np
import pytest
import torch

from int4_weight_kv_w4a16_gb300 import futr
from int4_weight_kv_w4a16_gb300.inputs import TOY
from tests._gen_ref import beam_best, beam_tolerance, beam_values
from tests._gpu_helpers import ensure_lib
from tests._paged_ref import ints, shape_of
from tests.test_gpu_step import Model

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def workspace(rows, keep):
    return futr.futr_beam_workspace_init(rows, keep, futr.alloc_bytes(futr.futr_beam_workspace_size(rows, keep)))


def select(logits, scores, keep, done=None, end=-1, stay=False, ws=None, status=futr.FUTR_OK):
    batch = scores.shape[0]
    out = [torch.full((batch, keep), 77, dtype=t, device="cuda") for t in (torch.float32, I32, I32, I32)]
    ws = ws or workspace(scores.numel(), keep)
    futr.futr_beam_select(logits, scores, out[0], out[1], out[2], ws, done=done, done_out=out[3], end=end, stay=stay)
    assert futr.futr_beam_check(ws) == status
    return out


def check(logits, scores, keep, done=None, end=-1, got=None, status=futr.FUTR_OK):
    """The chosen are the best but for values closer to each other than the tolerance, in order, each with its value."""
    batch, beams = scores.shape
    V = logits.shape[1]
    score, parent, token, ended = got or select(logits, scores, keep, done, end, status=status)
    values, _ = beam_values(logits, scores, done, end)
    want, at = beam_best(values, keep)
    none = at < 0
    assert torch.equal(parent < 0, none) and torch.equal(score == -math.inf, none)
    assert bool((token[none] == max(end, 0)).all()) and bool((ended[none] == 0).all())
    row = torch.arange(batch, device="cuda")[:, None] * beams
    place = torch.where(none, 0, (parent - row) * V + token).long()
    assert bool(((parent - row)[~none] >= 0).all()) and bool(((parent - row)[~none] < beams).all())
    assert bool((token >= 0).all()) and bool((token < V).all())
    for b in range(batch):
        assert len(set(place[b][~none[b]].tolist())) == int((~none[b]).sum())
    assert torch.equal((ended != 0)[~none], (token == end)[~none])
    tol = beam_tolerance(V)
    mine = values.gather(1, place)
    ok = torch.where(none, True, (mine - want).abs() <= 2 * tol)
    assert bool(ok.all())
    err = torch.where(none, 0.0, (score.double() - mine).abs() - mine.abs() * 2.0 ** -24)
    assert float(err.max()) <= tol
    # but where another beam's value is that near (within a beam logits are compared exactly), the very same
    near, place_of = beam_best(values, keep + 8)
    other = (place_of // V)[:, None, :keep + 8] != (at // V)[..., None]
    close = (near[:, None] - want[..., None]).abs() <= 4 * tol
    clear = ~(other & close & (place_of[:, None] >= 0)).any(-1) & ~none
    assert torch.equal(place[clear], at[clear])
    assert float((clear | none).double().mean()) > 0.95
    return score, parent, token, ended


def logits_of(rows, V, dtype, seed, ld=None, offset=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((rows, V), generator=g, device="cuda") * 3
    x.scatter_add_(1, torch.randint(0, V, (rows, 5), generator=g, device="cuda"),
                   8 * torch.rand((rows, 5), generator=g, device="cuda"))
    flat = torch.full((offset + rows * (ld or V) + 64,), math.nan, dtype=dtype, device="cuda")
    view = flat[offset:offset + rows * (ld or V)].view(rows, ld or V)[:, :V]
    view.copy_(x)
    return view


def scores_of(batch, beams, seed):
    g = torch.Generator(device="cuda").manual_seed(seed + 1000)
    return -20 * torch.rand((batch, beams), generator=g, device="cuda")


CASES = [
    # batch, beams, keep, vocab, type, ld, offset
    (1, 1, 1, 1, torch.float32, None, 0),
    (1, 1, 64, 3, torch.float32, None, 0),
    (1, 4, 4, 128256, torch.float32, None, 0),
    (2, 3, 6, 50257, torch.float32, None, 0),
    (3, 5, 10, 50257, torch.bfloat16, None, 0),
    (1, 32, 64, 32000, torch.float16, None, 0),
    (7, 8, 16, 4097, torch.float32, 4111, 3),
    (2, 2, 4, 151936, torch.bfloat16, 151943, 5),
    (40, 8, 8, 1001, torch.float16, None, 1),
    (300, 4, 4, 257, torch.float32, 260, 0),
    (1, 1, 1, 200000, torch.float32, None, 2),
    (1, 2, 64, 100, torch.bfloat16, None, 0),
    (5, 16, 64, 8192, torch.float32, None, 0),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_select(case):
    batch, beams, keep, V, dtype, ld, offset = CASES[case]
    x, s = logits_of(batch * beams, V, dtype, case, ld, offset), scores_of(batch, beams, case)
    got = check(x, s, keep)
    again = select(x, s, keep)
    assert all(torch.equal(a, b) for a, b in zip(got, again))   # nothing depends on timing


@pytest.mark.parametrize("V", [5, 1000, 40000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_equal_logits_go_by_the_lowest_token_and_beam(V, dtype):
    """All logits equal, and equal beams: the first tokens of the first beam.  -0 is 0."""
    x = torch.zeros((6, V), device="cuda", dtype=dtype)
    x[:, ::2] = -0.0
    s = torch.zeros((2, 3), device="cuda")
    for keep in (1, 4, 12):
        _, parent, token, _ = select(x, s, keep)
        order = [(w, v) for w in range(3) for v in range(V)][:keep]
        for b in range(2):
            assert parent[b].tolist() == [3 * b + w for w, _ in order] and token[b].tolist() == [v for _, v in order]


def test_equal_values_of_beams_on_any_alignment():
    """The same row four times, at four alignments: every value four times, the lowest beam first."""
    V = 30001
    one = logits_of(1, V, torch.float32, 5)
    x = torch.empty((4, V), device="cuda")
    x.copy_(one.expand(4, -1))
    best = torch.sort(one[0], descending=True, stable=True).indices[:8]
    _, parent, token, _ = select(x, torch.full((1, 4), -3.0, device="cuda"), 32)
    assert parent[0].tolist() == [0, 1, 2, 3] * 8
    assert token[0].tolist() == best.repeat_interleave(4).tolist()


@pytest.mark.parametrize("order", ["rising", "falling", "steps"])
def test_rows_in_order(order):
    """Rows that keep bringing larger logits fill the lists again and again."""
    V = 70000
    up = torch.arange(V, device="cuda", dtype=torch.float32) * 2.0 ** -12
    x = {"rising": up, "falling": up.flip(0), "steps": (up * 4).floor() / 4}[order]
    x = torch.stack([x, x - 1, x * 0.5])
    for keep in (1, 7, 64):
        check_order = select(x, torch.tensor([[0.0, 0.25, 0.5]], device="cuda"), keep)
        values, _ = beam_values(x, torch.tensor([[0.0, 0.25, 0.5]], device="cuda"))
        want, at = beam_best(values, keep)
        got = check_order[1].long() * V + check_order[2]
        # beams' values differ by their log-sums: equal within the tolerance, tokens of a beam in order
        assert float((values.gather(1, got) - want).abs().max()) <= 2 * beam_tolerance(V)
        for w in range(3):
            mine = check_order[2][0][check_order[1][0] == w].tolist()
            first = torch.sort(x[w], descending=True, stable=True).indices[:len(mine)].tolist()
            assert mine == first


def test_ended_and_dead_beams():
    """Ended beams offer one token at their score; beams at -inf offer nothing; neither is read."""
    V, end = 5000, 17
    x = logits_of(12, V, torch.float32, 3)
    s = scores_of(3, 4, 3)
    done = torch.zeros((3, 4), dtype=I32, device="cuda")
    done[0, 1], done[1, :], s[0, 2], s[2, 0] = 1, 5, -math.inf, -math.inf
    x[1], x[2], x[4:9] = math.nan, math.nan, math.inf      # rows that are not read
    ref = torch.where(torch.isfinite(x), x, 0.0)
    check(ref, s, 8, done, end, got=select(x, s, 8, done, end))
    score, parent, token, ended = select(x, s, 8, done, end)
    assert parent[1, 4:].tolist() == [-1] * 4 and token[1].tolist() == [end] * 8
    assert sorted(score[1, :4].tolist()) == sorted(s[1].tolist())
    assert ended[1].tolist() == [1] * 4 + [0] * 4
    # the first step of a search: one beam alive
    s = torch.full((3, 4), -math.inf, device="cuda")
    s[:, 0] = 0
    x = logits_of(12, V, torch.float32, 4)
    _, parent, _, _ = check(x, s, 4)
    assert parent.tolist() == [[4 * b] * 4 for b in range(3)]
    # nothing alive
    score, parent, token, _ = select(x, torch.full((3, 4), -math.inf, device="cuda"), 4)
    assert bool((score == -math.inf).all()) and bool((parent == -1).all()) and bool((token == 0).all())


def test_masked_logits():
    """Tokens at -inf are no candidates; a row of nothing else offers nothing; the types' lowest values count."""
    V = 9000
    x = logits_of(6, V, torch.float32, 8)
    x[0, 5:] = -math.inf
    x[1] = -math.inf
    x[2, 100:] = -3.4028234663852886e38
    x[3:, ::3] = -math.inf
    check(x, scores_of(1, 6, 1), 40)
    only = torch.full((2, V), -math.inf, device="cuda")
    only[0, 8999], only[1, 3] = 2.0, -7.0
    score, parent, token, _ = select(only, torch.tensor([[-1.0, -2.0]], device="cuda"), 4)
    assert score[0].tolist() == [-1.0, -2.0, -math.inf, -math.inf] and token[0, :2].tolist() == [8999, 3]
    assert parent[0].tolist() == [0, 1, -1, -1]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_rows_of_masks_alone(dtype):
    """Rows in which every token has the mask's large value: each has -log(their number).  Beside it, larger ones of
    whole steps of the type take all of the weight, in ranges where fp64 has the differences."""
    low = torch.finfo(dtype).min
    for mask in (low, -1e4, -1e9 if dtype != torch.float16 else -3e4, -2.0 ** 15,
                 -2.0 ** 20 if dtype != torch.float16 else -9.0, -1.1e6 if dtype != torch.float16 else -5e4, -low):
        for V in (10, 5000, 40000):
            x = torch.full((2, V), mask, device="cuda").to(dtype)
            x[1, V // 2:] = -math.inf
            score, parent, token, _ = select(x, torch.tensor([[-1.0, -3.0]], device="cuda"), 12)
            n = min(V, 12)
            assert parent[0, :min(n, 5)].tolist() == [0] * min(n, 5)
            for p, t, v in zip(parent[0].tolist(), token[0].tolist(), score[0].tolist()):
                if p >= 0:
                    want = -1.0 - math.log(V) if p == 0 else -3.0 - math.log(V // 2)
                    assert abs(v - want) <= beam_tolerance(V) + 2.0 ** -23 * abs(want)
    if dtype == torch.float32:
        x = torch.full((1, 20000), -1e9, device="cuda")
        x[0, 77] += 64                        # fp32's step there
        score, _, token, _ = select(x, torch.zeros((1, 1), device="cuda"), 2)
        assert token[0].tolist() == [77, 0] and float(score[0, 1]) == -64.0
        assert abs(float(score[0, 0])) <= 2 * 19999 * math.exp(-64)          # -log(1 + 19999 e^-64)
        x = torch.linspace(-2.0 ** 20 - 4, -2.0 ** 20 + 4, 30000, device="cuda")[None].repeat(3, 1)    # either side of a branch
        x[1] -= 8
        x[2] += 8
        check(x, scores_of(1, 3, 5), 20)


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("at", [0, 4095, 4999])
def test_rows_that_are_not_finite_are_reported(value, at):
    V = 5000
    x, s = logits_of(8, V, torch.float32, 11), scores_of(2, 4, 11)
    x[1, at] = value
    got = select(x, s, 8, status=futr.FUTR_ERR_NOT_FINITE)
    assert not bool((got[1] == 1).any())
    y, s2 = x.clone(), s.clone()
    y[1] = 0
    s2[0, 1] = -math.inf
    check(y, s2, 8, got=got)
    # a row of -inf with one NaN
    y[5] = -math.inf
    y[5, at] = math.nan
    got = select(y, s2, 8, status=futr.FUTR_ERR_NOT_FINITE)
    assert not bool((got[1] == 5).any())
    # a score
    s3 = s.clone()
    s3[1, 2] = value
    got = select(logits_of(8, V, torch.float32, 12), s3, 8, status=futr.FUTR_ERR_NOT_FINITE)
    assert not bool((got[1] == 6).any()) and bool((got[1] >= 0).all())


@pytest.mark.parametrize("beams", [1, 2, 5, 32])
def test_stay_keeps_the_best_child_in_its_place(beams):
    V = 700
    x, s = logits_of(9 * beams, V, torch.float32, beams), scores_of(9, beams, beams) * 0.2
    s[0, 1:] = -math.inf
    s[1] = -math.inf
    by_rank = [t.cpu() for t in select(x, s, beams, end=2)]
    stay = [t.cpu() for t in select(x, s, beams, end=2, stay=True)]
    for b in range(9):
        rows = list(zip(*(t[b].tolist() for t in by_rank)))
        places = [None] * beams
        late = []
        for r in rows:
            w = r[1] - b * beams
            if r[1] >= 0 and places[w] is None:
                places[w] = r
            else:
                late.append(r)
        for i in range(beams):
            if places[i] is None:
                places[i] = late.pop(0)
        assert places == list(zip(*(t[b].tolist() for t in stay)))


def test_outputs_over_inputs_in_a_graph_and_on_another_stream():
    """A captured step over its own scores, replayed with other logits, next to another workspace's."""
    V, batch, beams, end = 20000, 3, 4, 9
    x, s = logits_of(12, V, torch.float32, 1), scores_of(batch, beams, 1)
    done = torch.zeros((batch, beams), dtype=I32, device="cuda")
    parent, token = (torch.empty((batch, beams), dtype=I32, device="cuda") for _ in range(2))
    ws = workspace(12, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step():
        futr.futr_beam_select(x, s, s, parent, token, ws, done=done, done_out=done, end=end)

    keep_s, keep_d = s.clone(), done.clone()
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    s.copy_(keep_s)
    done.copy_(keep_d)
    for i in range(5):
        x.copy_(logits_of(12, V, torch.float32, 50 + i))
        x[2 * i, end] = 40.0       # a beam ends
        was = s.clone(), done.clone()
        graph.replay()
        assert futr.futr_beam_check(ws) == futr.FUTR_OK
        check(x, was[0], beams, was[1], end, got=(s.clone(), parent, token, done.clone()))
    assert int(done.sum()) > 0


def test_workspace_of_more_rows_and_two_at_once():
    """A workspace serves smaller calls; two streams with a workspace each."""
    ws = [workspace(600, 64) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    data = [(logits_of(8, 60000, torch.float32, i), scores_of(2, 4, i)) for i in range(2)]
    torch.cuda.synchronize()
    outs = [[torch.empty((2, 8), dtype=t, device="cuda") for t in (torch.float32, I32, I32)] for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            futr.futr_beam_select(*data[i], *outs[i], ws[i], stream=streams[i])
    for i in range(2):
        assert futr.futr_beam_check(ws[i], streams[i]) == futr.FUTR_OK
        want = select(*data[i], 8)
        assert all(torch.equal(a, b) for a, b in zip(outs[i], want))


def test_candidates_of_nearly_one_value():
    """Hundreds of candidates that agree in the first 24 bits of their values, and more than the pick's list holds:
    the order of the rest, then of the places."""
    V = 40000
    x = torch.full((8, V), -30.0, device="cuda")
    x[:, 7:207:2] = 0.0                       # a hundred tokens of each beam, equal
    s = torch.full((1, 8), -16384.0, device="cuda")
    s[0, 5] = -16384.0 + 2.0 ** -9
    for keep in (64, 16, 1):
        _, parent, token, _ = select(x, s, keep)
        assert parent[0].tolist() == [5] * keep and token[0].tolist() == [7 + 2 * i for i in range(keep)]
    s[0, 5] = -16384.0
    x[3, 8000] = 2.0 ** -9                    # 2^-9 - log(100 + e^(2^-9)) < -log 100: not among the best
    _, parent, token, _ = select(x, s, 64)
    assert parent[0].tolist() == [0] * 64 and token[0].tolist() == [7 + 2 * i for i in range(64)]


def test_logits_beyond_32_bits():
    """20000 rows, 2.6e9 logits: the last prompts by themselves give the same."""
    batch, beams, V = 2500, 8, 128256
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty((batch * beams, V), dtype=torch.bfloat16, device="cuda")
    for i in range(0, batch * beams, 2000):
        x[i:i + 2000] = torch.randn((2000, V), generator=g, device="cuda").to(torch.bfloat16) * 3
    s = scores_of(batch, beams, 2)
    score, parent, token, _ = select(x, s, beams)
    for b in (0, 1200, 2096, 2499):
        one = select(x[b * beams:(b + 1) * beams].clone(), s[b:b + 1].clone(), beams)
        # (other parts: the sums differ by their roundings)
        assert float((one[0] - score[b]).abs().max()) <= 2 * beam_tolerance(V) + 30 * 2.0 ** -23
        assert torch.equal(one[1] + b * beams, parent[b:b + 1]) and torch.equal(one[2], token[b:b + 1])
    check(x[-4 * beams:], s[-4:], beams, got=[score[-4:], parent[-4:] - (batch - 4) * beams, token[-4:],
                                              torch.zeros_like(token[-4:])])


# ----------------------------------------------------------------- reorder --

class Slots:
    """An INT4 cache of random bytes."""

    def __init__(self, layers, slots, hkv, d, cap, seed):
        s = shape_of(2 * hkv, hkv, d)
        self.cs = futr.make_shape(s)
        self.kv = futr.futr_kv_init(self.cs, layers, slots, cap, futr.alloc_bytes(futr.futr_kv_size(self.cs, layers, slots,
                                                                                                  cap)))
        self.cap, self.d = self.kv.capacity, d
        n = layers * slots * hkv * self.kv.stream_bytes
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.kv._mem[:n].copy_(torch.randint(0, 256, (n,), generator=g, device="cuda", dtype=torch.uint8))
        self.streams = self.kv._mem[:n].view(layers, slots, hkv, -1)

    def moved(self, parent, pos):
        """The streams after the call: tiles of 16 positions, keys, values, their scales."""
        x = self.streams.clone()
        c, d = self.cap, self.d
        for i, p in enumerate(parent):
            if p >= 0:
                t = -(-pos[p] // 16)
                for at, size in ((0, 8 * d), (c * d // 2, 8 * d), (c * d, 32), (c * d + 2 * c, 32)):
                    x[:, i, :, at:at + t * size] = self.streams[:, p, :, at:at + t * size]
        return x


REORDER = [
    # layers, slots, kv-heads, d, capacity, parent, pos
    (1, 1, 1, 64, 16, [0], [16]),
    (2, 4, 2, 128, 100, [1, 2, 3, 0], [100, 1, 33, 64]),
    (3, 5, 8, 64, 333, [0, 0, -1, 4, 3], [333, 0, 17, 16, 200]),
    (2, 32, 1, 128, 50, list(range(31, -1, -1)), list(range(1, 33))),
    (1, 32, 4, 128, 2048, [5] * 32, [2048] * 32),
    (2, 40, 2, 64, 70, [2, 0, 1, 3], [70, 20, 3, 8]),
    (1, 3, 2, 128, 4000, [2, 1, -1], [0, 4000, 3999]),
]


@pytest.mark.parametrize("case", range(len(REORDER)))
def test_reorder(case):
    layers, slots, hkv, d, cap, parent, pos = REORDER[case]
    s = Slots(layers, slots, hkv, d, cap, case)
    for _ in range(3):
        want = s.moved(parent, pos)
        p = ints(pos)
        futr.futr_kv_reorder(s.kv, ints(parent), p)
        assert futr.futr_check(kv=s.kv) == futr.FUTR_OK
        assert torch.equal(s.streams, want)
        pos = [pos[q] if q >= 0 else 0 for q in parent]
        assert p.tolist() == pos


def test_reorder_beyond_32_bits():
    """A cache of 8.9 GB: slots of the first and the last layer."""
    s = Slots(32, 32, 8, 128, 8192, 3)
    parent, pos = [(i * 7 + 3) % 32 for i in range(32)], [8192 - i for i in range(32)]
    first, last = s.streams[0].clone(), s.streams[-1].clone()
    futr.futr_kv_reorder(s.kv, ints(parent), ints(pos))
    assert futr.futr_check(kv=s.kv) == futr.FUTR_OK
    got = s.streams[0].clone(), s.streams[-1].clone()
    for was, now in zip((first, last), got):
        s.streams = was[None]
        assert torch.equal(s.moved(parent, pos)[0], now)


def test_reorder_moves_what_kv_read_gives():
    """The codes and scales of the moved slots, as the cache gives them."""
    s = Slots(2, 6, 2, 128, 200, 1)
    pos, parent = [37, 150, 200, 3, 90, 16], [2, 2, 5, 1, 4, 0]

    def read(slot, n):
        out = [torch.empty((2, n, 128), dtype=torch.int8, device="cuda") if i % 2 == 0 else
               torch.empty((2, n), dtype=torch.int16, device="cuda") for i in range(4)]
        futr.futr_kv_read(s.kv, 1, slot, n, *out)
        return out

    was = [read(i, pos[i]) for i in range(6)]
    p = ints(pos)
    futr.futr_kv_reorder(s.kv, ints(parent), p)
    for i, q in enumerate(parent):
        assert all(torch.equal(a, b) for a, b in zip(read(i, pos[q]), was[q]))


@pytest.mark.parametrize("parent,pos", [([0, 4, 1, 2], [5, 5, 5, 5]), ([0, -2, 1, 2], [5, 5, 5, 5]),
                                        ([1, 0, 3, 2], [5, 5, -1, 5]), ([1, 0, 3, 2], [5, 113, 5, 5]),
                                        ([1, 0, 2 ** 31 - 1, 2], [5, 5, 5, 2 ** 31 - 1])])
def test_reorder_reports_slots_out_of_range(parent, pos):
    s = Slots(1, 4, 2, 64, 112, 1)
    was, p = s.streams.clone(), ints(pos)
    futr.futr_kv_reorder(s.kv, ints(parent), p)
    assert futr.futr_check(kv=s.kv) == futr.FUTR_ERR_OUT_OF_RANGE
    assert torch.equal(s.streams, was) and p.tolist() == pos
    futr.futr_kv_reorder(s.kv, ints([1, 0, 3, 2]), ints([5, 5, 5, 5]))
    assert futr.futr_check(kv=s.kv) == futr.FUTR_OK


def test_reorder_in_a_graph_and_on_another_stream():
    s = Slots(2, 6, 2, 128, 300, 9)
    parent, pos = ints([0] * 6), ints([0] * 6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        futr.futr_kv_reorder(s.kv, parent, pos)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        futr.futr_kv_reorder(s.kv, parent, pos)
    r = np.random.default_rng(4)
    for _ in range(6):
        par, at = r.integers(-1, 6, 6).tolist(), r.integers(0, 301, 6).tolist()
        parent.copy_(ints(par))
        pos.copy_(ints(at))
        want = s.moved(par, at)
        graph.replay()
        assert futr.futr_check(kv=s.kv) == futr.FUTR_OK
        assert torch.equal(s.streams, want) and pos.tolist() == [at[q] if q >= 0 else 0 for q in par]


@pytest.mark.parametrize("stay", [False, True])
def test_a_search_with_the_decode_step(stay):
    """Beams over the INT4 cache: the complete step, the choice and the slots' new order, again and again; a beam's
    logits are those of its tokens decoded one after another by themselves."""
    W, groups, V = 3, 2, 512
    n = W * groups
    m, alone = (Model(TOY, 2, V, max_batch=n, capacity=40, seed=5, host_weights=False) for _ in range(2))
    m.lm_head.mul_(8)
    alone.lm_head.mul_(8)
    ws = workspace(n, W)
    token = torch.arange(n, dtype=I32, device="cuda").view(groups, W)
    scores = torch.full((groups, W), -math.inf, device="cuda")
    scores[:, 0] = 0
    parent, pos = torch.empty((groups, W), dtype=I32, device="cuda"), ints([0] * n)
    fed = [[t] for t in range(n)]
    moved = 0
    for i in range(30):
        logits = m.step(token.view(-1).cpu().numpy(), [i] * n)
        if i in (0, 9, 29):
            for j in range(i + 1):
                want = alone.step([f[j] for f in fed], [j] * n)
            assert torch.equal(logits, want)
        before = scores.clone()
        futr.futr_beam_select(logits, scores, scores, parent, token, ws, stay=stay)
        check(logits, before, W, got=ranked(scores, parent, token))
        pos.fill_(i + 1)
        futr.futr_kv_reorder(m.kv, parent.view(-1), pos)
        assert pos.tolist() == [i + 1] * n
        p = parent.view(-1).tolist()
        moved += sum(a != b for a, b in enumerate(p))
        fed = [fed[a] + [t] for a, t in zip(p, token.view(-1).tolist())]
    assert futr.futr_check(m.ws, m.kv) == futr.FUTR_OK and futr.futr_beam_check(ws) == futr.FUTR_OK
    assert moved > 30


def ranked(score, parent, token):
    """Outputs best first, as check() takes them (no beam ends)."""
    order = torch.sort(score, dim=1, descending=True, stable=True).indices
    return [t.gather(1, order) for t in (score, parent, token)] + [torch.zeros_like(token)]


# ------------------------------------------------- values of rows, to the bit --

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("V", [2, 1000, 8192, 50257, 128256, 1000003])
def test_the_log_sum_of_equal_logits(V, dtype):
    """n equal logits (the others -inf) have the log-sum M + log n.  Where M is 0 or a power of two, each exponent is
    0, and n ones add up as they are: only the logarithm's own error (2^-26), sums in two parts (2^-46 of 32768) and the
    value's rounding are left.  The score log n leaves a value near 0, which a rounding hides least."""
    for M in (0.0, 1.0, -0.5, -4.0, 64.0, -32768.0):
        for rows in (1, 40):
            for n in {V, V // 2 + 1}:
                x = torch.full((rows, V), -math.inf, dtype=dtype, device="cuda")
                x[:, torch.randperm(V, device="cuda")[:n]] = M
                s = torch.full((rows, 1), math.log(n), device="cuda")
                score, _, _, _ = select(x, s, 1)
                want = float(s[0, 0]) - math.log(n)
                assert float((score.double() - want).abs().max()) <= 2.0 ** -25 + 2.0 ** -24 * abs(want), (M, rows, n)


def log_sum_bound(x):
    """What a row's log-sum may be off by at most, in units of u = 2^-24: the exponentials and the first factor of a tile
    4 each (ex2.approx: 2^-22), 16 + 1 + 1 additions of a tile, 1 and 1/4 for the logarithm, two rescalings of 5 when a
    part's and a row's threads meet, and for every tile (of 8192 logits) that a part has, one addition and a rescaling of 5;
    the exponents' own roundings, and the constant's, 2.25 of the mean of max - x under the softmax."""
    m = x.double().amax(-1, keepdim=True)
    p = torch.softmax(x.double(), -1)
    mean = torch.where(p > 0, p * (m - x.double()), 0.0).sum(-1)
    return 2.0 ** -24 * (39 + 6 * -(-x.shape[-1] // 8192) + 2.25 * mean)


@pytest.mark.parametrize("kind", ["normal", "wide", "far", "rising", "falling", "large", "two", "halves"])
@pytest.mark.parametrize("V,rows", [(700, 5), (32000, 3), (128256, 1), (128256, 64), (128256, 700), (400000, 600)])
def test_values_of_rows(kind, V, rows):
    """The best token's value with a score that leaves it near 0, rows of one part and of many."""
    g = torch.Generator(device="cuda").manual_seed(V + rows)
    z = torch.randn((rows, V), generator=g, device="cuda")
    up = torch.linspace(0, 9, V, device="cuda")
    x = {"normal": z, "wide": 8 * z, "far": 2 * z - 3000, "rising": z * 0.1 + up, "falling": z * 0.1 + up.flip(0),
         "large": z * 300 + 2.0 ** 20, "two": torch.where(z > 2, 1.5, -7.7), "halves": 7.3 - (z > 0).float() * 0.1}[kind]
    m = x.double().amax(-1)
    lse = m + torch.log(torch.exp(x.double() - m[:, None]).sum(-1))
    s = (lse - m).float()[:, None].contiguous()
    score, _, token, _ = select(x, s, 1)
    want = x.double().gather(1, token.long())[:, 0] - lse + s[:, 0].double()
    assert torch.equal(x.double().gather(1, token.long())[:, 0], m)
    assert bool(((score[:, 0].double() - want).abs() <= log_sum_bound(x) + 2.0 ** -24 * want.abs()).all())


def test_no_value_is_above_its_score():
    """A token's probability is 1 at most, however near: one logit far above the others, at magnitudes whose exponents
    are rounded, in one part and in many."""
    for V, rows in ((50, 300), (20000, 300), (128256, 40), (128256, 700)):
        g = torch.Generator(device="cuda").manual_seed(V + rows)
        x = torch.randn((rows, V), generator=g, device="cuda")
        at = torch.randint(0, V, (rows, 1), generator=g, device="cuda")
        top = 200.0 + 900.0 * torch.rand((rows, 1), generator=g, device="cuda")
        x.scatter_(1, at, top)
        s = torch.where(torch.arange(rows, device="cuda") % 2 == 0, 0.0, -0.37)[:, None].contiguous()
        score, _, token, _ = select(x, s, 1)
        assert torch.equal(token, at.to(I32))
        assert torch.equal(score, s)       # the others weigh less than e^-150
        s = torch.zeros((rows, 1), device="cuda")
        x = torch.where(x < 100, x + top - 18.0 - math.log(V), x)     # and some 2^-26 of it
        score, _, token, _ = select(x, s, 1)
        assert bool((score <= 0).all())


@pytest.mark.parametrize("base", [-1e9, -3e7, 4096.0, -1e30, 1e30, 0.0])
@pytest.mark.parametrize("V", [500, 60000])
def test_a_beams_tokens_are_in_the_order_of_their_logits(base, V):
    """Scores that leave nothing of small differences between a beam's values: its tokens go by their logits all the
    same, equal logits by the lowest token, and none is left out for a lower token."""
    g = torch.Generator(device="cuda").manual_seed(V)
    near = 1.0 + torch.randint(0, 40, (6, V), generator=g, device="cuda") * 2.0 ** -23       # steps of fp32, ties among them
    spread = torch.randn((6, V), generator=g, device="cuda") * 20                            # about the sums' own steps
    tiny = torch.randint(-30, 30, (6, V), generator=g, device="cuda").float() * 1e-30
    for x in (near, spread, tiny):
        for dtype in (torch.float32, torch.bfloat16):
            y = x.to(dtype)
            order = torch.sort(y, dim=1, descending=True, stable=True).indices
            for step in (0.0, abs(base) * 2.0 ** -20):
                s = (base - step * torch.tensor([[0.0, 1, 2], [2, 0, 1]], device="cuda")).contiguous()
                for keep in (1, 3, 7, 64):
                    _, parent, token, _ = select(y, s, keep)
                    for w in range(6):
                        mine = token[w // 3][parent[w // 3] == w]
                        assert torch.equal(mine, order[w, :mine.numel()].to(I32)), (base, keep, w)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("V", [3, 128256])
def test_the_log_sum_of_equal_large_logits(V, dtype):
    """As above, where M is so large that M + log n has little of log n left.  Beyond 2^20 exponents are differences, and
    0 again; fp16's largest stay below it, where M log2 e is rounded unless M is a power of two: the exponentials of what it
    lost, 2^-22 off each, and additions of such numbers are those of log_sum_bound."""
    for M in (torch.finfo(dtype).min, torch.finfo(dtype).max, 3.0 * 2.0 ** (13 if dtype == torch.float16 else 21)):
        x = torch.full((4, V), M, device="cuda").to(dtype)
        s = torch.full((2, 2), math.log(V), device="cuda")
        score, _, _, _ = select(x, s, 3)
        want = float(s[0, 0]) - math.log(V)
        own = 2.0 ** -25 if abs(M) > 2.0 ** 20 else float(log_sum_bound(x).max())
        assert float((score.double() - want).abs().max()) <= own + 2.0 ** -24 * abs(want), M


def some_moves(batch, n, seed):
    """Parents of `batch` slots of which n take another's tokens, some slots are emptied, and the rest stay."""
    r = np.random.default_rng(seed)
    parent = list(range(batch))
    moved = r.permutation(batch)[:n].tolist()
    for i in moved:
        parent[i] = int((i + r.integers(1, batch)) % batch)
    for i in r.permutation(batch)[:batch // 5].tolist():
        if i not in moved:
            parent[i] = -1
    return parent


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("batch,moves", [(b, m) for b in (7, 8, 9, 12, 16, 17, 24, 32) for m in (0, 1, 2, 4, 5, 8, 9, 16, 17, 32)
                                         if m <= b] + [(9, 3), (16, 7), (16, 15), (32, 31)])
def test_reorder_of_every_number_of_moves(batch, moves, d):
    """Every kernel for a batch, each number of slots that move in it: few of many, and all."""
    r = np.random.default_rng(100 * batch + moves)
    s = Slots(2, batch + moves % 3, 3, d, 150, batch + moves)
    pos = r.integers(1, 151, batch).tolist()
    for i in range(2):
        parent = some_moves(batch, moves, 7 * batch + moves + i)
        if i == 1 and moves == batch:
            parent = [(j + 1) % batch for j in range(batch)]        # all change places
        assert sum(p >= 0 and p != j for j, p in enumerate(parent)) == moves
        want, p = s.moved(parent, pos), ints(pos)
        futr.futr_kv_reorder(s.kv, ints(parent), p)
        assert futr.futr_check(kv=s.kv) == futr.FUTR_OK
        assert torch.equal(s.streams, want)
        pos = [pos[q] if q >= 0 else 0 for q in parent]
        assert p.tolist() == pos


def test_the_largest_vocabulary():
    """A row of 2^31 - 1 logits, the best of them at its ends."""
    V = 2 ** 31 - 1
    x = torch.zeros((1, V), dtype=torch.bfloat16, device="cuda")
    best = [V - 1, 0, 7, V - 2, 2 ** 30, V - 9]
    x[0, best[0]], x[0, best[1]], x[0, best[2]] = 3.0, 3.0, 2.0
    x[0, best[3]], x[0, best[4]], x[0, best[5]] = 1.0, 0.5, 0.25
    score, parent, token, ended = select(x, torch.zeros((1, 1), device="cuda"), 8, end=V - 1)
    assert token[0].tolist() == [0, V - 1, 7, V - 2, 2 ** 30, V - 9, 1, 2]
    assert parent[0].tolist() == [0] * 8 and ended[0].tolist() == [0, 1] + [0] * 6
    x[0, best] = 0
    score, _, token, _ = select(x, torch.full((1, 1), math.log(V), device="cuda"), 2)
    # (a thread has 2^17 zeros at most, whose e^0 add up as they are)
    want = float(torch.tensor(math.log(V))) - math.log(V)
    assert token[0].tolist() == [0, 1] and float((score.double() - want).abs().max()) <= 2.0 ** -25 + 2.0 ** -24 * abs(want)
