"""Pages of a paged cache: take, share, give back, move, against Python lists; and a run of them with the model's calls."""
import numpy as np
import pytest
import torch

from int4_weight_kv_w4a16_gb300 import futr
from tests._gen_ref import Pool
from tests._gpu_helpers import ensure_lib
from tests._paged_ref import Paged, ints, shape_of, starts

pytestmark = pytest.mark.gpu
OK = futr.FUTR_OK


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


class Both:
    """A cache with its pool on the GPU, and the same as lists; pages of random bytes that tell them apart."""

    def __init__(self, n_pages, page, rows, width, layers=2, hkv=2, d=64, max_pos=None, max_seqs=None, seed=0):
        s = futr.make_shape(shape_of(2 * hkv, hkv, d))
        max_pos = max_pos or width * page
        size = futr.futr_paged_size(s, layers, n_pages, page, max_pos)
        self.cache = futr.futr_paged_init(s, layers, n_pages, page, max_pos, False, futr.alloc_bytes(size))
        self.codes, self.scales = futr.paged_views(self.cache)
        self.bits = self.codes.view(torch.uint8)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.bits.copy_(torch.randint(0, 256, self.bits.shape, generator=g, device="cuda", dtype=torch.uint8))
        self.scales.copy_(torch.rand(self.scales.shape, generator=g, device="cuda"))
        seqs = max_seqs or rows
        self.pool = futr.futr_pages_init(n_pages, seqs, futr.alloc_bytes(futr.futr_pages_size(n_pages, seqs)))
        self.table = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
        self.ref = Pool(n_pages, page, rows, width, max_pos)
        self.page = page

    def same(self, status=OK):
        assert futr.futr_pages_check(self.pool) == (status, len(self.ref.free()))
        assert self.table.tolist() == self.ref.table
        assert futr.pages_refs(self.pool).tolist() == self.ref.refs()
        n = self.ref.n
        at = self.pool.free_offset
        words = self.pool._mem[at:at + 4 * (-(-n // 32))].cpu().numpy().view(np.uint32)
        free = [p for p in range(n) if words[p // 32] >> (p % 32) & 1]
        assert free == self.ref.free()
        assert futr.futr_paged_check(self.cache) == OK

    def grow(self, pos, new, start=True):
        futr.futr_pages_grow(self.cache, self.pool, ints(pos), starts(new) if start else None, self.table)
        return self.ref.grow(pos, new)

    def free(self, pos, window=0, sinks=0):
        futr.futr_pages_free(self.cache, self.pool, ints(pos), self.table, window=window, sinks=sinks)
        self.ref.give(pos, window, sinks)

    def fork(self, parent, pos):
        """The new positions; the pages' contents are compared here."""
        bits, scales, p = self.bits.clone(), self.scales.clone(), ints(pos)
        futr.futr_pages_fork(self.cache, self.pool, ints(parent), p, self.table)
        done = self.ref.fork(parent, pos)
        if done is None:
            assert p.tolist() == pos
            new = pos
        else:
            copies, new = done
            assert p.tolist() == new
            for s, t, n in copies:
                bits[:, t, :, :, :n] = bits[:, s, :, :, :n]
                scales[:, t] = scales[:, s]
        assert torch.equal(self.bits, bits) and torch.equal(self.scales, scales)
        return None if done is None else new

    def compact(self, lo, hi):
        bits, scales = self.bits.clone(), self.scales.clone()
        futr.futr_pages_compact(self.cache, self.pool, self.table, lo, hi)
        to = self.ref.compact(lo, hi)
        for s, t in (to or {}).items():
            bits[:, t], scales[:, t] = bits[:, s].clone(), scales[:, s].clone()
        assert torch.equal(self.bits, bits) and torch.equal(self.scales, scales)
        return to is not None


@pytest.mark.parametrize("n_pages,max_seqs", [(1, 1), (31, 3), (32, 1024), (33, 5), (70001, 2)])
def test_a_new_pool_is_free(n_pages, max_seqs):
    b = Both(n_pages, 16, 1, 4, layers=1, hkv=1, max_seqs=max_seqs)
    b.same()


def test_grow_takes_the_lowest_pages_in_order():
    b = Both(40, 16, 4, 12)
    assert b.grow([0, 0, 5, 0], [33, 0, 1, 16])
    assert b.ref.table[0][:4] == [0, 1, 2, -1] and b.ref.table[2][0] == 3 and b.ref.table[3][:2] == [4, -1]
    b.same()
    assert b.grow([33, 0, 6, 16], [1, 1, 1, 1], start=False)    # one row each: two meet a new page
    b.same()
    b.free([0, 1, 7, 17])
    b.same()
    assert b.grow([0, 1, 7, 17], [192, 0, 0, 100])
    b.same()


def test_rows_that_do_not_fit_are_skipped():
    for max_pos in (100, None):
        b = Both(40, 16, 5, 8, max_pos=max_pos)
        pos, new = [90, -1, 0, 120, 2 ** 31 - 1], [20, 3, 5, 9, 4]
        futr.futr_pages_grow(b.cache, b.pool, ints(pos), starts(new), b.table)
        b.ref.grow(pos, new)
        b.same(futr.FUTR_ERR_OUT_OF_RANGE)
        # rows that are not in order
        futr.futr_pages_grow(b.cache, b.pool, ints([0] * 5), ints([0, 3, 1, 1, 2, 2]), b.table)
        b.ref.grow([0] * 5, [3, 0, 0, 1, 0])
        b.same(futr.FUTR_ERR_OUT_OF_RANGE)


def test_too_few_pages_change_nothing():
    b = Both(10, 16, 3, 12)
    assert b.grow([0, 0, 0], [100, 30, 0])          # 7 + 2 pages
    b.same()
    assert not b.grow([100, 30, 0], [1, 3, 17])     # one more for the second, two for the third
    b.same(futr.FUTR_ERR_NO_PAGES)
    assert b.fork([0, 0, 0], [100, 30, 0]) is None  # two copies
    b.same(futr.FUTR_ERR_NO_PAGES)
    assert not b.compact(0, 9)
    b.same(futr.FUTR_ERR_NO_PAGES)
    assert b.fork([0, 0, -1], [100, 30, 0]) == [100, 100, 0]   # one copy; row 1's pages are free afterwards
    b.same()


def test_rows_are_not_for_pages_that_others_hold():
    """Back to a position inside a page that a fork shared: refused, until a fork has made a copy."""
    b = Both(40, 16, 3, 8)
    assert b.grow([0, 0, 0], [70, 20, 0])
    pos = b.fork([0, 1, 0], [70, 20, 0])            # rows 0 and 2 share four pages
    b.same()
    b.free([40, 20, 70])                            # row 0 goes back into the third
    b.same()
    assert b.grow([40, 20, 70], [1, 1, 1]) is None
    b.same(futr.FUTR_ERR_SHARED)
    assert b.grow([48, 20, 70], [1, 1, 1])          # behind it, in a page of its own
    b.same()
    b.free([40, 20, 71])
    assert b.grow([64, 20, 70], [0, 13, 10]) is True
    b.same()
    # a fork of every row into itself copies the page, in the order of rows
    b.free([40, 0, 71])
    assert b.fork([0, 1, 2], [40, 0, 71]) == [40, 0, 71]
    b.same()
    assert b.grow([40, 0, 71], [30, 0, 1])
    b.same()
    # of two that share one, both copy, and the page is free; with further children
    b.free([70, 0, 72])
    b.free([35, 0, 36])
    assert b.fork([2, 2, 0], [35, 0, 36]) == [36, 36, 35]
    b.same()


def test_free_by_window_sinks_and_position():
    b = Both(200, 16, 4, 40)
    assert b.grow([0] * 4, [640, 640, 640, 640])
    for pos, window, sinks in (([640, 600, 17, 640], 0, 0), ([640, 600, 0, 639], 100, 0), ([640, 320, 0, 639], 50, 33),
                               ([640, 320, -5, 639], 1, 16), ([320, 64, 0, 1], 2 ** 31 - 1, 2 ** 31 - 1),
                               ([320, 64, 0, 0], 1, 0)):
        b.free(pos, window, sinks)
        b.same()


FORKS = [
    # rows, page, pos, parent
    (4, 16, [20, 20, 20, 20], [0, 0, 2, 2]),
    (4, 16, [32, 32, 32, 32], [3, 3, 3, 1]),        # full pages only
    (4, 16, [5, 40, 0, 63], [1, 0, 1, 3]),
    (5, 32, [1, 31, 33, 100, 0], [3, 2, 1, 0, -1]), # only moves
    (6, 128, [500, 7, 7, 129, 256, 1], [0, 0, 0, 0, 0, 0]),
    (3, 64, [64, 1, 191], [-1, -1, -1]),
    (1, 16, [9], [0]),
    (33, 16, list(range(1, 34)), [i // 2 for i in range(33)]),
]


@pytest.mark.parametrize("case", range(len(FORKS)))
def test_fork(case):
    rows, page, pos, parent = FORKS[case]
    width = max(pos) // page + 3
    b = Both(rows * (width + 4), page, rows, width, seed=case, d=128 if case % 2 else 64)
    assert b.grow([0] * rows, pos)
    for _ in range(3):
        pos = b.fork(parent, pos)
        b.same()


def test_fork_of_pages_taken_ahead_and_of_gaps():
    """Pages behind the written ones stay with the first child; places without a page stay without one."""
    b = Both(60, 16, 3, 12)
    assert b.grow([0, 0, 0], [150, 40, 0])
    b.free([150, 40, 0], window=60)                 # a gap at the front
    b.same()
    pos = b.fork([0, 0, 0], [135, 40, 0])           # page 9 was taken ahead
    assert b.ref.table[0][9] >= 0 and b.ref.table[1][9] == -1 and b.ref.table[1][0] == -1
    b.same()
    b.fork([1, 1, 0], pos)
    b.same()
    # the written page itself is missing
    b = Both(60, 16, 2, 4)
    assert b.fork([0, 0], [20, 0]) == [20, 20]
    b.same()


@pytest.mark.parametrize("parent,pos", [([0, 2], [5, 5]), ([-2, 0], [5, 5]), ([0, 0], [-1, 0]), ([0, 0], [65, 0]),
                                        ([1, 2 ** 31 - 1], [5, 5])])
def test_fork_out_of_range_changes_nothing(parent, pos):
    b = Both(20, 16, 2, 4)
    assert b.grow([0, 0], [40, 10])
    p = ints(pos)
    was = b.bits.clone()
    futr.futr_pages_fork(b.cache, b.pool, ints(parent), p, b.table)
    b.same(futr.FUTR_ERR_OUT_OF_RANGE)
    assert p.tolist() == pos and torch.equal(was, b.bits)


def test_compact_moves_the_end_to_the_front_and_back():
    b = Both(71, 16, 5, 20, layers=3, d=128)
    assert b.grow([0] * 5, [200, 16, 300, 1, 90])
    pos = b.fork([0, 0, 2, 3, 2], [200, 16, 300, 1, 90])
    b.free([0] + pos[1:])
    b.same()
    used = 71 - len(b.ref.free())
    assert b.compact(used, 71)
    assert sorted(b.ref.free()) == list(range(used, 71))
    b.same()
    for lo, hi in ((0, 30), (30, 71), (5, 5), (33, 34), (0, 1), (31, 65)):
        b.same(OK if b.compact(lo, hi) else futr.FUTR_ERR_NO_PAGES)


def test_hold_counts_a_table_made_by_hand():
    b = Both(30, 16, 3, 5)
    hand = [[3, 4, 29, -1, -1], [3, 4, 0, -7, -1], [-1] * 5]
    b.table.copy_(ints(hand))
    futr.futr_pages_hold(b.cache, b.pool, b.table)
    hand[1][3] = -7
    b.ref.table = hand
    b.same()
    b.free([48, 33, 0])
    b.ref.table[1][3] = -7                                      # what names no page stays as it is
    b.same()
    # ids out of range are no pages
    b.table[2, 0], b.table[2, 1] = 30, 2 ** 31 - 1
    futr.futr_pages_hold(b.cache, b.pool, b.table[2:].contiguous())
    assert futr.futr_pages_check(b.pool)[0] == futr.FUTR_ERR_OUT_OF_RANGE
    # pages that the pool has free cannot be given back
    b.table[2, 0], b.table[2, 1] = 7, -1
    futr.futr_pages_free(b.cache, b.pool, ints([48, 33, 0]), b.table)
    b.same(futr.FUTR_ERR_NOT_HELD)
    # nor written
    b.table[2, 0] = 8
    futr.futr_pages_grow(b.cache, b.pool, ints([48, 64, 0]), starts([0, 0, 20]), b.table)
    b.table[2, 0] = -1
    b.same(futr.FUTR_ERR_NOT_HELD)


@pytest.mark.parametrize("seed", range(6))
def test_random_runs(seed):
    """Hundreds of calls in a row give what the lists give."""
    r = np.random.default_rng(seed)
    page, rows = int(r.choice([16, 32, 64])), int(r.integers(1, 40))
    width = int(r.integers(2, 30))
    b = Both(int(r.integers(rows, rows * width)), page, rows, width, layers=1, hkv=1, seed=seed)
    pos = [0] * rows
    for step in range(60):
        op = r.choice(["grow", "grow", "free", "fork", "compact", "drop"])
        status = OK
        if op == "grow":
            new = [int(min(r.integers(0, 3 * page), width * page - p)) for p in pos]
            done = b.grow(pos, new)
            if done:
                pos = [p + n for p, n in zip(pos, new)]
            else:
                status = futr.FUTR_ERR_SHARED if done is None else futr.FUTR_ERR_NO_PAGES
        elif op == "free":
            pos = [max(0, p - int(r.integers(0, page))) if r.random() < 0.3 else p for p in pos]
            b.free(pos, *((int(r.integers(1, 6 * page)), int(r.integers(0, 2 * page))) if seed % 2 else ()))
        elif op == "drop":
            pos = [0 if r.random() < 0.3 else p for p in pos]
            b.free(pos)
        elif op == "fork":
            parent = [int(r.integers(-1, rows)) if r.random() < 0.5 else i for i in range(rows)]
            new = b.fork(parent, pos)
            status = OK if new is not None else futr.FUTR_ERR_NO_PAGES
            pos = pos if new is None else new
        else:
            lo, hi = sorted(r.integers(0, b.ref.n + 1, 2).tolist())
            status = OK if b.compact(lo, hi) else futr.FUTR_ERR_NO_PAGES
        b.same(status)


def test_pages_beyond_32_bits():
    """A cache of 5.4 GB: copies of a fork and moves of its pages in the last layer."""
    b = Both(300, 128, 4, 70, layers=70, hkv=8, d=128)
    pos = [8000, 120, 0, 0]
    assert b.grow([0] * 4, pos)
    pos = b.fork([0, 1, 1, 0], pos)
    b.same()
    assert b.compact(0, 140)
    b.same()


def test_many_sequences_and_pages():
    """The largest table: 1024 sequences, pages over several rounds of the search."""
    b = Both(70000, 16, 1024, 64, layers=1, hkv=1)
    r = np.random.default_rng(1)
    pos = r.integers(0, 1000, 1024).tolist()
    assert b.grow([0] * 1024, pos)
    b.same()
    parent = r.integers(-1, 1024, 1024).tolist()
    pos = b.fork(parent, pos)
    b.same()
    b.free(pos, window=300, sinks=20)
    b.same()
    assert b.compact(20000, 70000) and b.compact(0, 40000)
    b.same()
    new = [int(n) for n in r.integers(0, 40, 1024)]
    fits = lambda new: OK if all(p + n <= 1024 for p, n in zip(pos, new)) else futr.FUTR_ERR_OUT_OF_RANGE
    assert b.grow(pos, new)
    b.same(fits(new))
    pos = [p if i % 3 else 0 for i, p in enumerate(pos)]
    b.free(pos)
    b.same()
    assert b.grow(pos, [33] * 1024)
    b.same(fits([33] * 1024))


def test_a_search_in_a_graph():
    """Beams over a paged cache as one captured step (grow, append, attention, select, fork), replayed: the tables
    against lists, and each step's attention against a cache in which nothing is shared."""
    W, groups, V, layers, page, hkv, d, heads = 4, 2, 300, 2, 16, 2, 64, 4
    rows, width = W * groups, 8
    b = Both(rows * width, page, rows, width, layers=layers, hkv=hkv, d=d)
    cs = futr.make_shape(shape_of(heads, hkv, d))
    cache = futr.futr_paged_init(cs, layers, b.ref.n, page, width * page, True,
                                 futr.alloc_bytes(futr.futr_paged_size(cs, layers, b.ref.n, page, width * page)))
    b.cache, (b.codes, b.scales) = cache, futr.paged_views(cache)
    b.bits = b.codes.view(torch.uint8)
    own = Paged(heads, hkv, d, page, rows, width, layers=layers)      # a copy that shares nothing
    ws = futr.futr_paged_workspace_init(cs, futr.alloc_bytes(futr.futr_paged_workspace_size(cs)))
    bws = futr.futr_beam_workspace_init(rows, W, futr.alloc_bytes(futr.futr_beam_workspace_size(rows, W)))
    g = torch.Generator(device="cuda").manual_seed(3)
    emb = torch.randn((V, heads + 2 * hkv, d), generator=g, device="cuda")
    head = torch.randn((heads * d, V), generator=g, device="cuda") * 0.2
    token = torch.randint(0, V, (groups, W), generator=g, device="cuda", dtype=torch.int32)
    scores = torch.zeros((groups, W), device="cuda")
    parent = torch.empty((groups, W), dtype=torch.int32, device="cuda")
    pos, out = ints([0] * rows), torch.empty((layers, rows, heads, d), dtype=torch.bfloat16, device="cuda")
    logits = torch.empty((rows, V), device="cuda")

    def qkv():
        x = emb[token.reshape(-1).long()].to(torch.bfloat16)
        return x[:, :heads], x[:, heads:heads + hkv], x[:, heads + hkv:]

    def step():
        q, k, v = qkv()
        futr.futr_pages_grow(cache, b.pool, pos, None, b.table)
        for layer in range(layers):
            futr.futr_paged_append(cache, layer, rows, pos, None, b.table, k, v)
            futr.futr_paged_attention(cache, layer, rows, pos, None, b.table, q, out[layer], ws)
        logits.copy_(out.float().mean(0).reshape(rows, -1) @ head)
        pos.add_(1)
        futr.futr_beam_select(logits, scores, scores, parent, token, bws)
        futr.futr_pages_fork(cache, b.pool, parent.view(-1), pos, b.table)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    first = token.clone()
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    # from the start again
    futr.futr_pages_free(cache, b.pool, ints([0] * rows), b.table)
    token.copy_(first)
    scores.zero_()
    pos.zero_()
    for i in range(100):
        q, k, v = (t.clone() for t in qkv())
        for layer in range(layers):
            futr.futr_paged_append(own.cache, layer, rows, ints([i] * rows), None, own.table, k, v)
        want = torch.empty_like(out)
        for layer in range(layers):
            futr.futr_paged_attention(own.cache, layer, rows, ints([i] * rows), None, own.table, q, want[layer], own.ws)
        graph.replay()
        assert torch.equal(out, want), i
        assert b.ref.grow([i] * rows, [1] * rows)
        p = parent.view(-1).tolist()
        assert all(x // W == j // W for j, x in enumerate(p))
        assert b.ref.fork(p, [i + 1] * rows) is not None
        b.same()
        assert pos.tolist() == [i + 1] * rows and futr.futr_beam_check(bws) == OK
        # the copy: whole sequences move
        at = own.table.long()
        own.codes[:, at] = own.codes[:, at[p]].clone()
        own.scales[:, at] = own.scales[:, at[p]].clone()
    assert len(b.ref.free()) > rows * width // 3        # pages are shared


def counts_agree(b):
    """The free bits, their number and the counts say the same; returns the counts."""
    n_free = futr.futr_pages_check(b.pool)[1]
    refs = futr.pages_refs(b.pool).tolist()
    at = b.pool.free_offset
    words = b.pool._mem[at:at + 4 * (-(-b.ref.n // 32))].cpu().numpy().view(np.uint32)
    free = [p for p in range(b.ref.n) if words[p // 32] >> (p % 32) & 1]
    assert free == [p for p, r in enumerate(refs) if r == 0] and n_free == len(free)
    assert min(refs) >= 0
    return refs


@pytest.mark.parametrize("seed", range(8))
def test_tables_that_were_not_counted_in_full(seed):
    """Tables of which only some rows were counted, shared pages among them: places are given back that the pool knows
    nothing of, and others go on.  Whatever comes of the calls, the free bits follow the counts, and a page that is
    taken was free."""
    r = np.random.default_rng(seed)
    page, rows, width = 16, int(r.choice([2, 5, 32])), int(r.integers(3, 12))
    n = rows * width
    b = Both(n, page, rows, width, layers=1, hkv=1, seed=seed)
    for _ in range(12):
        hand = r.integers(-1, max(2, n // int(r.integers(2, 20))), (rows, width)).astype(np.int32)
        b.table.copy_(torch.from_numpy(hand))
        some = [i for i in range(rows) if r.random() < 0.5] or [0]
        futr.futr_pages_hold(b.cache, b.pool, b.table[some].contiguous())
        pos = ints(r.integers(0, width * page + 1, rows).tolist())
        counts_agree(b)
        for _ in range(3):
            parent = ints(r.integers(-1, rows, rows).tolist())
            futr.futr_pages_fork(b.cache, b.pool, parent, pos, b.table)
            counts_agree(b)
        futr.futr_pages_free(b.cache, b.pool, pos, b.table, window=40, sinks=5)
        was, before = counts_agree(b), b.table.clone()
        futr.futr_pages_grow(b.cache, b.pool, pos, starts(r.integers(0, 20, rows).tolist()), b.table)
        now = counts_agree(b)
        new = b.table[b.table != before].tolist()
        assert all(was[p] == 0 and now[p] == 1 for p in new) and len(set(new)) == len(new)
        assert sum(now) == sum(was) + len(new)
        futr.futr_pages_free(b.cache, b.pool, ints([0] * rows), b.table)
        counts_agree(b)
        futr.futr_pages_init(b.ref.n, rows, b.pool._mem)


NOT_HELD = [
    # row and place of a table that is held but for one page there; its parents
    (0, 0, [0, 0, -1]),       # shared with every child
    (0, 1, [0, 0, -1]),       # the page that is partly written
    (0, 3, [0, 0, -1]),       # taken ahead
    (2, 1, [0, 0, -1]),       # of a sequence that ends
    (1, 2, [0, 1, 2]),        # nothing to copy
]


@pytest.mark.parametrize("case", range(len(NOT_HELD)))
@pytest.mark.parametrize("width", [4, 30000])        # a CTA looks at the table, and several
def test_pages_that_are_not_held_are_not_written_over(case, width):
    """A table made by hand of which a page was not counted: fork and compact would take that page for a copy. They change
    nothing; once it is counted they do as ever."""
    row, place, parent = NOT_HELD[case]
    b = Both(40, 16, 3, width, seed=case, max_pos=1 << 16)
    hand, pos = [[5, 6, 0, 8], [9, 10, 11, 12], [13, 14, 15, 16]], [20, 40, 33]
    for i, r in enumerate(hand):
        b.ref.table[i][:4] = r
    b.ref.table[row][place] = 1 if (row, place) != (0, 2) else 0
    missing = ints([[b.ref.table[row][place]]])
    b.table.copy_(ints(b.ref.table))
    part = b.table.clone()
    part[row, place] = -1
    futr.futr_pages_hold(b.cache, b.pool, part)
    was = b.bits.clone(), b.scales.clone(), b.table.clone(), futr.pages_refs(b.pool).clone()

    def unchanged():
        now = b.bits, b.scales, b.table, futr.pages_refs(b.pool)
        assert all(torch.equal(x, y) for x, y in zip(was, now))
        assert futr.futr_pages_check(b.pool)[0] == OK
        assert sum(counts_agree(b)) == 11

    p = ints(pos)
    for lo, hi in ((0, 20), (20, 40), (0, 0)):
        for _ in range(2):
            futr.futr_pages_fork(b.cache, b.pool, ints(parent), p, b.table)
            assert futr.futr_pages_check(b.pool)[0] == futr.FUTR_ERR_NOT_HELD
            assert p.tolist() == pos
            unchanged()
        futr.futr_pages_compact(b.cache, b.pool, b.table, lo, hi)
        assert futr.futr_pages_check(b.pool)[0] == futr.FUTR_ERR_NOT_HELD
        unchanged()
    futr.futr_pages_hold(b.cache, b.pool, missing)
    b.same()
    pos = b.fork(parent, pos)
    b.same()
    assert b.compact(0, 20)
    b.same()


def test_a_table_that_is_not_counted_at_all():
    """Two rows of pages 0 and 1, none counted: the partly written page is not copied over the first."""
    b = Both(8, 16, 2, 4)
    b.table[0, :2] = ints([0, 1])
    was, p = b.bits.clone(), ints([20, 0])
    futr.futr_pages_fork(b.cache, b.pool, ints([0, 0]), p, b.table)
    assert futr.futr_pages_check(b.pool) == (futr.FUTR_ERR_NOT_HELD, 8)
    assert torch.equal(b.bits, was) and p.tolist() == [20, 0] and b.table.tolist() == [[0, 1, -1, -1], [-1] * 4]
    futr.futr_pages_compact(b.cache, b.pool, b.table, 0, 8)
    assert futr.futr_pages_check(b.pool) == (futr.FUTR_ERR_NOT_HELD, 8)
    assert torch.equal(b.bits, was) and b.table.tolist() == [[0, 1, -1, -1], [-1] * 4]


@pytest.mark.parametrize("rows,new", [(2, 40), (40, 500)])      # places of one round, and of several
def test_new_rows_take_pages_for_ids_out_of_range(rows, new):
    """An id that is no page's is reported and counts as no page: rows that meet it get one."""
    width = -(-new // 16) + 2
    b = Both(rows * width, 16, rows, width, layers=1, hkv=1)
    b.table[:, 1], b.table[0, 0], b.table[1, 2] = rows * width, 2 ** 31 - 1, -5
    b.table[:, width - 1] = rows * width + 3                    # not met
    futr.futr_pages_grow(b.cache, b.pool, ints([0] * rows), starts([new] * rows), b.table)
    assert b.ref.grow([0] * rows, [new] * rows)
    assert b.table[:, width - 1].tolist() == [rows * width + 3] * rows
    b.table[:, width - 1] = -1
    b.same(futr.FUTR_ERR_OUT_OF_RANGE)
