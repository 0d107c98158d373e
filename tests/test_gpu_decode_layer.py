"""The paged cache and the mixture-of-experts layer used together, as a decoding loop
uses them: append, attention, experts; captured, side by side, and far into memory."""
import pytest
import torch

from int4_weight_kv_w4a16_gb300 import futr
from tests._gpu_helpers import ensure_lib
from tests._paged_ref import F64, Paged, ints, starts
from tests.test_gpu_moe import Moe
from tests.test_gpu_paged import check_append, check_attention, rows

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def check_experts(m, x, resid, y, ids, weights):
    """As the experts' own tests: the output's half step, the activations' rounding, the sums'."""
    ry, rw, bound = m.reference(x, ids, resid)
    assert float((weights.to(F64) / rw - 1).abs().max()) < 2.0 ** -15
    err = (y.to(F64) - ry).abs()
    assert bool((err <= 2.0 ** -8 * ry.abs() + bound + 2.0 ** -24).all())


class Layer:
    """Buffers and workspaces of one user: h -> cache, attention -> experts -> h."""

    def __init__(self, c, m, layer, batch, seed):
        self.c, self.m, self.layer, self.batch, self.seed = c, m, layer, batch, seed
        self.qkv = torch.empty((batch, c.heads + 2 * c.kv_heads, c.d), dtype=BF, device="cuda")
        self.q, self.k, self.v = self.qkv.split([c.heads, c.kv_heads, c.kv_heads], 1)
        self.h = torch.empty((batch, m.H), dtype=BF, device="cuda")
        self.att = torch.empty((batch, c.heads, c.d), dtype=BF, device="cuda")
        self.y = torch.empty_like(self.h)
        self.ids = torch.empty((batch, m.K), dtype=torch.int32, device="cuda")
        self.weights = torch.empty((batch, m.K), dtype=torch.float32, device="cuda")
        self.pos = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.paged_ws = futr.futr_paged_workspace_init(c.cs, futr.alloc_bytes(futr.futr_paged_workspace_size(c.cs)))
        self.moe_ws = futr.futr_moe_workspace_init(m.ms, batch, futr.alloc_bytes(
            futr.futr_moe_workspace_size(m.ms, batch)))

    def new_rows(self, step):
        self.qkv.copy_(rows(self.batch, self.qkv.shape[1], self.c.d, BF, 1000 * self.seed + step))
        self.h.copy_(rows(self.batch, 1, self.m.H, BF, 1000 * self.seed + 500 + step)[:, 0])

    def step(self):
        c, m = self.c, self.m
        futr.futr_paged_append(c.cache, self.layer, self.batch, self.pos, None, c.table, self.k, self.v)
        futr.futr_paged_attention(c.cache, self.layer, self.batch, self.pos, None, c.table, self.q, self.att,
                                  self.paged_ws)
        futr.futr_moe_layer(self.att.view(self.batch, -1), m.gain, m.router, m.blob, self.h, self.y, self.moe_ws,
                            ids=self.ids, weights=self.weights)

    def capture(self):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.step()
        return graph

    def status(self):
        return futr.futr_paged_check(self.c.cache, self.paged_ws), futr.futr_moe_check(self.moe_ws)


@pytest.mark.parametrize("heads,kv_heads,d,page,lens", [(8, 2, 64, 16, [0, 15, 16, 200, 47]),
                                                        (4, 4, 128, 64, [300])], ids=["batch5", "single"])
def test_prompt_then_captured_decoding(heads, kv_heads, d, page, lens):
    """A prompt enters the cache in one call, then one captured step is replayed token by token."""
    B = len(lens)
    c = Paged(heads, kv_heads, d, page, B, -(-(max(lens) + 8) // page), layers=2)
    m = Moe(heads * d, 384, 16, 3, seed=2)
    u = Layer(c, m, 1, B, 3)
    n = sum(lens)
    q, k, v = (rows(n, h, d, BF, 70 + i) for i, h in enumerate((heads, kv_heads, kv_heads)))
    out = torch.empty_like(q)
    zero = ints([0] * B)
    futr.futr_paged_append(c.cache, 1, B, zero, starts(lens), c.table, k, v)
    futr.futr_paged_attention(c.cache, 1, B, zero, starts(lens), c.table, q, out, u.paged_ws)
    check_attention(c, q, out, [0] * B, lens, layer=1)
    u.new_rows(99)
    u.pos.copy_(ints(lens))
    graph = u.capture()
    lens = [p + 1 for p in lens]
    for i in range(5):
        u.pos.copy_(ints(lens))
        u.new_rows(i)
        before = c.codes[1].clone(), c.scales[1].clone()
        graph.replay()
        assert u.status() == (futr.FUTR_OK, futr.FUTR_OK)
        check_append(c, before, u.k, u.v, lens, [1] * B, layer=1)
        check_attention(c, u.q, u.att, lens, [1] * B, layer=1)
        check_experts(m, u.att.view(B, -1), u.h, u.y, u.ids, u.weights)
        lens = [p + 1 for p in lens]
    assert int(c.codes[0].view(torch.uint8).max()) == 0    # the other layer stays as it was


def test_two_users_side_by_side():
    """Two captured steps with a workspace each, replayed on two streams at once, give what they give alone."""
    c = Paged(32, 8, 128, 64, 4, 40, layers=2)
    m = Moe(4096, 512, 8, 2, seed=4)
    for layer in (0, 1):
        c.fill(layer, layer=layer)
    users = [Layer(c, m, layer, 4, 5 + layer) for layer in (0, 1)]
    graphs = []
    for i, u in enumerate(users):
        u.pos.copy_(ints([2000, 1, 900 + i, 2400]))
        u.new_rows(0)
        graphs.append(u.capture())
    torch.cuda.synchronize()
    alone = []
    for u, g in zip(users, graphs):
        g.replay()
        torch.cuda.synchronize()
        alone.append((u.att.clone(), u.y.clone(), u.ids.clone()))
    streams = [torch.cuda.Stream() for _ in users]
    for _ in range(20):
        for u, g, s in zip(users, graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for u, (att, y, ids) in zip(users, alone):
        assert torch.equal(u.att, att) and torch.equal(u.y, y) and torch.equal(u.ids, ids)
        assert u.status() == (futr.FUTR_OK, futr.FUTR_OK)


@pytest.mark.parametrize("counts", [[1, 1], [40, 33], [150, 101]], ids=["rows1", "rows40", "rows150"])
def test_pages_past_four_gigabytes(counts):
    """Page ids whose codes lie more than 2^32 bytes into the cache's second layer."""
    c = Paged(8, 8, 128, 128, 2, 4, layers=2)
    n_pages = 10000                                   # 2^18 bytes a page: 2.6 GB a layer
    size = futr.futr_paged_size(c.cs, 2, n_pages, 128, c.max_pos)
    assert size > 2 ** 32 + 2 ** 29
    c.cache = futr.futr_paged_init(c.cs, 2, n_pages, 128, c.max_pos, True, futr.alloc_bytes(size))
    c.codes, c.scales = futr.paged_views(c.cache)
    c.n_pages = n_pages
    c.table = n_pages - 1 - c.table                   # the last pages, in a shuffled order
    lens = [200, 131]
    k, v = (rows(sum(lens), 8, 128, BF, s) for s in (1, 2))
    futr.futr_paged_append(c.cache, 1, 2, ints([0, 0]), starts(lens), c.table, k, v)
    before = c.codes[1].clone(), c.scales[1].clone()
    q, k, v = (rows(sum(counts), 8, 128, BF, s) for s in (3, 4, 5))
    out = torch.empty_like(q)
    futr.futr_paged_append(c.cache, 1, 2, ints(lens), starts(counts), c.table, k, v)
    futr.futr_paged_attention(c.cache, 1, 2, ints(lens), starts(counts), c.table, q, out, c.ws)
    assert futr.futr_paged_check(c.cache, c.ws) == futr.FUTR_OK
    check_append(c, before, k, v, lens, counts, layer=1)
    check_attention(c, q, out, lens, counts, layer=1)


def test_experts_past_four_gigabytes():
    """The last of 256 experts of the 8B block's width, more than 2^32 bytes into the blob."""
    H, I, E = 4096, 4096, 256
    m = Moe.__new__(Moe)
    m.H, m.I, m.E, m.K, m.renorm, m.eps, m.gain = H, I, E, 2, True, 1e-5, None
    m.ms = futr.make_moe_shape(H, I, E, 2)
    size = futr.futr_moe_weights_size(m.ms)
    assert size > 2 ** 32 + 2 ** 31
    m.blob = futr.alloc_bytes(size)
    g = torch.Generator(device="cuda").manual_seed(3)
    for e in range(E):
        if e in (0, 1, 253, 254, 255):
            w = [torch.randn(s, generator=g, device="cuda") * 0.02 for s in ((I, H), (I, H), (H, I))]
        futr.futr_moe_pack(m.ms, e, *w, None, m.blob)
    m.router = torch.full((E, H), -2.0 ** -7, device="cuda", dtype=BF)
    for i, e in enumerate((255, 254, 0)):
        m.router[e] = (3 - i) * 2.0 ** -7
    m.ws = futr.futr_moe_workspace_init(m.ms, 9, futr.alloc_bytes(futr.futr_moe_workspace_size(m.ms, 9)))
    for T in (1, 9):
        x = rows(T, 1, H, BF, T)[:, 0].abs()          # positive: the order of the experts is the router's
        y, ids, weights = m.run(x)
        assert ids.tolist() == [[255, 254]] * T
        check_experts(m, x, None, y, ids, weights)
