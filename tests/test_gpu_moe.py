"""INT4 mixture-of-experts layer against a plain 64-bit form."""
import numpy as np
import pytest
import torch

import oracle
from int4_weight_kv_w4a16_gb300 import futr
from tests._gpu_helpers import ensure_lib

pytestmark = pytest.mark.gpu
F64 = torch.float64


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


class Moe:
    def __init__(self, H, I, E, K, renorm=True, eps=1e-5, seed=0, max_batch=32):
        self.H, self.I, self.E, self.K, self.renorm, self.eps = H, I, E, K, renorm, eps
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.g = g
        self.ms = futr.make_moe_shape(H, I, E, K, renorm=renorm, rms_eps=eps)
        self.blob = futr.alloc_bytes(futr.futr_moe_weights_size(self.ms))
        self.gain = torch.rand(H, generator=g, device="cuda") + 0.5 if eps else None
        self.router = (torch.randn((E, H), generator=g, device="cuda") * H ** -0.5).to(torch.bfloat16)
        self.w = []
        for e in range(E):
            w = [torch.randn(s, generator=g, device="cuda") * 0.05 for s in ((I, H), (I, H), (H, I))]
            futr.futr_moe_pack(self.ms, e, *w, self.gain, self.blob)
            self.w.append(w if E <= 8 else None)
        self.ws = futr.futr_moe_workspace_init(self.ms, max_batch, futr.alloc_bytes(
            futr.futr_moe_workspace_size(self.ms, max_batch)))

    def unpack(self, e, which):
        r, c = (self.H, self.I) if which == futr.FUTR_PROJ_DOWN else (self.I, self.H)
        codes = torch.empty((r, c), dtype=torch.int8, device="cuda")
        scales = torch.empty((r, c // 128), dtype=torch.float16, device="cuda")
        futr.futr_moe_unpack(self.ms, self.blob, e, which, codes, scales)
        return codes, scales

    def full(self, e, which):
        c, s = self.unpack(e, which)
        return c.to(F64) * s.to(F64).repeat_interleave(128, 1)

    def run(self, x, resid=None, y=None):
        T = x.shape[0]
        y = torch.empty_like(x) if y is None else y
        ids = torch.empty((T, self.K), dtype=torch.int32, device="cuda")
        weights = torch.empty((T, self.K), dtype=torch.float32, device="cuda")
        futr.futr_moe_layer(x, self.gain, self.router, self.blob, resid, y, self.ws, ids=ids, weights=weights)
        assert futr.futr_moe_check(self.ws) == futr.FUTR_OK
        return y, ids, weights

    def reference(self, x, ids, resid=None):
        """(y, weights, bound): the layer in 64 bits for the choice `ids`, which has to
        be the largest logits within what fp32 can tell apart: a logit is a sum of
        H products, each rounded, in chains of 8 + H / 256 + 5 additions, times a
        factor good to 4 roundings: under 2^-18 of the sum of magnitudes.  bound:
        what rounding the activations to bf16, 2^-8 each, and the fp32 sums (2^-16)
        can move an output by."""
        x = x.to(F64)
        r = 1 / torch.sqrt((x * x).mean(1, keepdim=True) + self.eps) if self.eps else torch.ones_like(x[:, :1])
        h = x * self.gain.to(F64) if self.gain is not None else x
        logits = r * (h @ self.router.to(F64).t())
        doubt = 2.0 ** -18 * (r * (h.abs() @ self.router.to(F64).abs().t())).amax(1, keepdim=True)
        ids = ids.long()
        best = torch.sort(logits, dim=1, descending=True).values[:, :self.K]
        assert bool(((logits.gather(1, ids) - best).abs() <= 2 * doubt).all())
        assert all(len(set(row)) == self.K for row in ids.tolist())
        w = torch.softmax(logits, 1).gather(1, ids)
        if self.renorm:
            w = w / w.sum(1, keepdim=True)
        y = resid.to(F64).clone() if resid is not None else torch.zeros_like(x)
        bound = torch.zeros_like(y)
        for e in torch.unique(ids).tolist():
            t, slot = (ids == e).nonzero(as_tuple=True)
            gate, up = ((r[t] * x[t]) @ self.full(e, p).t() for p in (futr.FUTR_PROJ_GATE, futr.FUTR_PROJ_UP))
            a = w[t, slot][:, None] * gate * torch.sigmoid(gate) * up
            down = self.full(e, futr.FUTR_PROJ_DOWN).t()
            y[t] += a @ down
            bound[t] += (2.0 ** -8 + 2.0 ** -16) * (a.abs() @ down.abs())
        return y, w, bound

    def check(self, x, resid=None):
        y, ids, w = self.run(x, resid)
        ry, rw, bound = self.reference(x, ids, resid)
        # twice a logit's error: 2^-18 of a sum of magnitudes under 4
        assert float((w.to(F64) / rw - 1).abs().max()) < 2.0 ** -15
        err = (y.to(F64) - ry).abs()
        tol = 2.0 ** -8 * ry.abs() + bound + 2.0 ** -24
        assert bool((err <= tol).all()), float((err / tol).max())
        # roundings of both signs: the whole differs by less than one half step of each kind
        assert float(err.norm() / ry.norm()) <= 2 * 2.0 ** -8
        return y


def rows(m, T, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((T, m.H), generator=g, device="cuda").to(torch.bfloat16)


@pytest.mark.parametrize("H,I,E,K,renorm,eps", [
    (256, 768, 4, 2, True, 1e-5),
    (128, 128, 1, 1, False, 0.0),
    (384, 256, 5, 5, False, 1e-5),
    (1024, 384, 64, 6, True, 0.0),
    (256, 128, 256, 16, True, 1e-5),
    (640, 1408, 60, 4, False, 1e-5),
], ids=lambda v: str(v))
def test_layer(H, I, E, K, renorm, eps):
    m = Moe(H, I, E, K, renorm, eps, seed=3)
    for T in (1, 2, 7, 8, 9, 16, 17, 32):
        x = rows(m, T, T)
        res = rows(m, T, 50 + T) if T % 2 else None
        y = m.check(x, res)
        assert torch.equal(m.run(x, res)[0], y)   # no sum depends on timing


def test_packed_codes_match_the_quantizer():
    m = Moe(256, 384, 3, 2, seed=8)
    for e in range(3):
        for which, w, gain in ((futr.FUTR_PROJ_GATE, m.w[e][0], m.gain), (futr.FUTR_PROJ_UP, m.w[e][1], m.gain),
                               (futr.FUTR_PROJ_DOWN, m.w[e][2], None)):
            w = (w * gain if gain is not None else w).cpu().numpy()
            codes, scales = m.unpack(e, which)
            g = w.reshape(w.shape[0], -1, 128)
            s = np.minimum((np.abs(g).max(-1) / np.float32(7)).astype(np.float32), np.float32(65504)).astype(np.float16)
            c = np.clip(np.rint((g / s.astype(np.float32)[..., None]).astype(np.float32)), -8, 7).astype(np.int8)
            np.testing.assert_array_equal(codes.cpu().numpy(), c.reshape(w.shape))
            np.testing.assert_array_equal(scales.cpu().numpy(), s)


def test_larger_layer_with_split_rows():
    """The 8B block's width: each row block is shared by several CTAs."""
    m = Moe(4096, 14336, 2, 2, seed=4)
    m.check(rows(m, 1), rows(m, 1, 9))
    m.check(rows(m, 20), None)


@pytest.mark.parametrize("I", [128, 1280])
def test_more_row_blocks_than_ctas(I):
    """A wide layer: CTAs of the down product own several row blocks, whole ones beside parts."""
    m = Moe(65536, I, 1, 1, eps=0.0, seed=11)
    for T in (1, 8, 9, 20):
        m.check(rows(m, T, T), rows(m, T, 30 + T))


def test_every_token_with_one_expert_and_equal_logits():
    """All tokens at the same experts (full columns), and ties: the lowest experts first."""
    m = Moe(256, 256, 8, 3, seed=5)
    m.router.zero_()
    y, ids, w = m.run(rows(m, 32))
    assert torch.equal(ids.cpu(), torch.arange(3, dtype=torch.int32).expand(32, 3))
    assert bool((w == torch.full_like(w, 1 / 3)).all())
    x = rows(m, 32)
    ry = torch.zeros((32, 256), dtype=F64, device="cuda")
    r = 1 / torch.sqrt((x.to(F64) ** 2).mean(1, keepdim=True) + 1e-5)
    for e in range(3):
        gate, up = ((r * x.to(F64)) @ m.full(e, p).t() for p in (futr.FUTR_PROJ_GATE, futr.FUTR_PROJ_UP))
        ry += (gate * torch.sigmoid(gate) * up / 3) @ m.full(e, futr.FUTR_PROJ_DOWN).t()
    assert float((y.to(F64) - ry).norm() / ry.norm()) <= 2 * 2.0 ** -8


def test_output_over_input_and_residual():
    m = Moe(512, 256, 8, 2, seed=6)
    x, res = rows(m, 5), rows(m, 5, 2)
    want = m.run(x, res)[0]
    a = x.clone()
    assert torch.equal(m.run(a, res, y=a)[0], want)
    b = res.clone()
    assert torch.equal(m.run(x, b, y=b)[0], want)


def test_rows_with_nan_stay_their_own():
    m = Moe(256, 256, 8, 2, seed=7)
    x = rows(m, 6)
    want, ids, _ = m.run(x)
    bad = x.clone()
    bad[2, 17] = float("nan")
    y, bids, w = m.run(bad)
    assert bool(torch.isnan(w[2]).all()) and bool(torch.isnan(y[2]).all())
    keep = [0, 1, 3, 4, 5]
    assert torch.equal(bids[keep], ids[keep])
    assert bool(((bids[2] >= 0) & (bids[2] < 8)).all())
    # (a row's columns are its own; how the shares cut depends on the whole batch's routing, so the
    # fp32 sums may come in another order)
    assert float((y[keep].float() - want[keep].float()).norm() / want[keep].float().norm()) <= 2.0 ** -8


def test_foreign_blob_is_reported():
    m = Moe(256, 256, 4, 2, seed=9)
    x = rows(m, 2)
    keep = m.blob[:16].clone()
    m.blob[:8] = 0
    y = torch.empty_like(x)
    futr.futr_moe_layer(x, m.gain, m.router, m.blob, None, y, m.ws)
    assert futr.futr_moe_check(m.ws) == futr.FUTR_ERR_BAD_BLOB
    m.blob[:16] = keep
    m.check(x)


def test_graph_replay_with_other_tokens():
    m = Moe(1024, 512, 16, 4, seed=10)
    x, res = rows(m, 3), rows(m, 3, 2)
    y = torch.empty_like(x)
    ids = torch.empty((3, 4), dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        futr.futr_moe_layer(x, m.gain, m.router, m.blob, res, y, m.ws, ids=ids)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        futr.futr_moe_layer(x, m.gain, m.router, m.blob, res, y, m.ws, ids=ids)
    for i in range(3):
        x.copy_(rows(m, 3, 30 + i))
        graph.replay()
        assert futr.futr_moe_check(m.ws) == futr.FUTR_OK
        ry, _, bound = m.reference(x, ids, res)
        assert bool(((y.to(F64) - ry).abs() <= 2.0 ** -8 * ry.abs() + bound + 2.0 ** -24).all())


@pytest.mark.parametrize("T", [1, 9, 32])
@pytest.mark.parametrize("word,value", [(0, 0), (3, 128), (4, 128), (5, 3)], ids=["magic", "hidden", "inter", "experts"])
def test_foreign_blob_is_not_read(word, value, T):
    """A header of another layer: the status, and an output that stays as it was."""
    m = Moe(256, 256, 4, 2, seed=9)
    x = rows(m, T)
    header = m.blob[:24].view(torch.int32)
    keep = header.clone()
    header[word] = value
    y = torch.full_like(x, 7.0)
    futr.futr_moe_layer(x, m.gain, m.router, m.blob, None, y, m.ws)
    assert futr.futr_moe_check(m.ws) == futr.FUTR_ERR_BAD_BLOB
    assert bool((y == 7).all())
    header.copy_(keep)
    m.check(x)


def moe_error(m, x):
    """The layer's error next to its own size: the residual takes the expected output away, so that
    the bf16 rounding of what is left says nothing."""
    ids = m.run(x)[1]
    ry, _, _ = m.reference(x, ids)
    resid = (-ry).to(torch.bfloat16)
    y, again, _ = m.run(x, resid)
    assert torch.equal(again, ids)
    return float((y.to(F64) - (resid.to(F64) + ry)).norm() / ry.norm())


# activations w * silu * up are rounded to 11 bits: 2^-11 / sqrt(3) of each at the most, in the mean square
# and of both signs; inputs of the first product that are exact, or rounded the same way, add less;
# the sums are fp32
MOE_ERROR = 3e-4


@pytest.mark.parametrize("T", [1, 8, 20, 32])
@pytest.mark.parametrize("H,I", [(16384, 128), (128, 16384), (4096, 512)])
def test_inputs_of_one_sign(H, I, T):
    """Positive inputs: codes of both signs cancel, the sums of what carries them do not."""
    m = Moe(H, I, 1, 1, eps=0.0, seed=12)
    wg, _, wd = m.w[0]
    futr.futr_moe_pack(m.ms, 0, wg, wg, wd, None, m.blob)       # silu(g) g: (nearly) one sign, too
    g = torch.Generator(device="cuda").manual_seed(T)
    x = (0.5 + torch.rand((T, H), generator=g, device="cuda")).to(torch.bfloat16)
    assert moe_error(m, x) <= MOE_ERROR


@pytest.mark.parametrize("T", [1, 9, 32])
def test_activations_keep_eleven_bits(T):
    m = Moe(1024, 640, 4, 2, seed=13)
    assert moe_error(m, rows(m, T)) <= MOE_ERROR


@pytest.mark.parametrize("T", [1, 9, 32])
def test_activations_far_apart(T):
    """Groups whose activations are 2^16 apart and count the same: each has a factor of its own."""
    m = Moe(512, 640, 1, 1, eps=0.0, seed=14)
    wg, wu, wd = m.w[0]
    f = 2.0 ** (8 - 4 * torch.arange(5, device="cuda").repeat_interleave(128).float())
    futr.futr_moe_pack(m.ms, 0, wg, wu * f[:, None], wd / f, None, m.blob)
    assert moe_error(m, rows(m, T)) <= MOE_ERROR


@pytest.mark.parametrize("T", [1, 20])
def test_a_copy_that_never_comes(monkeypatch, T):
    """The first CTA's waits run out (test hook): the call ends with a status, and the next is exact again."""
    m = Moe(512, 640, 8, 2, seed=15)
    x = rows(m, T)
    good = m.check(x)
    for _ in range(2):
        monkeypatch.setenv("FUTR_TEST_WITHHOLD_COPY", "1")
        futr.futr_moe_layer(x, m.gain, m.router, m.blob, None, torch.empty_like(x), m.ws)
        monkeypatch.delenv("FUTR_TEST_WITHHOLD_COPY")
        assert futr.futr_moe_check(m.ws) == futr.FUTR_ERR_TIMEOUT
        assert torch.equal(m.run(x)[0], good)
