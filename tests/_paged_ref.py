"""The paged 8-bit cache in 64 bits: plain restatements that the GPU tests
compare with, and the set-up they share."""
import dataclasses
import math

import numpy as np
import torch

from int4_weight_kv_w4a16_gb300 import futr, inputs

F64 = torch.float64


def shape_of(heads, kv_heads, d, theta=500000.0):
    return inputs.BlockShape(hidden=128, n_q_heads=heads, n_kv_heads=kv_heads, head_dim=d, inter=128, had_block=d,
                             rope_theta=theta)


def rotate(x, pos, theta):
    """x [rows, heads, d] (64 bits), dims i and i + d/2 turned by pos * theta^(-2i/d)."""
    d = x.shape[-1]
    f = theta ** (-torch.arange(0, d, 2, dtype=F64, device=x.device) / d)
    a = pos.to(F64)[:, None, None] * f
    x1, x2 = x[..., :d // 2], x[..., d // 2:]
    return torch.cat([x1 * a.cos() - x2 * a.sin(), x2 * a.cos() + x1 * a.sin()], -1)


def page_scale(amax: float) -> float:
    """The smallest power of two s with amax <= 448 s, at least 2^-60."""
    if amax == 0:
        return 2.0 ** -60
    m, e = math.frexp(amax)   # 448 = 0.875 * 2^9
    return 2.0 ** max(e - 9 if m <= 0.875 else e - 8, -60)


@dataclasses.dataclass
class Paged:
    """A cache with its page table (a shuffled pool), on cuda:0."""
    heads: int
    kv_heads: int
    d: int
    page: int
    batch: int
    width: int          # pages of a sequence
    layers: int = 1
    rope: bool = True
    seed: int = 0

    def __post_init__(self):
        self.shape = shape_of(self.heads, self.kv_heads, self.d)
        self.cs = futr.make_shape(self.shape)
        self.n_pages = self.batch * self.width + 2
        self.max_pos = self.width * self.page
        size = futr.futr_paged_size(self.cs, self.layers, self.n_pages, self.page, self.max_pos)
        self.cache = futr.futr_paged_init(self.cs, self.layers, self.n_pages, self.page, self.max_pos, self.rope,
                                          futr.alloc_bytes(size))
        self.ws = futr.futr_paged_workspace_init(self.cs, futr.alloc_bytes(futr.futr_paged_workspace_size(self.cs)))
        r = np.random.default_rng(self.seed + 99)
        self.table = torch.from_numpy(r.permutation(self.n_pages)[:self.batch * self.width].astype(np.int32)
                                      .reshape(self.batch, self.width)).cuda()
        self.codes, self.scales = futr.paged_views(self.cache)

    def fill(self, seed=0, gain=20.0, layer=0):
        """Every page of the layer: normal values, four key channels a head times gain."""
        g = torch.Generator(device="cuda").manual_seed(seed)
        x = torch.randn(self.codes.shape[1:], generator=g, device="cuda")
        x[:, :, 0, :, :4] *= gain
        m, e = torch.frexp(x.abs().amax((3, 4)))
        s = torch.ldexp(torch.ones_like(m), torch.where(m <= 0.875, e - 9, e - 8))
        self.codes[layer].copy_((x / s[..., None, None]).to(torch.float8_e4m3fn))
        self.scales[layer].copy_(s)

    def values(self, b, n, layer=0):
        """Keys and values of positions 0..n-1 of sequence b: [kv-heads, n, d] in 64 bits."""
        tab = self.table[b, :-(-n // self.page)].long()
        v = self.codes[layer][tab].to(F64) * self.scales[layer][tab].to(F64)[..., None, None]
        v = v.permute(1, 2, 0, 3, 4).reshape(self.kv_heads, 2, -1, self.d)[:, :, :n]
        return v[:, 0], v[:, 1]

    def attention(self, q, pos, counts, window=0, scale=None, layer=0):
        """Outputs [rows, heads, d] in 64 bits, and each element's bound on what the
        kernel's roundings may add (see the caller)."""
        out = torch.zeros(q.shape, dtype=F64, device="cuda")
        bound = torch.zeros_like(out)
        scale = scale or self.d ** -0.5
        G, r = self.heads // self.kv_heads, 0
        for b, n in enumerate(counts):
            if n:
                p0 = pos[b]
                at = torch.arange(p0, p0 + n, device="cuda")
                x = q[r:r + n].to(F64)
                x = (rotate(x, at, self.shape.rope_theta) if self.rope else x).transpose(0, 1)   # [heads, n, d]
                k, v = (t.repeat_interleave(G, 0) for t in self.values(b, p0 + n, layer))
                s = x @ k.transpose(1, 2) * scale
                age = at[:, None] - torch.arange(p0 + n, device="cuda")
                s[:, (age < 0) | ((age >= window) if window else (age < 0))] = -math.inf
                w = torch.softmax(s, -1)
                out[r:r + n] = (w @ v).transpose(0, 1)
                spread = (w @ v.abs()).transpose(0, 1)                      # mean |v| under the weights
                # the largest sum of |q_i k_i| of a visible key: what a query
                # rounded to 11 bits can move a score by, times 2^-11
                mag = (x.abs() @ k.abs().transpose(1, 2) * scale).masked_fill(s == -math.inf, 0).amax(-1)
                moved = (2.0 ** -11 + 2.0 ** -18) * mag.transpose(0, 1)[..., None]
                bound[r:r + n] = (2.0 ** -11 + 2.0 ** -16 + 2 * moved) * spread
            r += n
        return out, bound


def starts(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")
