"""Workloads of the paged 8-bit key/value cache and of the mixture-of-experts layer, and their plain forms.

Three operators, as one decode layer of a served model uses them:

* ``append``: new key and value rows of ragged sequences go into a paged cache. Keys are rotated by position on the
  way; a page holds e4m3 codes with one power-of-two scale for each (page, kv-head) of keys and of values, and a
  page whose scale has to grow is brought to the new scale.
* ``attention``: causal grouped-query attention of the new rows over that cache, the query rotated by position.
* ``moe``: RMSNorm factor, router, top-k experts with INT4 weights (SwiGLU) and the weighted sum, for 1 to 32 tokens.

With ``own`` false, ``run`` computes them in elementary torch operations in 32 bits (angles and router logits in 64);
with ``own`` true it calls the framework. ``prepare`` builds what a program keeps: the page pool, the page table, the
packed experts, the workspaces.
"""
import math

import torch

own = False

THETA = 500000.0
EPS = 1e-5
E4M3_MAX = 448.0
MIN_EXP = -60        # the smallest page scale is 2^-60
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------- cases --

def _kv(name, op, batch, lo, hi, new, heads, kv_heads, d, page, dtype, window=0, fused=False, hole=False):
    c = {"op": op, "batch": batch, "lo": lo, "hi": hi, "new": new, "heads": heads, "kv_heads": kv_heads, "d": d,
         "page": page, "dtype": dtype, "window": window, "fused": fused, "hole": hole}
    return dict(c, name=name) if name else c


def _moe(name, tokens, experts, top_k, hidden, inter, renorm, norm, resid):
    c = {"op": "moe", "tokens": tokens, "experts": experts, "top_k": top_k, "hidden": hidden, "inter": inter,
         "renorm": renorm, "norm": norm, "resid": resid}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one user, one new token of the 8B-shaped block: what a call costs at the least
        _kv("append_b1", "append", 1, 1023, 1023, 1, 32, 8, 128, 16, "bf16"),
        # a served batch of 32 at ragged lengths, one new token each, rows cut out of a fused QKV product
        _kv("append_b32", "append", 32, 512, 4096, 1, 32, 8, 128, 64, "bf16", fused=True),
        # prompts that enter the cache: four sequences of up to 4095 new tokens, pages that start and end ragged
        _kv("append_prompts", "append", 4, 5, 300, 4095, 32, 8, 128, 64, "f16"),
        # one user at 1024 cached tokens: the latency case of decoding
        _kv("attn_b1_ctx1024", "attention", 1, 1024, 1024, 1, 32, 8, 128, 16, "bf16"),
        # the served batch of 32 at ragged lengths
        _kv("attn_b32_ragged", "attention", 32, 512, 4096, 1, 32, 8, 128, 64, "bf16", fused=True),
        # few users with long documents, the 70B-shaped block's heads
        _kv("attn_b4_long", "attention", 4, 20000, 50000, 1, 64, 8, 128, 64, "bf16"),
        # checking drafted tokens: up to 5 new tokens a sequence, head size 64, a window, one idle sequence
        _kv("attn_draft", "attention", 16, 300, 3000, 5, 16, 4, 64, 32, "f16", window=1000, hole=True),
        # a chunk of a prompt behind what is cached already: the product-bound end
        _kv("attn_chunk", "attention", 4, 500, 4000, 511, 32, 8, 128, 64, "bf16", fused=True),
        # one token through 2 of 8 experts of the 8B-shaped block
        _moe("moe_t1_8of2", 1, 8, 2, 4096, 14336, True, True, True),
        # a batch of 32 through them: all experts are read
        _moe("moe_t32_8of2", 32, 8, 2, 4096, 14336, True, True, True),
        # many small experts, one token: the smallest call
        _moe("moe_t1_64of6", 1, 64, 6, 2048, 1408, False, False, False),
        # many experts, a batch of 17: most of them see one or two tokens
        _moe("moe_t17_128of8", 17, 128, 8, 4096, 1536, True, True, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_kv(rng, op):
    d = rng.choice([64, 128, 128])
    kv_heads = rng.choice([2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 4, 4, 5, 7, 8, 8, 16])
    page = rng.choice([16, 32, 64, 128])
    window = rng.choice([0, 0, 0, _log(rng, 17, 4000)]) if op == "attention" else 0
    dtype, fused, hole = rng.choice(["bf16", "f16"]), rng.random() < 0.5, rng.random() < 0.3
    if op == "append" and rng.random() < 0.5:      # prompts
        batch, new = _log(rng, 1, 6), _log(rng, 9, 2500)
    elif op == "attention" and rng.random() < 0.3:  # chunks
        batch, new = _log(rng, 1, 4), _log(rng, 9, 300)
    else:                                           # decoding, drafted tokens
        batch, new = _log(rng, 1, 48), rng.choice([1, 1, 1, 2, 3, 8])
    most = max(64, min(50000, (1 << 20) // (batch * kv_heads)))
    hi = _log(rng, 16, most)
    lo = rng.choice([hi, int(hi * rng.random())])
    return _kv(None, op, batch, lo, hi, new, heads, kv_heads, d, page, dtype, window, fused, hole and batch > 1)


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "moe", "moe"])
    if op != "moe":
        return _draw_kv(rng, op)
    tokens = rng.choice([1, 1, 2, 3, 32, _log(rng, 1, 32), _log(rng, 1, 32)])
    experts = rng.choice([4, 8, 16, 60, 64, 128])
    hidden = 128 * _log(rng, 4, 40)
    most = max(2, (8 * 4096 * 14336 // 2) // (experts * hidden * 128))
    inter = 128 * _log(rng, 1, min(112, most))
    return _moe(None, tokens, experts, rng.choice([k for k in (1, 2, 4, 6, 8) if k <= experts]), hidden, inter,
                rng.random() < 0.5, rng.random() < 0.7, rng.random() < 0.7)


def _lens(case):
    """Cached tokens and new rows of each sequence: spread over their ranges, fixed by the case."""
    past, new = [], []
    for b in range(case["batch"]):
        f = (0.5 + 0.6180339887498949 * b) % 1.0
        past.append(case["lo"] + int(round((case["hi"] - case["lo"]) * f)))
        n = case["new"] if b == case["batch"] - 1 else 1 + int((case["new"] - 1) * f)
        new.append(0 if case["hole"] and b == 0 else n)
    return past, new


def _visible(case):
    """(query, key) pairs that the mask leaves, and cached tokens that some query sees."""
    pairs = keys = 0
    w = case["window"] or (1 << 40)
    for p, n in zip(*_lens(case)):
        if n:
            pairs += sum(min(w, p + i + 1) for i in range(n))
            keys += min(p + n, w + n - 1)
    return pairs, keys


def work(case):
    if case["op"] == "moe":
        T, E, K, H, I = (case[k] for k in ("tokens", "experts", "top_k", "hidden", "inter"))
        used = E * (1 - (1 - K / E) ** T)              # experts that T tokens are expected to meet
        weight = 8448 / 16384                          # bytes a weight: a nibble and its share of the scales
        return {"bytes": used * 3 * H * I * weight + E * H * 2 + T * H * 2 * (3 if case["resid"] else 2),
                "flops": 2.0 * 3 * H * I * T * K + 2.0 * T * E * H}
    past, new = _lens(case)
    rows, Hkv, d = sum(new), case["kv_heads"], case["d"]
    if case["op"] == "append":
        return {"bytes": rows * (Hkv * d * 2 * 3 + 4 * d), "flops": rows * Hkv * d * 12.0}
    pairs, keys = _visible(case)
    return {"bytes": keys * Hkv * 2 * (d + 4 / case["page"]) + rows * case["heads"] * d * 4,
            "flops": 4.0 * pairs * case["heads"] * d}


# ------------------------------------------------------------------ inputs --

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(1000003 * (int(seed) + 1))


def _page_scale(amax):
    """The smallest power of two 2^e with amax <= 448 * 2^e, and at least 2^MIN_EXP."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=MIN_EXP)
    return torch.ldexp(torch.ones_like(amax), e)


def _kv_inputs(case, seed):
    """The page pool with its history, the table, and this step's rows: plain tensors, the same for both sides."""
    g = _generator(seed)
    past, new = _lens(case)
    B, Hq, Hkv, d, page = (case[k] for k in ("batch", "heads", "kv_heads", "d", "page"))
    need = [-(-(p + n) // page) if p + n else 1 for p, n in zip(past, new)]
    width, total = max(need), sum(need)
    n_pages = total + 3
    perm = torch.randperm(n_pages, generator=g, device="cuda", dtype=torch.int64)[:total]
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    at = torch.tensor([b * width + i for b in range(B) for i in range(need[b])], device="cuda")
    table.view(-1)[at] = perm.to(torch.int32)
    # history: normal keys and values, four key channels of each head 20 times as large
    codes = torch.empty((n_pages, Hkv, 2, page, d), dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty((n_pages, Hkv, 2), dtype=torch.float32, device="cuda")
    gain = torch.ones((Hkv, 2, 1, d), device="cuda")
    gain[:, 0, :, torch.randperm(d, generator=g, device="cuda")[:4]] = 20.0
    step = max(1, (1 << 27) // (Hkv * 2 * page * d))
    for i in range(0, n_pages, step):
        x = torch.randn((min(step, n_pages - i), Hkv, 2, page, d), generator=g, device="cuda") * gain
        s = _page_scale(x.abs().amax((3, 4)))
        codes[i:i + step] = (x / s[..., None, None]).to(torch.float8_e4m3fn)
        scales[i:i + step] = s
    rows, dt = sum(new), DTYPES[case["dtype"]]
    qkv = torch.randn((rows, Hq + 2 * Hkv, d), generator=g, device="cuda")
    qkv[:, Hq:Hq + Hkv] *= gain[:, 0, 0]
    qkv = qkv.to(dt)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    if not case["fused"]:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    start = torch.tensor([sum(new[:b]) for b in range(B + 1)], dtype=torch.int32, device="cuda")
    # rows of the sequences in order, each with its sequence and its position
    seq = torch.tensor([b for b in range(B) for _ in range(new[b])], dtype=torch.int64, device="cuda")
    where = torch.tensor([past[b] + i for b in range(B) for i in range(new[b])], dtype=torch.int64, device="cuda")
    st = {"case": case, "codes": codes, "scales": scales, "table": table, "q": q, "k": k, "v": v, "start": start,
          "pos": torch.tensor(past, dtype=torch.int32, device="cuda"), "seq": seq, "where": where,
          "longest": max(p + n for p, n in zip(past, new)), "most": max(new), "n_pages": n_pages}
    if case["op"] == "attention":
        # the step's keys and values are in the cache already: their pages' codes above stand for them
        del st["k"], st["v"]
    else:
        del st["q"]
    return st


def _moe_inputs(case, seed):
    g = _generator(seed)
    T, E, H, I = (case[k] for k in ("tokens", "experts", "hidden", "inter"))
    gain = torch.rand(H, generator=g, device="cuda") + 0.5 if case["norm"] else None
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    resid = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16) if case["resid"] else None
    router = (torch.randn((E, H), generator=g, device="cuda") * H ** -0.5).to(torch.bfloat16)
    return g, {"case": case, "x": x, "gain": gain, "resid": resid, "router": router}


def _quantized(w, gain):
    """INT4 codes and fp16 scales of each (output row, 128 inputs), the gain folded in first."""
    if gain is not None:
        w = w * gain
    w = w.view(w.shape[0], -1, 128)
    s = (w.abs().amax(-1) / 7.0).clamp(max=65504.0).to(torch.float16)
    sf = s.float()[..., None]
    c = torch.where(sf > 0, torch.round(w / sf), torch.zeros_like(w)).clamp(-8, 7)
    return c.to(torch.int8).view(w.shape[0], -1), s


def _experts(case, g):
    """Each expert's gate, up and down weights in fp32, one expert after another."""
    H, I = case["hidden"], case["inter"]
    for e in range(case["experts"]):
        yield e, [torch.randn(s, generator=g, device="cuda") * 0.02 for s in ((I, H), (I, H), (H, I))]


def prepare(case, seed):
    if case["op"] != "moe":
        st = _kv_inputs(case, seed)
        if own:
            from int4_weight_kv_w4a16_gb300 import futr, inputs
            sh = futr.make_shape(inputs.BlockShape(hidden=128, n_q_heads=case["heads"], n_kv_heads=case["kv_heads"],
                                                   head_dim=case["d"], inter=128, had_block=case["d"],
                                                   rope_theta=THETA))
            size = (1, st["n_pages"], case["page"], st["longest"])
            cache = futr.futr_paged_init(sh, *size, True, futr.alloc_bytes(futr.futr_paged_size(sh, *size)))
            codes, scales = futr.paged_views(cache)
            codes[0].copy_(st["codes"])
            scales[0].copy_(st["scales"])
            st |= {"cache": cache, "codes": codes[0], "scales": scales[0]}
            if case["op"] == "attention":
                st["ws"] = futr.futr_paged_workspace_init(sh, futr.alloc_bytes(futr.futr_paged_workspace_size(sh)))
        if case["op"] == "attention":
            st["out"] = torch.empty(st["q"].shape, dtype=st["q"].dtype, device="cuda")
        return st
    g, st = _moe_inputs(case, seed)
    T, E, H, I = (case[k] for k in ("tokens", "experts", "hidden", "inter"))
    if own:
        from int4_weight_kv_w4a16_gb300 import futr
        ms = futr.make_moe_shape(H, I, E, case["top_k"], renorm=case["renorm"], rms_eps=EPS if case["norm"] else 0.0)
        blob = futr.alloc_bytes(futr.futr_moe_weights_size(ms))
        for e, (wg, wu, wd) in _experts(case, g):
            futr.futr_moe_pack(ms, e, wg, wu, wd, st["gain"], blob)
        ws = futr.futr_moe_workspace_init(ms, T, futr.alloc_bytes(futr.futr_moe_workspace_size(ms, T)))
        st |= {"blob": blob, "ws": ws, "y": torch.empty((T, H), dtype=torch.bfloat16, device="cuda"),
               "ids": torch.empty((T, case["top_k"]), dtype=torch.int32, device="cuda"),
               "weights": torch.empty((T, case["top_k"]), dtype=torch.float32, device="cuda")}
    else:
        st |= _moe_codes(case, g, st["gain"])
    return st


def _moe_codes(case, g, gain):
    E, H, I = (case[k] for k in ("experts", "hidden", "inter"))
    p = {}
    for n, (r, c) in {"gate": (I, H), "up": (I, H), "down": (H, I)}.items():
        p[n] = (torch.empty((E, r, c), dtype=torch.int8, device="cuda"),
                torch.empty((E, r, c // 128), dtype=torch.float16, device="cuda"))
    for e, w in _experts(case, g):
        for n, x in zip(("gate", "up", "down"), w):
            p[n][0][e], p[n][1][e] = _quantized(x, gain if n != "down" else None)
    return {"experts": p}


# ------------------------------------------------------------------ plain --

def _rotated(x, where, d):
    """x [rows, heads, d] in fp32, dims i and i + d/2 turned by where * THETA^(-2i/d)."""
    i = torch.arange(d // 2, dtype=torch.float64, device=x.device)
    a = where.double()[:, None] * torch.pow(THETA, -2.0 * i / d)
    c, s = torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]
    x1, x2 = x[..., :d // 2], x[..., d // 2:]
    return torch.cat([x1 * c - x2 * s, x2 * c + x1 * s], -1)


def _append_plain(st):
    case, codes, scales = st["case"], st["codes"], st["scales"]
    page, d, Hkv = case["page"], case["d"], case["kv_heads"]
    x = torch.stack([_rotated(st["k"].float(), st["where"], d), st["v"].float()], 2)      # [rows, Hkv, 2, d]
    at = st["table"][st["seq"], st["where"] // page].long()
    slot = st["where"] % page
    touched = torch.zeros(codes.shape[0], device=x.device).index_fill_(0, at, 1.0)
    fresh = torch.zeros(codes.shape[0], device=x.device).index_fill_(0, at[slot == 0], 1.0)
    amax = torch.zeros_like(scales).scatter_reduce_(0, at[:, None, None].expand(-1, Hkv, 2), x.abs().amax(-1), "amax")
    old = torch.where(fresh[:, None, None] > 0, torch.zeros_like(scales), scales)
    s = torch.where(touched[:, None, None] > 0, torch.maximum(old, _page_scale(amax)), scales)
    # a page that goes on and whose scale grows: its codes at the new scale
    ratio = torch.where((old > 0) & (s > old), old / s, torch.ones_like(s))
    pages = torch.unique(at)
    codes[pages] = (codes[pages].float() * ratio[pages][..., None, None]).to(torch.float8_e4m3fn)
    codes[at, :, :, slot] = (x / s[at][..., None]).to(torch.float8_e4m3fn)
    scales.copy_(s)
    return codes, scales


def _attention_plain(st):
    case = st["case"]
    B, Hq, Hkv, d, n, L = case["batch"], case["heads"], case["kv_heads"], case["d"], st["most"], st["longest"]
    G = Hq // Hkv
    tab = st["table"].long().clamp(min=0)
    kv = st["codes"][tab].float() * st["scales"][tab][..., None, None]     # [B, width, Hkv, 2, page, d]
    kv = kv.permute(0, 2, 3, 1, 4, 5).reshape(B, Hkv, 2, -1, d)[:, :, :, :L]
    q = _rotated(st["q"].float(), st["where"], d)
    row = torch.arange(q.shape[0], device=q.device) - st["start"].long()[st["seq"]]
    qp = torch.zeros((B, n, Hq, d), device=q.device)
    qp[st["seq"], row] = q
    qp = qp.view(B, n, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, d)
    s = torch.matmul(qp, kv[:, :, 0].transpose(-1, -2)) * (d ** -0.5)
    key = torch.arange(L, device=q.device)
    p = st["pos"].long()[:, None] + torch.arange(n, device=q.device)
    see = key <= p[..., None]
    if case["window"]:
        see = see & (key > p[..., None] - case["window"])
    see = see[:, None, :, None].expand(B, 1, n, G, L).reshape(B, 1, n * G, L)
    s = torch.where(see, s, torch.full_like(s, -math.inf))
    w = torch.exp(s - s.amax(-1, keepdim=True))
    o = torch.matmul(w, kv[:, :, 1]) / w.sum(-1, keepdim=True)
    o = o.view(B, Hkv, n, G, d).permute(0, 2, 1, 3, 4).reshape(B, n, Hq, d)
    st["out"].copy_(o[st["seq"], row])
    return st["out"]


def _dequantized(w, at=None):
    c, s = (t if at is None else t[at] for t in w)
    return (c.float().view(*s.shape, 128) * s.float()[..., None]).view(c.shape)


def _moe_plain(st):
    case, p, x = st["case"], st["experts"], st["x"].float()
    T, E, K = case["tokens"], case["experts"], case["top_k"]
    r = torch.rsqrt((x.double() ** 2).mean(-1, keepdim=True) + EPS) if case["norm"] else torch.ones((T, 1), device=x.device)
    xg = x * st["gain"] if case["norm"] else x
    logits = (r.double() * torch.matmul(xg.double(), st["router"].double().t())).float()
    prob = torch.exp(logits - logits.amax(-1, keepdim=True))
    prob = prob / prob.sum(-1, keepdim=True)
    # the K largest, equal ones by the lowest index
    ids = torch.sort(logits, dim=-1, descending=True, stable=True).indices[:, :K]
    w = prob.gather(1, ids)
    if case["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    r = r.float()
    if T * K <= E:  # few experts: each token's own
        at = ids.reshape(-1)
        xe = x.repeat_interleave(K, 0)[..., None]
        re = r.repeat_interleave(K, 0)
        g = torch.matmul(_dequantized(p["gate"], at), xe)[..., 0] * re
        u = torch.matmul(_dequantized(p["up"], at), xe)[..., 0] * re
        a = g / (1.0 + torch.exp(-g)) * u
        o = torch.matmul(_dequantized(p["down"], at), a[..., None])[..., 0].view(T, K, -1)
        y = (o * w[..., None]).sum(1)
    else:           # most experts: all of them
        xt = x.t().expand(E, -1, -1)
        g = torch.matmul(_dequantized(p["gate"]), xt) * r[:, 0]
        u = torch.matmul(_dequantized(p["up"]), xt) * r[:, 0]
        a = g / (1.0 + torch.exp(-g)) * u
        dense = torch.zeros((T, E), device=x.device).scatter_(1, ids, w)
        y = (torch.matmul(_dequantized(p["down"]), a) * dense.t()[:, None]).sum(0).t()
    if case["resid"]:
        y = y + st["resid"].float()
    return {"y": y.to(torch.bfloat16), "ids": ids.to(torch.int32), "weights": w}


def run(st):
    case = st["case"]
    if case["op"] == "append":
        if own:
            from int4_weight_kv_w4a16_gb300 import futr
            futr.futr_paged_append(st["cache"], 0, case["batch"], st["pos"], st["start"], st["table"], st["k"], st["v"])
            return st["codes"], st["scales"]
        return _append_plain(st)
    if case["op"] == "attention":
        if own:
            from int4_weight_kv_w4a16_gb300 import futr
            futr.futr_paged_attention(st["cache"], 0, case["batch"], st["pos"], st["start"], st["table"], st["q"],
                                      st["out"], st["ws"], window=case["window"])
            return st["out"]
        return _attention_plain(st)
    if own:
        from int4_weight_kv_w4a16_gb300 import futr
        futr.futr_moe_layer(st["x"], st["gain"], st["router"], st["blob"], st["resid"], st["y"], st["ws"],
                            ids=st["ids"], weights=st["weights"])
        return {"y": st["y"], "ids": st["ids"], "weights": st["weights"]}
    return _moe_plain(st)


# ------------------------------------------------------------------ exact --

def _turned(x, p):
    """One row's heads [heads, d] in 64 bits as complex numbers, turned by position p."""
    d = x.shape[-1]
    f = THETA ** (-torch.arange(0, d, 2, dtype=torch.float64, device=x.device) / d)
    z = torch.complex(x[..., :d // 2], x[..., d // 2:]) * torch.polar(torch.ones_like(f), p * f)
    return torch.cat([z.real, z.imag], -1)


def _on_grid(v):
    """64-bit values rounded to e4m3's: steps of 2^(e-3) in [2^e, 2^(e+1)), of 2^-9 below 2^-6, at most 448."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _append_exact(case, st):
    page = case["page"]
    codes, scales = st["codes"].double(), st["scales"].double()
    table, seq, where = st["table"].tolist(), st["seq"].tolist(), st["where"].tolist()
    rows = {}
    for i, (b, p) in enumerate(zip(seq, where)):
        rows.setdefault(table[b][p // page], []).append((i, p))
    k = torch.stack([_turned(x, p) for x, p in zip(st["k"].double(), where)]) if len(where) <= 64 else None
    if k is None:
        d = case["d"]
        f = THETA ** (-torch.arange(0, d, 2, dtype=torch.float64, device="cuda") / d)
        a = st["where"].double()[:, None] * f
        z = torch.complex(st["k"].double()[..., :d // 2], st["k"].double()[..., d // 2:])
        z = z * torch.polar(torch.ones_like(a), a)[:, None]
        k = torch.cat([z.real, z.imag], -1)
    kv = torch.stack([k, st["v"].double()], 2)
    for at, r in rows.items():
        i, slot = [x[0] for x in r], [x[1] % page for x in r]
        x = kv[i]
        need = torch.exp2(torch.ceil(torch.log2(x.abs().amax((0, 3)).clamp(min=1e-300) / E4M3_MAX))).clamp(min=2.0 ** MIN_EXP)
        was = torch.zeros_like(need) if 0 in slot else scales[at]
        s = torch.maximum(was, need)
        grow = torch.where((was > 0) & (s > was), was / s, torch.ones_like(s))
        codes[at] = _on_grid(codes[at] * grow[..., None, None])
        codes[at, :, :, slot] = _on_grid(x / s[..., None]).permute(1, 2, 0, 3)
        scales[at] = s
    return codes, scales


def _attention_exact(case, st):
    page, d, G = case["page"], case["d"], case["heads"] // case["kv_heads"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    past, new = _lens(case)
    r = 0
    for b in range(case["batch"]):
        n, L = new[b], past[b] + new[b]
        if n:
            tab = st["table"][b, :-(-L // page)].long()
            kv = (st["codes"][tab].double() * st["scales"][tab].double()[..., None, None])
            K = kv[:, :, 0].transpose(0, 1).reshape(case["kv_heads"], -1, d)[:, :L].repeat_interleave(G, 0)
            V = kv[:, :, 1].transpose(0, 1).reshape(case["kv_heads"], -1, d)[:, :L].repeat_interleave(G, 0)
            q = torch.stack([_turned(st["q"][r + i].double(), past[b] + i) for i in range(n)], 1)   # [Hq, n, d]
            s = q @ K.transpose(1, 2) / math.sqrt(d)
            ages = (past[b] + torch.arange(n, device="cuda"))[:, None] - torch.arange(L, device="cuda")
            hidden = (ages < 0) | (ages >= case["window"] if case["window"] else ages < 0)
            s[:, hidden] = -math.inf
            out[r:r + n] = (torch.softmax(s, -1) @ V).transpose(0, 1)
        r += n
    return out


def _moe_exact(case, g, st):
    p = _moe_codes(case, g, st["gain"])["experts"]
    T, K = case["tokens"], case["top_k"]
    x = st["x"].double()
    if case["norm"]:
        x = x / torch.sqrt((x * x).sum(1, keepdim=True) / case["hidden"] + EPS)
    h = x * st["gain"].double() if case["norm"] else x
    logits = h @ st["router"].double().t()
    prob = torch.softmax(logits, -1)
    ids = torch.argsort(-logits, dim=-1, stable=True)[:, :K]
    w = prob.gather(1, ids)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    y = st["resid"].double() if case["resid"] else torch.zeros_like(x)
    y = y.clone()

    def full(n, e):
        c, s = p[n][0][e], p[n][1][e]
        return c.double() * s.double().repeat_interleave(128, 1)

    for e in sorted(set(ids.reshape(-1).tolist())):
        t, slot = (ids == e).nonzero(as_tuple=True)
        gate, up = x[t] @ full("gate", e).t(), x[t] @ full("up", e).t()
        y[t] += w[t, slot][:, None] * ((gate * torch.sigmoid(gate) * up) @ full("down", e).t())
    return {"y": y, "ids": ids.to(torch.int32), "weights": w}


def exact(case, seed):
    if case["op"] == "moe":
        g, st = _moe_inputs(case, seed)
        return _moe_exact(case, g, st)
    st = _kv_inputs(case, seed)
    return _append_exact(case, st) if case["op"] == "append" else _attention_exact(case, st)
