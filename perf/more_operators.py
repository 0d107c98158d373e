"""Workloads of generation with several continuations over the caches, and their plain forms.

Six operators, as a server uses them between the steps of a model:

* ``select``: the best continuations of each prompt's beams over the vocabulary: log-softmax of the step's logits, the
  beams' scores added, the ``keep`` largest sums of a prompt's beams, equal ones by the lowest (beam, token).
* ``reorder``: the slots of the INT4 cache follow the chosen beams, in place: slot i continues slot parent[i].
* ``fork``: the sequences of a paged cache do. Full pages are shared and counted, a page that is partly written is
  copied for every child but the first, pages that nobody holds any more are free again.
* ``turn``: between two steps of a served batch: pages that no later row sees (behind the window, of sequences that
  ended, of drafts that were refused) are given back, and the pages of the next rows are taken.
* ``compact``: the pages in use of one half of a pool move to the other half, and back.
* ``sinks``: causal grouped-query attention over the paged e4m3 cache with a window and the first tokens of a sequence,
  which every row sees; the pages in between have been given back.

With ``own`` false, ``run`` computes them in elementary torch operations (32 bits; sums of exponentials, scores and
angles in 64); with ``own`` true it calls the framework.
"""
import math

import torch

own = False

THETA = 500000.0
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------- cases --

def _named(name, **c):
    return dict(c, name=name) if name else c


def _select(name, batch, beams, keep, vocab, dtype, first=False, done=0, pad=0):
    return _named(name, op="select", batch=batch, beams=beams, keep=keep, vocab=vocab, dtype=dtype, first=first, done=done,
                  pad=pad)


def _reorder(name, groups, beams, drop, shuffle, layers, kv_heads, d, capacity, lo, hi):
    return _named(name, op="reorder", groups=groups, beams=beams, drop=drop, shuffle=shuffle, layers=layers,
                  kv_heads=kv_heads, d=d, capacity=capacity, lo=lo, hi=hi)


def _fork(name, groups, beams, drop, shuffle, layers, kv_heads, d, page, lo, hi):
    return _named(name, op="fork", groups=groups, beams=beams, drop=drop, shuffle=shuffle, layers=layers,
                  kv_heads=kv_heads, d=d, page=page, lo=lo, hi=hi)


def _turn(name, batch, page, lo, hi, new, leave, window, sinks):
    return _named(name, op="turn", batch=batch, page=page, lo=lo, hi=hi, new=new, leave=leave, window=window, sinks=sinks)


def _compact(name, batch, pages, shared, layers, kv_heads, d, page):
    return _named(name, op="compact", batch=batch, pages=pages, shared=shared, layers=layers, kv_heads=kv_heads, d=d,
                  page=page)


def _sinks(name, batch, lo, hi, new, heads, kv_heads, d, page, dtype, window, sinks, fused=False):
    return _named(name, op="sinks", batch=batch, lo=lo, hi=hi, new=new, heads=heads, kv_heads=kv_heads, d=d, page=page,
                  dtype=dtype, window=window, sinks=sinks, fused=fused)


def listed():
    return [
        # one prompt with four beams after the 8B model's complete step: what a choice costs at the least
        _select("select_b1_w4", 1, 4, 4, 128256, "f32"),
        # 32 prompts of eight beams, twice as many candidates as beams, as a search that sets finished ones aside asks
        _select("select_b32_w8", 32, 8, 16, 128256, "f32"),
        # four beams of one prompt, of which one was dropped, the 8B model's 32 layers
        _reorder("reorder_b1_w4", 1, 4, 1, False, 32, 8, 128, 1024, 900, 900),
        # the largest batch: four prompts of eight beams in the order of their scores, so that every slot moves
        _reorder("reorder_b4_w8", 4, 8, 3, True, 16, 8, 128, 2048, 500, 2000),
        # one prompt's four beams in pages, one dropped
        _fork("fork_b1_w4", 1, 4, 1, False, 32, 8, 128, 64, 1000, 1000),
        # 32 prompts of four beams each, every slot with another parent
        _fork("fork_b32_w4", 32, 4, 2, True, 8, 8, 128, 128, 200, 1000),
        # eight users, one token each: page numbers only
        _turn("turn_b8", 8, 16, 100, 2000, 1, 0, 0, 0),
        # a large served batch with a window and sinks, some sequences replaced by new prompts
        _turn("turn_b256", 256, 16, 1000, 16000, 700, 32, 4096, 64),
        # a small pool changes halves
        _compact("compact_64", 8, 64, 8, 4, 8, 128, 16),
        # a pool of 500 pages of four layers (262 MB) changes halves
        _compact("compact_500", 32, 500, 60, 4, 8, 128, 64),
        # long answers of 16 users in a window of 4096 with four sinks, one token each
        _sinks("sinks_b16", 16, 3000, 20000, 1, 32, 8, 128, 64, "bf16", 4096, 4, fused=True),
        # prompts' chunks behind long texts, a window of 1000, sinks that end inside a page
        _sinks("sinks_chunk", 4, 2000, 8000, 511, 32, 8, 128, 32, "f16", 1000, 100),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_select(rng):
    beams = rng.choice([1, 2, 3, 4, 5, 8, 12, 16, 32])
    keep = rng.choice([beams, beams, min(64, 2 * beams), _log(rng, 1, 64)])
    vocab = max(keep, rng.choice([128256, 32000, 50257, 151936, _log(rng, 100, 200000)]))
    batch = _log(rng, 1, max(1, min(256, (256 * 128256) // (beams * vocab))))
    return _select(None, batch, beams, keep, vocab, rng.choice(["f32", "f32", "bf16", "f16"]), rng.random() < 0.1,
                   rng.choice([0, 0, min(1, beams - 1), beams // 2]), rng.choice([0, 0, _log(rng, 1, 300)]))


def _draw_beams(rng):
    beams = rng.choice([2, 3, 4, 5, 8, 16])
    return beams, rng.randint(0, beams // 2), rng.random() < 0.4


def draw(rng):
    op = rng.choice(["select", "reorder", "fork", "turn", "compact", "sinks", "select", "sinks"])
    if op == "select":
        return _draw_select(rng)
    kv_heads, d, page = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128])
    if op == "reorder":
        beams, drop, shuffle = _draw_beams(rng)
        groups, capacity = rng.randint(1, 32 // beams), _log(rng, 60, 2000)
        layers = _log(rng, 1, max(1, min(40, (16 * 32 * 8 * 2048 * 128) // (groups * beams * kv_heads * capacity * d))))
        hi = _log(rng, 20, capacity)
        return _reorder(None, groups, beams, drop, shuffle, layers, kv_heads, d, capacity, rng.randint(0, hi), hi)
    if op == "fork":
        beams, drop, shuffle = _draw_beams(rng)
        groups, hi = _log(rng, 1, 128 // beams), _log(rng, 10, 4000)
        pages = groups * (hi // page + 3 * beams)
        layers = _log(rng, 1, max(1, min(32, (8 << 30) // 16 // (pages * kv_heads * 2 * page * d))))
        return _fork(None, groups, beams, drop, shuffle, layers, kv_heads, d, page, rng.randint(0, hi), hi)
    if op == "turn":
        batch, hi = _log(rng, 1, 300), _log(rng, 20, 16000)
        window = rng.choice([0, 0, _log(rng, 10, 5000)])
        return _turn(None, batch, page, rng.randint(0, hi), hi, _log(rng, 1, 1000), rng.randint(0, batch // 4), window,
                     rng.choice([0, 4, 100]) if window else 0)
    if op == "compact":
        batch, pages = _log(rng, 1, 64), _log(rng, 8, 2000)
        layers = _log(rng, 1, max(1, min(32, (500 * 4 * 8 * 64 * 128) // (pages * kv_heads * page * d))))
        return _compact(None, batch, pages, rng.randint(0, pages // 4), layers, kv_heads, d, page)
    heads = kv_heads * rng.choice([1, 2, 4, 4, 5, 8, 16])
    if heads * d % 128:                             # a model's width is a multiple of 128
        kv_heads, heads = 2 * kv_heads, 2 * heads
    if rng.random() < 0.3:                          # chunks
        batch, new, hi = _log(rng, 1, 4), _log(rng, 9, 300), _log(rng, 100, 8000)
    else:                                           # decoding, drafted tokens
        batch, new, hi = _log(rng, 1, 32), rng.choice([1, 1, 2, 3, 8]), _log(rng, 100, 16000)
        hi = min(hi, max(100, (1 << 19) // (batch * kv_heads)))
    return _sinks(None, batch, rng.choice([hi, int(hi * rng.random())]), hi, new, heads, kv_heads, d, page,
                  rng.choice(["bf16", "f16"]), _log(rng, 17, 4000), rng.choice([1, 4, 16, _log(rng, 1, 600)]),
                  rng.random() < 0.5)


def _spread(case, b):
    """A length of the case's range: spread over it, fixed by the case."""
    return case["lo"] + int(round((case["hi"] - case["lo"]) * ((0.5 + 0.6180339887498949 * b) % 1.0)))


def _lens(case):
    """Cached tokens and new rows of each sequence."""
    past, new = [], []
    for b in range(case["batch"]):
        past.append(_spread(case, b))
        new.append(case["new"] if b == case["batch"] - 1 else
                   1 + int((case["new"] - 1) * ((0.5 + 0.6180339887498949 * b) % 1.0)))
    return past, new


def _moves(case):
    """Distinct parents that are read and slots that are written, of a group."""
    left, drop = case["beams"] - case["drop"], case["drop"]
    if case["shuffle"]:
        return (left, case["beams"]) if left > 1 else (1, drop)
    return min(left, drop), drop


def work(case):
    op = case["op"]
    if op == "select":
        rows = case["batch"] * (1 if case["first"] else case["beams"] - case["done"])
        n = rows * case["vocab"]
        return {"bytes": n * (4 if case["dtype"] == "f32" else 2) + case["batch"] * (case["keep"] * 12 + case["beams"] * 8),
                "flops": 4.0 * n}
    if op == "reorder":
        read, written = _moves(case)
        tiles = sum(-(-_spread(case, g) // 16) for g in range(case["groups"]))
        return {"bytes": tiles * 16 * (case["d"] + 4) * case["kv_heads"] * case["layers"] * (read + written) +
                case["groups"] * case["beams"] * 12, "flops": 0}
    if op == "fork":
        _, copies = _moves(dict(case, shuffle=False))
        slots = sum(_spread(case, g) % case["page"] for g in range(case["groups"])) * copies
        reads = sum(_spread(case, g) % case["page"] for g in range(case["groups"])) * min(copies, case["beams"] - case["drop"])
        row = case["layers"] * case["kv_heads"] * 2 * case["d"]
        table = sum(_spread(case, g) // case["page"] + 1 for g in range(case["groups"])) * case["beams"] * 8
        return {"bytes": (slots + reads) * row + table, "flops": 0}
    if op == "turn":
        past, new = _lens(case)
        return {"bytes": sum(-(-(p + n) // case["page"]) for p, n in zip(past, new)) * 8 + case["batch"] * 8, "flops": 0}
    if op == "compact":
        return {"bytes": case["pages"] * case["layers"] * case["kv_heads"] * 2 * (case["page"] * case["d"] + 4) * 4.0 +
                case["pages"] * 16, "flops": 0}
    past, new = _lens(case)
    w, s = case["window"], case["sinks"]
    pairs = sum(min(p + i + 1, w) + min(s, max(0, p + i + 1 - w)) for p, n in zip(past, new) for i in range(n))
    keys = sum(min(p + n, w + n - 1) + min(s, max(0, p + 1 - w)) for p, n in zip(past, new))
    return {"bytes": keys * case["kv_heads"] * 2 * (case["d"] + 4 / case["page"]) + sum(new) * case["heads"] * case["d"] * 4,
            "flops": 4.0 * pairs * case["heads"] * case["d"]}


# ------------------------------------------------------------------ inputs --

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(1000003 * (int(seed) + 1))


def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _select_inputs(case, g):
    R, V = case["batch"] * case["beams"], case["vocab"]
    x = torch.randn((R, V + case["pad"]), generator=g, device="cuda") * 2.0
    # a few tokens of each row stand out, as a model's do
    at = torch.randint(0, V, (R, 12), generator=g, device="cuda")
    x.scatter_add_(1, at, torch.rand((R, 12), generator=g, device="cuda") * 8.0 + 4.0)
    scores = -30.0 * torch.rand((case["batch"], case["beams"]), generator=g, device="cuda")
    done = torch.zeros((case["batch"], case["beams"]), dtype=torch.int32, device="cuda")
    if case["first"]:
        scores[:, 0], scores[:, 1:] = 0.0, -math.inf
    else:
        done[:, :case["done"]] = 1
    return {"logits": x.to(DTYPES[case["dtype"]])[:, :V], "scores": scores, "done": done}


def _parents(case, g):
    """Parents of the slots: of each group `drop` beams end, and others go on twice (shuffle: none in its own slot)."""
    G, W, left = case["groups"], case["beams"], case["beams"] - case["drop"]
    order = torch.argsort(torch.rand((G, W), generator=g, device="cuda"), dim=1)
    j = torch.arange(W, device="cuda")
    of = (j + 1) % left if case["shuffle"] else torch.where(j < left, j, (j - left) % left)
    parent = torch.empty_like(order).scatter_(1, order, order[:, of])
    return (parent + W * torch.arange(G, device="cuda")[:, None]).reshape(-1).to(torch.int32)


def _reorder_inputs(case, g):
    slots, C = case["groups"] * case["beams"], -(-case["capacity"] // 16) * 16
    shape = (case["layers"], slots, case["kv_heads"], C * (case["d"] + 4))
    streams = torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8)
    return {"streams": streams, "parent": _parents(case, g),
            "pos": _int32([_spread(case, i // case["beams"]) for i in range(slots)])}


def _pool_inputs(case, g, n_pages):
    """Codes and scales of a pool: normal values at scales of their own."""
    lead = (case.get("layers", 1), n_pages, case["kv_heads"], 2)
    codes = (torch.randn(lead + (case["page"], case["d"]), generator=g, device="cuda") * 60.0).to(torch.float8_e4m3fn)
    scales = torch.ldexp(torch.ones(lead, device="cuda"), torch.randint(-9, -3, lead, generator=g, device="cuda"))
    return {"codes": codes, "scales": scales}


def _table_inputs(g, width, rows, spare):
    """Page numbers, shuffled, for rows of places in use (-1: none, equal numbers: one page), and how often each is held."""
    local = torch.full((len(rows), width), -1, dtype=torch.int64)
    for b, r in enumerate(rows):
        local[b, :len(r)] = torch.tensor(r, dtype=torch.int64)
    used = int(local.max()) + 1
    perm = torch.randperm(used + spare, generator=g, device="cuda")
    table = torch.where(local.cuda() >= 0, perm[local.cuda().clamp(min=0)], -1).to(torch.int32)
    return {"table": table, "n_pages": used + spare, "refs": _held(table, used + spare)}


def _fork_inputs(case, g):
    W, page = case["beams"], case["page"]
    rows, n = [], 0
    for grp in range(case["groups"]):
        full, part = divmod(_spread(case, grp), page)
        shared = list(range(n, n + max(0, full - 1)))
        n += len(shared)
        for _ in range(W):   # the last full page and the one being written are a beam's own
            mine = list(range(n, n + min(full, 1) + (part > 0)))
            n += len(mine)
            rows.append(shared + mine)
    st = _table_inputs(g, max(len(r) for r in rows) + 3, rows, case["groups"] * W + 5)
    return st | {"parent": _parents(case, g), "pos": _int32([_spread(case, i // W) for i in range(len(rows))])}


def _turn_inputs(case, g):
    past, new = _lens(case)
    page, w = case["page"], case["window"]
    rows, n, late = [], 0, 3 * page
    for b, p in enumerate(past):   # what a window left behind is gone, but for the last few pages
        seen = max(0, p - late - w + 1) // page if w else 0
        r = [-1 if -(-case["sinks"] // page) <= i < seen else n + i for i in range(-(-p // page))]
        n += len(r)
        rows.append(r)
    keep = [x for r in rows for x in r if x >= 0]
    number = {x: i for i, x in enumerate(keep)}
    rows = [[number.get(x, -1) for x in r] for r in rows]
    out = [case["leave"] > b for b in range(case["batch"])]
    more = sum(-(-(m + page) // page) for m in new)
    width = max(-(-(p + m) // page) for p, m in zip(past, new)) + 2
    st = _table_inputs(g, width, rows, more + 4)
    # a sequence that ended is followed by a prompt; the others take a token or a few
    rows_of = [m if o else 1 + m % 8 for m, o in zip(new, out)]
    starts = [sum(rows_of[:b]) for b in range(case["batch"] + 1)]
    return st | {"pos": _int32([0 if o else p for p, o in zip(past, out)]), "start": _int32(starts)}


def _compact_inputs(case, g):
    per = -(-case["pages"] // case["batch"])
    rows = [list(range(min(case["pages"], b * per), min(case["pages"], (b + 1) * per))) for b in range(case["batch"])]
    # the first sequence's first pages are the others' prefix, too
    rows = [list(range(max(0, min(case["shared"] - b, per)) if b else 0)) + r for b, r in enumerate(rows)]
    return _table_inputs(g, max(len(r) for r in rows), rows, case["pages"] + 6)


def _sinks_inputs(case, g):
    past, new = _lens(case)
    Hq, Hkv, d, page, w = (case[k] for k in ("heads", "kv_heads", "d", "page", "window"))
    rows, n = [], 0
    for p, m in zip(past, new):
        seen = max(0, p - w + 1) // page
        live = [i for i in range(-(-(p + m) // page)) if i * page < case["sinks"] or i >= seen]
        at = {i: n + k for k, i in enumerate(live)}
        n += len(live)
        rows.append([at.get(i, -1) for i in range(live[-1] + 1)])
    st = _table_inputs(g, max(len(r) for r in rows), rows, 3)
    # keys with four channels of each head 20 times as large, as the models' are
    gain = torch.ones((Hkv, 2, 1, d), device="cuda")
    gain[:, 0, :, torch.randperm(d, generator=g, device="cuda")[:4]] = 20.0
    x = torch.randn((st["n_pages"], Hkv, 2, page, d), generator=g, device="cuda") * gain
    m, e = torch.frexp(x.abs().amax((3, 4)))
    s = torch.ldexp(torch.ones_like(m), torch.where(m <= 0.875, e - 9, e - 8))
    qkv = torch.randn((sum(new), Hq + 2 * Hkv, d), generator=g, device="cuda").to(DTYPES[case["dtype"]])
    q = qkv[:, :Hq] if case["fused"] else qkv[:, :Hq].contiguous()
    return st | {"codes": (x / s[..., None, None]).to(torch.float8_e4m3fn)[None], "scales": s[None], "q": q,
                 "pos": _int32(past), "start": _int32([sum(new[:b]) for b in range(len(new) + 1)]),
                 "seq": torch.tensor([b for b, m in enumerate(new) for _ in range(m)], device="cuda"),
                 "where": torch.tensor([p + i for p, m in zip(past, new) for i in range(m)], device="cuda"),
                 "longest": max(p + m for p, m in zip(past, new)), "most": max(new)}


def _inputs(case, seed):
    g, op = _generator(seed), case["op"]
    st = {"select": _select_inputs, "reorder": _reorder_inputs, "fork": _fork_inputs, "turn": _turn_inputs,
          "compact": _compact_inputs, "sinks": _sinks_inputs}[op](case, g)
    if op in ("fork", "compact"):
        st |= _pool_inputs(case, g, st["n_pages"])
    return st | {"case": case}


def prepare(case, seed):
    st, op = _inputs(case, seed), case["op"]
    if op == "select":
        shape, i32 = (case["batch"], case["keep"]), torch.int32
        st["out"] = [torch.empty(shape, dtype=t, device="cuda") for t in (torch.float32, i32, i32, i32)]
    if op == "sinks":
        st["out"] = torch.empty(st["q"].shape, dtype=st["q"].dtype, device="cuda")
    if own:   # the framework's handles, with the same contents
        from int4_weight_kv_w4a16_gb300 import futr, inputs
        if op == "select":
            n = (case["batch"] * case["beams"], case["keep"])
            st["ws"] = futr.futr_beam_workspace_init(*n, futr.alloc_bytes(futr.futr_beam_workspace_size(*n)))
            return st
        kv_heads, d = case.get("kv_heads", 1), case.get("d", 128)
        sh = futr.make_shape(inputs.BlockShape(hidden=128, n_q_heads=case.get("heads", 2 * kv_heads), n_kv_heads=kv_heads,
                                               head_dim=d, inter=128, had_block=d, rope_theta=THETA))
        if op == "reorder":
            size = (case["layers"], case["groups"] * case["beams"], case["capacity"])
            st["kv"] = futr.futr_kv_init(sh, *size, futr.alloc_bytes(futr.futr_kv_size(sh, *size)))
            view = st["kv"]._mem[:st["streams"].numel()].view(st["streams"].shape)
            view.copy_(st["streams"])
            st["streams"] = view
            return st
        size = (case.get("layers", 1), st["n_pages"], case["page"], st["table"].shape[1] * case["page"])
        st["cache"] = futr.futr_paged_init(sh, *size, True, futr.alloc_bytes(futr.futr_paged_size(sh, *size)))
        codes, scales = futr.paged_views(st["cache"])
        if "codes" in st:
            codes.copy_(st["codes"])
            scales.copy_(st["scales"])
            st |= {"codes": codes, "scales": scales}
        if op == "sinks":
            st["ws"] = futr.futr_paged_workspace_init(sh, futr.alloc_bytes(futr.futr_paged_workspace_size(sh)))
        else:
            rows = st["table"].shape[0]
            size = futr.futr_pages_size(st["n_pages"], rows)
            st["pool"] = futr.futr_pages_init(st["n_pages"], rows, futr.alloc_bytes(size))
            futr.futr_pages_hold(st["cache"], st["pool"], st["table"])
            st["refs"] = futr.pages_refs(st["pool"])
    return st


# ------------------------------------------------------------------- plain --

def _held(table, n_pages):
    """How many places of the table name each page."""
    flat = table.reshape(-1).long()
    n = torch.zeros(n_pages + 1, dtype=torch.int32, device=table.device)
    n.index_add_(0, torch.where(flat >= 0, flat, n_pages), torch.ones_like(flat, dtype=torch.int32))
    return n[:n_pages]


def _taken(table, need, refs):
    """The table with the lowest free pages in the places that need one, in order."""
    free = torch.sort((refs > 0).to(torch.int32), stable=True).indices
    k = (torch.cumsum(need.reshape(-1).to(torch.int64), 0) - 1).clamp(min=0).view(need.shape)
    return torch.where(need, free[k.clamp(max=free.numel() - 1)].to(torch.int32), table)


def _select_plain(st):
    case, x = st["case"], st["logits"].double().view(st["case"]["batch"], st["case"]["beams"], -1)
    V, end = case["vocab"], case["vocab"] - 1
    m = x.amax(-1, keepdim=True)
    lse = m + torch.log(torch.exp(x - m).sum(-1, keepdim=True))
    value = x - lse
    only = torch.arange(V, device=x.device) == end
    value = torch.where(st["done"][..., None] > 0, torch.where(only, 0.0, -math.inf).to(value.dtype), value)
    value = (value + st["scores"].double()[..., None]).view(case["batch"], -1)
    best = torch.sort(value, dim=1, descending=True, stable=True)
    v, at = best.values[:, :case["keep"]], best.indices[:, :case["keep"]]
    row = torch.arange(case["batch"], device=x.device)[:, None] * case["beams"]
    token = at % V
    return [v.float(), (row + at // V).to(torch.int32), token.to(torch.int32), (token == end).to(torch.int32)]


def _reorder_plain(st):
    case, x = st["case"], st["streams"]
    parent = st["parent"].long()
    pos = st["pos"][parent]
    d, C = case["d"], x.shape[-1] // (case["d"] + 4)
    # byte i of a stream belongs to a tile of 16 positions: codes of keys, then of values, then their scales
    i = torch.arange(x.shape[-1], device=x.device)
    code, scale = i % (C * d // 2) // (8 * d), (i - C * d).clamp(min=0) % (2 * C) // 32
    tile = torch.where(i < C * d, code, scale)
    moved = tile < ((pos + 15) // 16)[:, None]                                  # [slots, bytes]
    x.copy_(torch.where(moved[None, :, None], x[:, parent], x))
    st["pos"].copy_(pos)
    return x, st["pos"]


def _fork_plain(st):
    case, table, codes, scales = st["case"], st["table"], st["codes"], st["scales"]
    page, parent, n = case["page"], st["parent"].long(), st["table"].shape[0]
    pos = st["pos"][parent]
    col = (pos // page).long()
    src = table[parent, col.clamp(max=table.shape[1] - 1)]
    me = torch.arange(n, device=table.device)
    first = torch.full((n,), n, device=table.device).scatter_reduce_(0, parent, me, "amin")
    need = (pos % page > 0) & (src >= 0) & (first[parent] != me)
    dst = _taken(src, need, st["refs"]).long()
    new = table[parent]
    new[me, col.clamp(max=table.shape[1] - 1)] = torch.where(need, dst.to(torch.int32), new[me, col.clamp(max=table.shape[1] - 1)])
    # (a sequence that needs no copy copies its page onto itself)
    to, at = dst.clamp(min=0), src.long().clamp(min=0)
    raw = codes.view(torch.uint8)
    written = torch.arange(page, device=table.device) < (pos % page)[:, None]
    raw[:, to] = torch.where(written[None, :, None, None, :, None], raw[:, at], raw[:, to])
    scales[:, to] = torch.where(need[None, :, None, None], scales[:, at], scales[:, to])
    table.copy_(new)
    st["pos"].copy_(pos)
    st["refs"].copy_(_held(table, st["n_pages"]))
    return table, st["refs"], st["pos"], codes, scales


def _turn_plain(st):
    case, table, page = st["case"], st["table"], st["case"]["page"]
    p, i = st["pos"].long()[:, None], torch.arange(table.shape[1], device=table.device)
    keep = i * page < p
    if case["window"]:
        keep = keep & ((i * page < case["sinks"]) | ((i + 1) * page > p - case["window"] + 1))
    table.copy_(torch.where(keep, table, -1))
    refs = _held(table, st["n_pages"])
    rows = (st["start"][1:] - st["start"][:-1]).long()[:, None]
    need = ((i + 1) * page > p) & (i * page < p + rows) & (table < 0)
    table.copy_(_taken(table, need, refs))
    st["refs"].copy_(_held(table, st["n_pages"]))
    return table, st["refs"]


def _moved_plain(st, lo, hi):
    """The pages in use of [lo, hi) move to the lowest free pages outside of it."""
    table, refs, n = st["table"], st["refs"], st["n_pages"]
    i = torch.arange(n, device=table.device)
    inside = (i >= lo) & (i < hi)
    move, room = (refs > 0) & inside, (refs == 0) & ~inside
    srcs = torch.sort((~move).to(torch.int32), stable=True).indices
    dsts = torch.sort((~room).to(torch.int32), stable=True).indices
    some = i < move.sum()
    to = i.scatter(0, srcs, torch.where(some, dsts, srcs))     # page -> where it goes, and the other way round
    whence = torch.cat([i, i[:1]]).scatter(0, torch.where(some, dsts, n), torch.where(some, srcs, 0))[:n]
    st["codes"].copy_(st["codes"].view(torch.uint8)[:, whence].view(torch.float8_e4m3fn))
    st["scales"].copy_(st["scales"][:, whence])
    table.copy_(torch.where(table >= 0, to[table.long().clamp(min=0)].to(torch.int32), table))
    refs.copy_(_held(table, n))


def _compact_plain(st):
    half = st["n_pages"] // 2
    _moved_plain(st, half, st["n_pages"])
    _moved_plain(st, 0, half)
    return st["table"], st["refs"], st["codes"], st["scales"]


def _sinks_plain(st):
    case = st["case"]
    B, Hq, Hkv, d, n, L = case["batch"], case["heads"], case["kv_heads"], case["d"], st["most"], st["longest"]
    G = Hq // Hkv
    tab = st["table"].long().clamp(min=0)
    kv = st["codes"][0][tab].float() * st["scales"][0][tab][..., None, None]     # [B, width, Hkv, 2, page, d]
    kv = kv.permute(0, 2, 3, 1, 4, 5).reshape(B, Hkv, 2, -1, d)[:, :, :, :L]
    i = torch.arange(d // 2, dtype=torch.float64, device=tab.device)
    a = st["where"].double()[:, None, None] * torch.pow(THETA, -2.0 * i / d)
    c, s = torch.cos(a).float(), torch.sin(a).float()
    q1, q2 = st["q"].float()[..., :d // 2], st["q"].float()[..., d // 2:]
    q = torch.cat([q1 * c - q2 * s, q2 * c + q1 * s], -1)
    row = torch.arange(q.shape[0], device=q.device) - st["start"].long()[st["seq"]]
    qp = torch.zeros((B, n, Hq, d), device=q.device)
    qp[st["seq"], row] = q
    qp = qp.view(B, n, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, d)
    s = torch.matmul(qp, kv[:, :, 0].transpose(-1, -2)) * (d ** -0.5)
    key = torch.arange(L, device=q.device)
    p = (st["pos"].long()[:, None] + torch.arange(n, device=q.device))[..., None]
    see = (key <= p) & ((key > p - case["window"]) | (key < case["sinks"]))
    see = see[:, None, :, None].expand(B, 1, n, G, L).reshape(B, 1, n * G, L)
    s = torch.where(see, s, torch.full_like(s, -math.inf))
    w = torch.exp(s - s.amax(-1, keepdim=True))
    o = torch.matmul(w, kv[:, :, 1]) / w.sum(-1, keepdim=True)
    o = o.view(B, Hkv, n, G, d).permute(0, 2, 1, 3, 4).reshape(B, n, Hq, d)
    st["out"].copy_(o[st["seq"], row])
    return st["out"]


_PLAIN = {"select": _select_plain, "reorder": _reorder_plain, "fork": _fork_plain, "turn": _turn_plain,
          "compact": _compact_plain, "sinks": _sinks_plain}


def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        return _PLAIN[op](st)
    from int4_weight_kv_w4a16_gb300 import futr
    if op == "select":
        score, parent, token, ended = st["out"]
        futr.futr_beam_select(st["logits"], st["scores"], score, parent, token, st["ws"], done=st["done"], done_out=ended,
                              end=case["vocab"] - 1)
        return st["out"]
    if op == "reorder":
        futr.futr_kv_reorder(st["kv"], st["parent"], st["pos"])
        return st["streams"], st["pos"]
    if op == "fork":
        futr.futr_pages_fork(st["cache"], st["pool"], st["parent"], st["pos"], st["table"])
        return st["table"], st["refs"], st["pos"], st["codes"], st["scales"]
    if op == "turn":
        futr.futr_pages_free(st["cache"], st["pool"], st["pos"], st["table"], window=case["window"], sinks=case["sinks"])
        futr.futr_pages_grow(st["cache"], st["pool"], st["pos"], st["start"], st["table"])
        return st["table"], st["refs"]
    if op == "compact":
        half = st["n_pages"] // 2
        futr.futr_pages_compact(st["cache"], st["pool"], st["table"], half, st["n_pages"])
        futr.futr_pages_compact(st["cache"], st["pool"], st["table"], 0, half)
        return st["table"], st["refs"], st["codes"], st["scales"]
    futr.futr_paged_attention(st["cache"], 0, case["batch"], st["pos"], st["start"], st["table"], st["q"], st["out"],
                              st["ws"], window=case["window"], sinks=case["sinks"])
    return st["out"]


# ------------------------------------------------------------------- exact --

def _select_exact(case, st):
    out = []
    V, keep, end = case["vocab"], case["keep"], case["vocab"] - 1
    for b in range(case["batch"]):
        rows = st["logits"][b * case["beams"]:(b + 1) * case["beams"]].double()
        logp = torch.log_softmax(rows, -1)
        ended = st["done"][b] > 0
        logp[ended] = -math.inf
        logp[ended, end] = 0.0
        flat = (logp + st["scores"][b].double()[:, None]).reshape(-1)
        at = torch.argsort(-flat, stable=True)[:keep]
        out.append((flat[at], b * case["beams"] + torch.div(at, V, rounding_mode="floor"), at % V, at % V == end))
    return [torch.stack([o[k] for o in out]).to(t) for k, t in enumerate((torch.float64, torch.int32, torch.int32, torch.int32))]


def _sinks_exact(case, st):
    page, d, G = case["page"], case["d"], case["heads"] // case["kv_heads"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    past, new = _lens(case)
    r = 0
    f = THETA ** (-torch.arange(0, d, 2, dtype=torch.float64, device="cuda") / d)
    for b in range(case["batch"]):
        n, L = new[b], past[b] + new[b]
        tab = st["table"][b, :-(-L // page)].long().clamp(min=0)
        kv = st["codes"][0][tab].double() * st["scales"][0][tab].double()[..., None, None]
        K = kv[:, :, 0].transpose(0, 1).reshape(case["kv_heads"], -1, d)[:, :L].repeat_interleave(G, 0)
        V = kv[:, :, 1].transpose(0, 1).reshape(case["kv_heads"], -1, d)[:, :L].repeat_interleave(G, 0)
        x = st["q"][r:r + n].double()
        z = torch.complex(x[..., :d // 2], x[..., d // 2:])
        a = (past[b] + torch.arange(n, device="cuda", dtype=torch.float64))[:, None] * f
        z = z * torch.polar(torch.ones_like(a), a)[:, None]
        q = torch.cat([z.real, z.imag], -1).transpose(0, 1)                       # [Hq, n, d]
        s = q @ K.transpose(1, 2) / math.sqrt(d)
        j = torch.arange(L, device="cuda")
        age = (past[b] + torch.arange(n, device="cuda"))[:, None] - j
        s[:, (age < 0) | ((age >= case["window"]) & (j >= case["sinks"]))] = -math.inf
        out[r:r + n] = (torch.softmax(s, -1) @ V).transpose(0, 1)
        r += n
    return out


def exact(case, seed):
    """The other operators move and count what is there: whole numbers and codes, nothing computed."""
    if case["op"] not in ("select", "sinks"):
        return None
    st = _inputs(case, seed)
    return _select_exact(case, st) if case["op"] == "select" else _sinks_exact(case, st)
