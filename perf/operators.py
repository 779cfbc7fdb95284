"""The cache operators as they are measured: rotary positions with several axes (alone, and written
straight into a paged cache), the attention of one new token over that cache, and eviction by
accumulated attention weight.

``run`` computes a case in plain torch operations, or, where ``own`` is set, through the package.
Shapes follow the package's workloads: 32 / 8 heads of 128 (llama), 28 / 4 heads of 128 with frames of
256 tokens (video) and 8 / 8 heads of 64 (tiny).
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # --- rotary positions -------------------------------------------------------------------
        # one decoding step of 64 sequences: rotate q and k, write k and v into the pages
        {"name": "append_step_b64", "kind": "append", "batch": 64, "tokens": 1, "heads_q": 32,
         "heads_kv": 8, "head_dim": 128, "rotary": 128, "axes": 1, "pairing": "halves",
         "page_size": 16, "capacity": 256, "layout": "HND", "dtype": "bf16", "far": 131072},
        # a ragged chunk of a video prompt (time, height, width), token-major cache pages
        {"name": "append_video_chunk", "kind": "append", "batch": 3, "tokens": 2500, "heads_q": 28,
         "heads_kv": 4, "head_dim": 128, "rotary": 128, "axes": 3, "pairing": "halves",
         "page_size": 64, "capacity": 4096, "layout": "NHD", "dtype": "bf16", "far": 65536},
        # the whole 64K video prompt from the projection's layout into the prefill's
        {"name": "rotate_video_64k", "kind": "rotate", "batch": 1, "tokens": 65536, "heads_q": 28,
         "heads_kv": 4, "head_dim": 128, "rotary": 128, "axes": 3, "pairing": "halves",
         "inverse": False, "dtype": "bf16", "far": 65536},
        # gradients of a small layer: adjacent pairs, half of the head rotated, odd length
        {"name": "rotate_back_tiny", "kind": "rotate", "batch": 3, "tokens": 1023, "heads_q": 8,
         "heads_kv": 8, "head_dim": 64, "rotary": 32, "axes": 2, "pairing": "adjacent",
         "inverse": True, "dtype": "fp16", "far": 8192},
        # --- attention of one new token ---------------------------------------------------------
        # one user, a short context: latency
        {"name": "decode_one_1k", "kind": "decode", "batch": 1, "low": 1000, "high": 1000,
         "heads_q": 32, "heads_kv": 8, "head_dim": 128, "page_size": 16, "layout": "HND",
         "weights": False, "dtype": "bf16"},
        # a serving batch of mixed lengths
        {"name": "decode_batch_8k", "kind": "decode", "batch": 32, "low": 500, "high": 8192,
         "heads_q": 32, "heads_kv": 8, "head_dim": 128, "page_size": 16, "layout": "NHD",
         "weights": False, "dtype": "bf16"},
        # one user behind a 128K prompt
        {"name": "decode_long_128k", "kind": "decode", "batch": 1, "low": 131072, "high": 131072,
         "heads_q": 32, "heads_kv": 8, "head_dim": 128, "page_size": 128, "layout": "HND",
         "weights": False, "dtype": "bf16"},
        # several video prompts, the attention weights accumulated for eviction
        {"name": "decode_video_weights", "kind": "decode", "batch": 6, "low": 9000, "high": 65536,
         "heads_q": 28, "heads_kv": 4, "head_dim": 128, "page_size": 64, "layout": "HND",
         "weights": True, "dtype": "fp16"},
        # many heads without sharing, small ones, a page size that divides nothing, empty sequences
        {"name": "decode_mha_odd_pages", "kind": "decode", "batch": 9, "low": 0, "high": 3001,
         "heads_q": 8, "heads_kv": 8, "head_dim": 64, "page_size": 20, "layout": "HND",
         "weights": True, "dtype": "bf16"},
        # --- eviction ---------------------------------------------------------------------------
        # a prompt's cache halved after its prefill
        {"name": "evict_half_8k", "kind": "evict", "batch": 1, "low": 8192, "high": 8192,
         "budget": 4096, "sinks": 4, "recent": 256, "heads_kv": 8, "head_dim": 128,
         "page_size": 16, "layout": "HND", "dtype": "bf16"},
        # the steady state of a bounded cache: one entry too many in every sequence
        {"name": "evict_step_b32", "kind": "evict", "batch": 32, "low": 2049, "high": 2049,
         "budget": 2048, "sinks": 4, "recent": 128, "heads_kv": 8, "head_dim": 128,
         "page_size": 16, "layout": "NHD", "dtype": "bf16"},
        # long ragged prompts cut to a budget that some of them do not reach
        {"name": "evict_long_ragged", "kind": "evict", "batch": 5, "low": 5000, "high": 131072,
         "budget": 16384, "sinks": 16, "recent": 1000, "heads_kv": 4, "head_dim": 128,
         "page_size": 64, "layout": "HND", "dtype": "fp16"},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    kind = rng.choice(["append", "rotate", "decode", "evict"])
    heads_kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 5, 7, 8])
    c = {"kind": kind, "heads_kv": heads_kv, "head_dim": rng.choice([64, 128, 128]),
         "dtype": rng.choice(["bf16", "bf16", "fp16"])}
    if kind != "evict":
        c["heads_q"] = heads_kv * group
    if kind != "rotate":
        c["page_size"] = rng.choice([1, 7, 16, 16, 20, 32, 64, 128])
        c["layout"] = rng.choice(["HND", "NHD"])
    if kind in ("append", "rotate"):
        c["batch"] = _log(rng, 1, 64)
        c["tokens"] = 1 if rng.random() < 0.3 else _log(rng, 2, max(2, 16384 // c["batch"]))
        c["rotary"] = rng.choice([c["head_dim"], c["head_dim"], c["head_dim"] // 2])
        c["axes"] = rng.choice([1, 2, 3, 3])
        c["pairing"] = rng.choice(["halves", "halves", "adjacent"])
        c["far"] = _log(rng, 2 * c["tokens"], 1 << 20)
        if kind == "append":
            c["capacity"] = c["tokens"] + rng.randint(0, 300)
        else:
            c["inverse"] = rng.random() < 0.4
        return c
    entries = 2 ** 19 // heads_kv      # entries per head over all sequences: at most 134 MB of K
    if kind == "decode":
        c["batch"] = _log(rng, 1, 48)
        c["high"] = _log(rng, 1, min(131072, entries // c["batch"]))
        c["low"] = rng.choice([0, c["high"] // 8, c["high"]])
        c["weights"] = rng.random() < 0.4
        return c
    c["batch"] = _log(rng, 1, 24)
    c["high"] = _log(rng, 32, min(131072, entries // c["batch"]))
    c["low"] = rng.choice([c["high"] // 4, c["high"]])
    c["budget"] = rng.choice([c["high"] - 1, c["high"] // 2, max(8, c["high"] // 8)])
    c["sinks"] = rng.randint(0, c["budget"] // 4)
    c["recent"] = rng.randint(0, c["budget"] // 2)
    return c


# ------------------------------------------------------------------------------------ preparation
def _lengths(case):
    """Lengths spread evenly over [low, high], both ends among them where there are two or more."""
    n, low, high = case["batch"], case["low"], case["high"]
    if n == 1:
        return [high]
    return [low + (high - low) * i // (n - 1) for i in range(n)]


def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _pages(case, capacities, g):
    """An empty cache whose sequences own pages in random order: k, v [pages, heads, entries, d]."""
    ps, dt = case["page_size"], TYPES[case["dtype"]]
    need = [-(-max(c, 1) // ps) for c in capacities]
    total = sum(need) + 3
    order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    width = max(need)
    first = torch.tensor([sum(need[:i]) for i in range(len(need))], device=DEV)
    col = torch.arange(width, device=DEV)
    at = first[:, None] + col[None, :]
    have = col[None, :] < torch.tensor(need, device=DEV)[:, None]
    table = torch.where(have, order[at.clamp(max=total - 1)], -1).to(torch.int32)

    def make():
        x = torch.randn(total, case["heads_kv"], ps, case["head_dim"], generator=g, device=DEV,
                        dtype=torch.float32).to(dt)
        if case["layout"] == "NHD":
            x = x.transpose(1, 2).contiguous().transpose(1, 2)
        return x

    return make(), make(), table.contiguous()


def _angles_in(case, b, t, start, g):
    """int32 positions [axes, b, t]: ordinals, or frames, rows and columns of a video."""
    if case["axes"] == 1:
        return (start[:, None] + torch.arange(t, device=DEV)[None, :])[None].to(torch.int32)
    n = start[:, None] + torch.arange(t, device=DEV)[None, :]
    axes = [n // 256, (n // 16) % 16, n % 16][:case["axes"]]
    return torch.stack(axes).to(torch.int32).contiguous()


def _sections(case):
    """Pairs of each axis: a quarter for the first of three, the rest shared evenly."""
    pairs, axes = case["rotary"] // 2, case["axes"]
    if axes == 1:
        return [pairs]
    if axes == 2:
        return [pairs // 2, pairs - pairs // 2]
    first = pairs // 4
    second = (pairs - first) // 2
    return [first, second, pairs - first - second]


def _table(case):
    from long_context_prefill_rr_b200 import cache
    return cache.RopeTable(case["head_dim"], rotary_dim=case["rotary"], theta=500000.0,
                           sections=_sections(case), pairing=case["pairing"])


def prepare(case, seed):
    g = _generator(seed)
    kind, b, d = case["kind"], case["batch"], case["head_dim"]
    dt = TYPES[case["dtype"]]
    s = {"case": case}
    if kind in ("append", "rotate"):
        t, hq, hkv = case["tokens"], case["heads_q"], case["heads_kv"]
        # q, k, v are slices of one projection [b, t, heads, d], seen head-first
        x = torch.randn(b, t, hq + 2 * hkv, d, generator=g, device=DEV).to(dt).transpose(1, 2)
        s["q"], s["k"], s["v"] = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        start = torch.randint(0, max(1, case["far"] - t), (b,), generator=g, device=DEV)
        s["positions"] = _angles_in(case, b, t, start, g)
        s["q_out"] = torch.zeros(b, hq, t, d, device=DEV, dtype=dt)
        s["k_out"] = torch.zeros(b, hkv, t, d, device=DEV, dtype=dt)
        if kind == "append":
            kc, vc, table = _pages(case, [case["capacity"]] * b, g)
            new = torch.full((b,), t, dtype=torch.int32, device=DEV)
            if t > 1:
                new -= torch.randint(0, t // 2 + 1, (b,), generator=g, device=DEV).to(torch.int32)
            room = case["capacity"] - t
            length = torch.randint(0, room + 1, (b,), generator=g, device=DEV).to(torch.int32)
            s.update(k_cache=kc, v_cache=vc, page_table=table, len=length, new_len=new)
            s["seen"] = start.to(torch.int32)
            s["weight"] = torch.rand(kc.shape[:3], generator=g, device=DEV)
            s["order"] = torch.zeros(kc.shape[:3], dtype=torch.int32, device=DEV)
    else:
        lens = torch.tensor(_lengths(case), device=DEV)
        lens = lens[torch.randperm(b, generator=g, device=DEV)].to(torch.int32)
        cap = [int(n) for n in lens.tolist()]
        s["k_cache"], s["v_cache"], s["page_table"] = _pages(case, cap, g)
        s["len"] = lens
        shape = s["k_cache"].shape[:3]
        if kind == "decode":
            # queries that lean towards some keys: weights from flat to sharp
            q = torch.randn(b, case["heads_q"], d, generator=g, device=DEV)
            s["q"] = (q * torch.linspace(0.5, 3.0, case["heads_q"], device=DEV)[:, None]).to(dt)
            s["out"] = torch.empty(b, case["heads_q"], d, device=DEV, dtype=dt)
            s["lse"] = torch.empty(b, case["heads_q"], device=DEV)
            if case["weights"]:
                s["weight0"] = torch.rand(shape, generator=g, device=DEV) * 1e-3
                s["weight"] = s["weight0"].clone()
                s["order"] = torch.zeros(shape, dtype=torch.int32, device=DEV)
                s["seen"] = lens.clone()
        else:
            # long-tailed weights, a tenth of them exactly zero; ordinals as earlier evictions
            # leave them: distinct, in any order
            w = torch.exp(2.0 * torch.randn(shape, generator=g, device=DEV))
            w *= torch.rand(shape, generator=g, device=DEV) > 0.1
            hkv, longest = case["heads_kv"], max(cap)
            s["seen"] = (lens + lens // 4).to(torch.int32)
            r = torch.rand(b, hkv, longest + longest // 4, generator=g, device=DEV)
            past = torch.arange(r.shape[2], device=DEV) >= s["seen"][:, None]
            r.masked_fill_(past[:, None, :], 2.0)
            ordinal = r.argsort(dim=2)[:, :, :longest].to(torch.int32)
            order = torch.zeros(shape, dtype=torch.int32, device=DEV)
            page, off, valid = _slots(s["page_table"], lens, case["page_size"], longest)
            head = torch.arange(hkv, device=DEV)[None, :, None]
            put = valid[:, None, :].expand(b, hkv, longest)
            order[page[:, None].expand_as(put)[put], head.expand_as(put)[put],
                  off[:, None].expand_as(put)[put]] = ordinal[put]
            s["weight0"], s["order0"] = w, order
            s["weight"], s["order"] = w.clone(), order.clone()
    if own:
        from long_context_prefill_rr_b200 import cache
        if kind in ("append", "rotate"):
            s["table"] = _table(case)
        if kind != "rotate":
            s["cache"] = cache.PagedCache(
                s["k_cache"], s["v_cache"], s["page_table"], s["len"],
                heads_q=case.get("heads_q", case["heads_kv"]), weight=s.get("weight"),
                order=s.get("order"), seen=s.get("seen"))
    return s


# ----------------------------------------------------------------------------------- plain forms
def _slots(table, lens, page_size, count):
    """Page, place in the page and validity of entries 0 .. count-1 of every sequence."""
    e = torch.arange(count, device=table.device)
    page = table[:, (e // page_size).clamp(max=table.shape[1] - 1)].long().clamp(min=0)
    off = (e % page_size)[None, :].expand_as(page)
    return page, off, e[None, :] < lens[:, None]


def _cos_sin(case, positions):
    """fp32 cosine and sine [b, 1, t, pairs] of angles taken in 64 bits: far positions turn often."""
    rot = case["rotary"]
    axis = torch.repeat_interleave(torch.arange(case["axes"], device=DEV),
                                   torch.tensor(_sections(case), device=DEV))
    freq = 500000.0 ** (-2.0 * torch.arange(rot // 2, device=DEV, dtype=torch.float64) / rot)
    angle = positions[axis].permute(1, 2, 0).double() * freq
    if case.get("inverse"):
        angle = -angle
    return torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]


def _rotate(case, x, cos, sin):
    rot = case["rotary"]
    y = x.float()
    if case["pairing"] == "halves":
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    else:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    return torch.cat([turned, y[..., rot:]], dim=-1).to(x.dtype)


def _plain_rotate(s):
    c = s["case"]
    cos, sin = _cos_sin(c, s["positions"])
    s["q_out"].copy_(_rotate(c, s["q"], cos, sin))
    s["k_out"].copy_(_rotate(c, s["k"], cos, sin))


def _plain_append(s):
    c = s["case"]
    cos, sin = _cos_sin(c, s["positions"])
    t = torch.arange(c["tokens"], device=DEV)
    real = t[None, :] < s["new_len"][:, None]
    q, k = _rotate(c, s["q"], cos, sin), _rotate(c, s["k"], cos, sin)
    s["q_out"].copy_(torch.where(real[:, None, :, None], q, s["q_out"]))
    e = (s["len"][:, None] + t[None, :])[real]
    row = torch.arange(c["batch"], device=DEV)[:, None].expand_as(real)[real]
    page = s["page_table"][row, e // c["page_size"]].long()
    off = e % c["page_size"]
    s["k_cache"][page, :, off] = k.transpose(1, 2)[real]
    s["v_cache"][page, :, off] = s["v"].transpose(1, 2)[real]
    s["weight"][page, :, off] = 0.0
    s["order"][page, :, off] = (s["seen"][:, None] + t[None, :].int())[real][:, None]


def _plain_decode(s):
    c = s["case"]
    b, hq, hkv, d = c["batch"], c["heads_q"], c["heads_kv"], c["head_dim"]
    longest = s["page_table"].shape[1] * c["page_size"]
    page, off, valid = _slots(s["page_table"], s["len"], c["page_size"], longest)
    q = s["q"].float().view(b, hkv, hq // hkv, d)
    k = s["k_cache"][page, :, off].float()                 # [b, entries, hkv, d]
    logit = torch.einsum("bhgd,behd->bhge", q, k) / math.sqrt(d)
    logit = logit.masked_fill(~valid[:, None, None, :], -math.inf)
    top = logit.amax(dim=-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp(logit - top)
    total = p.sum(dim=-1, keepdim=True)
    p = p / torch.where(total > 0, total, torch.ones_like(total))
    del k, logit
    o = torch.einsum("bhge,behd->bhgd", p, s["v_cache"][page, :, off].float())
    s["out"].copy_(o.reshape(b, hq, d))
    s["lse"].copy_((top + torch.log(total)).reshape(b, hq))
    if c["weights"]:
        s["weight"].copy_(s["weight0"])
        share = p.sum(dim=2)                               # [b, hkv, entries]
        s["weight"][page[valid], :, off[valid]] += share.transpose(1, 2)[valid]


def _plain_evict(s):
    c = s["case"]
    s["weight"].copy_(s["weight0"])
    s["order"].copy_(s["order0"])
    longest = s["page_table"].shape[1] * c["page_size"]
    page, off, valid = _slots(s["page_table"], s["len"], c["page_size"], longest)
    w = s["weight"][page, :, off].transpose(1, 2).double()           # [b, hkv, entries]
    order = s["order"][page, :, off].transpose(1, 2)
    seen = s["seen"][:, None, None]
    safe = (order < c["sinks"]) | (order >= seen - c["recent"])
    key = torch.where(safe, torch.full_like(w, 1e300), w)
    key = torch.where(valid[:, None, :], key, torch.full_like(w, -1.0))
    ranked = key.argsort(dim=2, descending=True, stable=True)
    rank = torch.empty_like(ranked)
    rank.scatter_(2, ranked, torch.arange(longest, device=DEV).expand_as(ranked))
    keep = torch.minimum(s["len"], torch.full_like(s["len"], c["budget"]))[:, None, None]
    kept = rank < keep
    e = torch.arange(longest, device=DEV)[None, None, :]
    over = valid[:, None, :] & (s["len"] > c["budget"])[:, None, None]
    bh, hh, eh = (over & ~kept & (e < keep)).nonzero(as_tuple=True)   # evicted places in front
    bm, hm, em = (over & kept & (e >= keep)).nonzero(as_tuple=True)   # kept entries behind
    to = (page[bh, eh], hh, off[bh, eh])
    frm = (page[bm, em], hm, off[bm, em])
    s["k_cache"][to] = s["k_cache"][frm]
    s["v_cache"][to] = s["v_cache"][frm]
    s["weight"][to] = s["weight"][frm]
    s["order"][to] = s["order"][frm]


# ------------------------------------------------------------------------------------------- run
def run(state):
    """One pass. The evicted cache is put back to its weights and ordinals first, the decoded one to
    its weights, so that a pass can be repeated: the rows that eviction moves come from places
    that it does not write."""
    s, c = state, state["case"]
    kind = c["kind"]
    if kind == "rotate":
        if own:
            from long_context_prefill_rr_b200 import cache
            cache.rope(s["table"], s["positions"], s["q"], s["k"], q_out=s["q_out"],
                       k_out=s["k_out"], inverse=c["inverse"])
        else:
            _plain_rotate(s)
        return {"q": s["q_out"], "k": s["k_out"]}
    if kind == "append":
        if own:
            # one of several layers that share the lengths: they advance with the last
            s["cache"].append(s["table"], s["positions"], s["q"], s["k"], s["v"],
                              new_len=s["new_len"], q_out=s["q_out"], advance=False)
        else:
            _plain_append(s)
        return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"],
                "weight": s["weight"], "order": s["order"]}
    if kind == "decode":
        if own:
            if c["weights"]:
                s["weight"].copy_(s["weight0"])
            s["cache"].decode(s["q"], out=s["out"], lse=s["lse"], add_weight=c["weights"])
        else:
            _plain_decode(s)
        got = {"out": s["out"], "lse": s["lse"]}
        if c["weights"]:
            got["weight"] = s["weight"]
        return got
    if own:
        s["weight"].copy_(s["weight0"])
        s["order"].copy_(s["order0"])
        s["cache"].evict(c["budget"], sinks=c["sinks"], recent=c["recent"], advance=False)
    else:
        _plain_evict(s)
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "weight": s["weight"],
            "order": s["order"]}


# ------------------------------------------------------------------------------------------ work
def work(case):
    b, d, hkv, kind = case["batch"], case["head_dim"], case["heads_kv"], case["kind"]
    if kind in ("append", "rotate"):
        hq, t = case["heads_q"], case["tokens"]
        if kind == "append" and t > 1:
            t = t - (t // 2) / 2          # padding is neither read nor written: the mean length
        rows = hq + hkv * (2 if kind == "append" else 1)
        flops = 3 * case["rotary"] * b * t * (hq + hkv)
        moved = b * t * (rows * d * 2 * 2 + 4 * case["axes"])
        if kind == "append":
            moved += b * t * hkv * 8
        return {"bytes": moved, "flops": flops}
    lens = _lengths(case)
    pages = sum(-(-n // case["page_size"]) for n in lens) * 4
    if kind == "decode":
        hq = case["heads_q"]
        moved = sum(lens) * hkv * d * 2 * 2 + b * hq * (d * 2 * 2 + 4) + pages
        if case["weights"]:
            moved += sum(lens) * hkv * 8
        return {"bytes": moved, "flops": 4 * d * hq * sum(lens)}
    budget = case["budget"]
    over = [n for n in lens if n > budget]
    # weights in any order: a share budget / n of the n - budget entries behind is kept
    rows = sum(budget * (n - budget) / n for n in over) * hkv
    return {"bytes": sum(over) * hkv * 8 + rows * (2 * 2 * d * 2 + 8) + pages, "flops": 0}


# ----------------------------------------------------------------------------------------- exact
def _turned(case, x, positions):
    """Pairs as complex numbers times e^(i angle), in 64 bits."""
    rot, pairs = case["rotary"], case["rotary"] // 2
    which = []
    for axis, n in enumerate(_sections(case)):
        which += [axis] * n
    inv = torch.tensor([math.pow(500000.0, -2.0 * i / rot) for i in range(pairs)],
                       dtype=torch.float64, device=x.device)
    angle = torch.stack([positions[a].double() for a in which], dim=-1) * inv
    turn = torch.polar(torch.ones_like(angle), -angle if case.get("inverse") else angle)
    y = x.double()
    z = (torch.complex(y[..., :pairs], y[..., pairs:rot]) if case["pairing"] == "halves" else
         torch.view_as_complex(y[..., :rot].unflatten(-1, (pairs, 2)).contiguous()))
    z = z * turn[:, None]
    y = y.clone()
    if case["pairing"] == "halves":
        y[..., :pairs], y[..., pairs:rot] = z.real, z.imag
    else:
        y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    kind, ps = case["kind"], case["page_size"] if "page_size" in case else 0
    if kind == "rotate":
        return {"q": _turned(case, s["q"], s["positions"]),
                "k": _turned(case, s["k"], s["positions"])}
    lens = s["len"].tolist()
    table = s["page_table"].long()

    def slots(b, first, last):
        e = torch.arange(first, last, device=table.device)
        return table[b, e // ps], e % ps

    if kind == "append":
        q, k = (_turned(case, s[n], s["positions"]) for n in ("q", "k"))
        q_out, kc, vc = s["q_out"].double(), s["k_cache"].double(), s["v_cache"].double()
        weight, order = s["weight"].double(), s["order"].clone()
        for b, n in enumerate(s["new_len"].tolist()):
            page, off = slots(b, lens[b], lens[b] + n)
            q_out[b, :, :n] = q[b, :, :n]
            kc[page, :, off] = k[b, :, :n].transpose(0, 1)
            vc[page, :, off] = s["v"][b, :, :n].transpose(0, 1).double()
            weight[page, :, off] = 0.0
            first = int(s["seen"][b])
            order[page, :, off] = torch.arange(first, first + n, device=table.device,
                                               dtype=torch.int32)[:, None]
        return {"q": q_out, "k_cache": kc, "v_cache": vc, "weight": weight, "order": order}
    if kind == "decode":
        hq, hkv, d = case["heads_q"], case["heads_kv"], case["head_dim"]
        out = torch.zeros(case["batch"], hq, d, dtype=torch.float64, device=table.device)
        lse = torch.full((case["batch"], hq), -math.inf, dtype=torch.float64, device=table.device)
        weight = s["weight0"].double() if case["weights"] else None
        for b, n in enumerate(lens):
            if n == 0:
                continue
            page, off = slots(b, 0, n)
            for h in range(hkv):
                mine = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
                x = s["q"][b, mine].double() @ s["k_cache"][page, h, off].double().T / math.sqrt(d)
                lse[b, mine] = torch.logsumexp(x, dim=1)
                p = torch.softmax(x, dim=1)
                out[b, mine] = p @ s["v_cache"][page, h, off].double()
                if weight is not None:
                    weight[page, h, off] += p.sum(dim=0)
        got = {"out": out, "lse": lse}
        if weight is not None:
            got["weight"] = weight
        return got
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    weight, order = s["weight0"].double(), s["order0"].clone()
    budget = case["budget"]
    for b, n in enumerate(lens):
        if n <= budget:
            continue
        page, off = slots(b, 0, n)
        seen = int(s["seen"][b])
        for h in range(case["heads_kv"]):
            o, w = order[page, h, off].long(), weight[page, h, off]
            safe = (o < case["sinks"]) | (o >= seen - case["recent"])
            free = torch.nonzero(~safe)[:, 0]
            # largest weight first, ties by place: a stable ascending sort of the negated weights
            best = free[torch.sort(-w[free], stable=True)[1]][:budget - int(safe.sum())]
            kept = safe.clone()
            kept[best] = True
            hole = torch.nonzero(~kept[:budget])[:, 0]
            move = torch.nonzero(kept[budget:])[:, 0] + budget
            for x in (kc, vc, weight, order):
                x[page[hole], h, off[hole]] = x[page[move], h, off[move]]
    return {"k_cache": kc, "v_cache": vc, "weight": weight, "order": order}
