"""The operators between a decoder block's linears, as cases that can be timed.

Three operators of the serving path around the delta linears:

  norm       h = residual + scale * gate * RMSNorm(y; w_post), x = RMSNorm(h; w_pre),
             the norm weights chosen per row segment (variant id, 0 = base)
  append     rotary positions on the query and key heads of a QKV row, the rotated
             keys and the values written to a paged cache
  attention  causal attention of ragged query runs over that cache, for prompts and
             single tokens, with a prefix that groups of sequences share

`run` computes each either in its plain form (elementary torch operations in 32
bits, rounded once) or, where `own` is true, by the calls a user makes.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-5
ROPE_BASE = 10000.0


def listed():
    return [
        # one decode step of a 70B-shaped slice: 8 rows alternating two variants
        _norm("norm_decode", 8, 8192, variants=2, post=False, gate="none", res="bf16"),
        # multi-tenant batch: 64 one-row and four 512-row segments over 14 variants, norms
        # before and after the block, a gate per channel, an fp32 residual stream
        _norm("norm_tenants", 2112, 4096, variants=14, post=True, gate="channel", res="fp32"),
        # the new token of 8 sequences in a decode step (64 query and 8 key/value heads x 128)
        _append("append_decode", 8, 1, 0, 0, 300, 1800, 64, 8, 128, 16, 128, False),
        # multi-tenant batch: 64 decode rows and four 512-token chunks, half of each head
        # rotated in pairs, 64-token pages
        _append("append_mixed", 64, 1, 4, 512, 513, 4100, 32, 8, 128, 64, 64, True),
        # four 2048-token prompts at once
        _append("append_prompts", 0, 1, 4, 2048, 2048, 2048, 64, 8, 128, 16, 128, False),
        # a decode step of 8 short conversations: latency
        _attn("decode_8", 8, 1, 0, 0, 120, 1000, 64, 8, 128, 16),
        # a full decode batch with ragged contexts
        _attn("decode_64", 64, 1, 0, 0, 500, 8000, 64, 8, 128, 64),
        # one conversation with a very long context: few rows, one long axis
        _attn("decode_1_long", 1, 1, 0, 0, 131071, 131071, 64, 8, 128, 16),
        # 64 requests in two groups, each behind its own long system prompt
        _attn("shared_64", 64, 1, 0, 0, 8192 + 37, 8192 + 700, 64, 8, 128, 64, prefix=8192,
              group=32),
        # multi-tenant batch: 64 decode rows and four 512-token chunks over earlier context
        _attn("mixed_68", 64, 1, 4, 512, 513, 2500, 32, 8, 128, 32),
        # one 2048-token prompt
        _attn("prompt_2048", 0, 1, 1, 2048, 2048, 2048, 64, 8, 128, 16),
        # one long prompt
        _attn("prompt_8192", 0, 1, 1, 8192, 8192, 8192, 64, 8, 128, 64),
    ]


def _norm(name, rows, d, variants, post, gate, res):
    return {"name": name, "op": "norm", "rows": rows, "d": d, "variants": variants, "post": post,
            "gate": gate, "res": res}


def _append(name, short, q_short, long, q_long, kv_lo, kv_hi, hq, hkv, dim, page, rot,
            interleaved):
    return {"name": name, "op": "append", "short": short, "q_short": q_short, "long": long,
            "q_long": q_long, "kv_lo": kv_lo, "kv_hi": kv_hi, "hq": hq, "hkv": hkv, "dim": dim,
            "page": page, "rot": rot, "interleaved": interleaved, "prefix": 0, "group": 0}


def _attn(name, short, q_short, long, q_long, kv_lo, kv_hi, hq, hkv, dim, page, prefix=0,
          group=0):
    return {"name": name, "op": "attention", "short": short, "q_short": q_short, "long": long,
            "q_long": q_long, "kv_lo": kv_lo, "kv_hi": kv_hi, "hq": hq, "hkv": hkv, "dim": dim,
            "page": page, "prefix": prefix, "group": group}


def draw(rng):
    def size(lo, hi):  # spread over the logarithm
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    kind = rng.choice(["norm", "append", "decode", "decode", "shared", "mixed", "prompt"])
    if kind == "norm":
        d = rng.choice([1024, 2048, 4096, 5120, 8192, 16384, 8 * size(64, 2048)])
        rows = size(1, max(2, min(8192, (1 << 24) // d)))
        c = _norm("", rows, d, rng.choice([0, 1, 2, 14]), rng.random() < 0.5,
                  rng.choice(["none", "channel", "row"]), rng.choice(["bf16", "fp32"]))
        c.pop("name")
        return c
    hq, hkv = rng.choice([(64, 8), (32, 8), (40, 8), (24, 8), (32, 4), (16, 16), (16, 2), (28, 4)])
    dim, page = rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128])
    if kind == "append":
        rot = rng.choice([dim, dim, dim // 2])
        n = size(1, 256)
        long = rng.choice([0, 0, 1, 3])
        q_long = size(17, 2048) if long else 0
        kv_lo = max(q_long, size(1, 2000)) + 1
        c = _append("", n, rng.choice([1, 1, 3]), long, q_long, kv_lo + 3, kv_lo + 3 + size(1, 2000),
                    hq, hkv, dim, page, rot, rng.random() < 0.5)
    elif kind == "decode":
        n = size(1, 256)
        most = 270000 * 1024 // (hkv * dim)  # keys in all: no more bytes than the largest case
        kv_hi = size(16, max(32, min(131071, most // n)))
        c = _attn("", n, rng.choice([1, 1, 1, 2]), 0, 0, max(2, kv_hi // rng.choice([1, 3, 10])),
                  kv_hi, hq, hkv, dim, page)
    elif kind == "shared":
        group = rng.choice([8, 16, 33, 64])
        n = group * rng.choice([1, 2, 3])
        prefix = page * max(1, size(256, 16384) // page)
        own_lo = size(1, 200) + 1
        c = _attn("", n, 1, 0, 0, prefix + own_lo, prefix + own_lo + size(1, 800), hq, hkv, dim,
                  page, prefix=prefix, group=group)
    elif kind == "mixed":
        long, q_long = rng.choice([1, 2, 4]), size(40, 600)
        kv_lo = q_long + size(1, 600)
        c = _attn("", size(1, 64), 1, long, q_long, kv_lo, kv_lo + size(1, 1500), hq, hkv, dim, page)
    else:
        q_long, long = size(33, 4096), 1
        if q_long < 1024:
            long = rng.choice([1, 2, 5])
        c = _attn("", 0, 1, long, q_long, q_long, q_long + rng.choice([0, 0, size(1, 2000)]), hq,
                  hkv, dim, page)
    c.pop("name")
    return c


# ------------------------------------------------------------------ sizes


def _lengths(c):
    """Query and key/value lengths of a case's sequences before the seed's shuffle: the short
    ones first, the key/value lengths spread evenly over the case's range."""
    q, kv = [], []
    for n, ql in ((c["short"], c["q_short"]), (c["long"], c["q_long"])):
        for i in range(n):
            q.append(ql)
            kv.append(c["kv_lo"] + (c["kv_hi"] - c["kv_lo"]) * i // max(1, n - 1))
    return q, [max(a, b) for a, b in zip(kv, q)]


def work(case):
    c = case
    if c["op"] == "norm":
        r = 2 if c["res"] == "bf16" else 4
        n, d = c["rows"], c["d"]
        per_row = 2 + 2 * r + 2 + (2 if c["gate"] == "row" else 0)
        weights = (2 if c["post"] else 1) * min(c["variants"] + 1, n) + (c["gate"] == "channel")
        return {"bytes": n * d * per_row + 2 * weights * d, "flops": n * d * (8 if c["post"] else 5)}
    q, kv = _lengths(c)
    hq, hkv, dim = c["hq"], c["hkv"], c["dim"]
    tables = 4 * (2 * len(q) + 1) + sum(4 * -(-k // c["page"]) for k in kv)
    if c["op"] == "append":
        t = sum(q)
        return {"bytes": t * (4 * (hq + 2 * hkv) * dim + 4 * c["rot"]) + tables,
                "flops": 3 * t * (hq + hkv) * c["rot"]}
    groups = len(q) // c["group"] if c["prefix"] else 0
    keys = sum(kv) - (len(q) - groups) * c["prefix"]
    seen = sum(ql * (k - ql) + ql * (ql + 1) // 2 for ql, k in zip(q, kv))
    return {"bytes": 4 * sum(q) * hq * dim + 4 * sum(q) * hq + 4 * keys * hkv * dim + tables,
            "flops": 4 * seen * hq * dim}


# ------------------------------------------------------------------ inputs


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.bfloat16):
        return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dtype)

    if c["op"] == "norm":
        return _prepare_norm(c, seed, normal)
    rng = np.random.default_rng(seed)
    q_len, kv_len = (np.array(v, np.int64) for v in _lengths(c))
    n, ns = len(q_len), c["short"]
    for lo, hi in ((0, ns), (ns, n)):  # which sequence has which length goes by the seed
        kv_len[lo:hi] = rng.permutation(kv_len[lo:hi])
    off = np.concatenate([[0], np.cumsum(q_len)])
    page, prefix = c["page"], c["prefix"]
    pages_of = -(-kv_len // page)
    # the first prefix // page pages of a group's sequences are one and the same
    shared = [prefix // page if prefix and s % c["group"] else 0 for s in range(n)]
    n_pages = int(pages_of.sum()) - sum(shared) + 3
    order, used = rng.permutation(n_pages), 0
    table = np.zeros((n, int(pages_of.max())), np.int32)
    for s in range(n):
        table[s, :shared[s]] = table[s - 1, :shared[s]]
        fresh = int(pages_of[s]) - shared[s]
        table[s, shared[s]:pages_of[s]] = order[used:used + fresh]
        used += fresh
    hq, hkv, dim, tokens = c["hq"], c["hkv"], c["dim"], int(off[-1])
    state = {
        "case": c, "tokens": tokens, "max_kv": int(kv_len.max()),
        "seq_offsets": torch.from_numpy(off.astype(np.int32)).cuda(),
        "kv_len": torch.from_numpy(kv_len.astype(np.int32)).cuda(),
        "page_table": torch.from_numpy(table).cuda(),
        # every page holds values: a recycled cache is full of earlier tokens
        "k_pages": normal(n_pages, hkv, page, dim, std=1.2),
        "v_pages": normal(n_pages, hkv, page, dim),
    }
    if c["op"] == "append":
        state["qkv"] = normal(tokens, (hq + 2 * hkv) * dim)
        pos = torch.arange(int(kv_len.max()), device="cuda", dtype=torch.float64)
        half = torch.arange(c["rot"] // 2, device="cuda", dtype=torch.float64)
        angle = pos[:, None] * ROPE_BASE ** (-2.0 * half / c["rot"])
        state["rope"] = torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32)
    else:
        state["q"] = normal(tokens, hq, dim, std=1.5)
        if prefix:
            state["group_offsets"] = torch.arange(0, n + 1, c["group"], device="cuda",
                                                  dtype=torch.int32)
            state["prefix_len"] = torch.full((n // c["group"],), prefix, device="cuda",
                                             dtype=torch.int32)
    if own:  # a serving loop keeps the batch and its plan for all layers of a step
        import bit_weight_delta_gb300 as bd
        state["batch"] = bd.AttentionBatch(
            state["seq_offsets"], state["kv_len"], state["page_table"], n_tokens=tokens,
            max_q_len=int(q_len.max()), max_kv_len=int(kv_len.max()), n_q_heads=hq,
            n_kv_heads=hkv, head_dim=dim, page_size=page,
            group_offsets=state.get("group_offsets"), prefix_len=state.get("prefix_len"))
    return state


def _prepare_norm(c, seed, normal):
    rows, d, nv = c["rows"], c["d"], c["variants"]
    res = torch.bfloat16 if c["res"] == "bf16" else torch.float32
    state = {
        "case": c,
        "y": normal(rows, d, std=0.7),
        "residual": normal(rows, d, std=3.0, dtype=res),
        "pre": normal(nv + 1, d, std=0.1, mean=1.0),
        "post": normal(nv + 1, d, std=0.1, mean=0.5) if c["post"] else None,
        "gate": {"none": lambda: None, "channel": lambda: normal(d, std=0.3, mean=0.8),
                 "row": lambda: normal(rows, d, std=0.3, mean=0.8)}[c["gate"]](),
        "scale": 0.75 if c["gate"] != "none" else 1.0,
        "seg_offsets": None, "seg_variant": None,
    }
    if nv:  # decode rows are one-row segments; of many rows, all but 64 in four long segments
        rng = np.random.default_rng(seed)
        ones = min(rows, 64)
        cuts = list(range(ones + 1))
        rest = rows - ones
        cuts += [ones + rest * i // 4 for i in range(1, 5)] if rest >= 4 else ([rows] if rest else [])
        state["seg_offsets"] = torch.tensor(cuts, dtype=torch.int32).cuda()
        state["seg_variant"] = torch.from_numpy(
            rng.integers(0, nv + 1, len(cuts) - 1).astype(np.int32)).cuda()
    if own:
        import bit_weight_delta_gb300 as bd
        state["pre_table"] = bd.norm_table(list(state["pre"]))
        state["post_table"] = bd.norm_table(list(state["post"])) if c["post"] else None
    return state


# ------------------------------------------------------------------ one pass


def run(state):
    op = state["case"]["op"]
    if own:
        import bit_weight_delta_gb300 as bd
        if op == "norm":
            h, x = bd.bitdelta_add_norm(
                state["y"], state["residual"], state["pre_table"], post_table=state["post_table"],
                gate=state["gate"], scale=state["scale"], eps=EPS,
                seg_offsets=state["seg_offsets"], seg_variant=state["seg_variant"])
            return {"h": h, "x": x}
        if op == "append":
            q = bd.bitdelta_kv_append(state["batch"], state["qkv"], state["rope"],
                                      state["k_pages"], state["v_pages"],
                                      interleaved=state["case"]["interleaved"])
            return {"q": q, "k_pages": state["k_pages"], "v_pages": state["v_pages"]}
        out, lse = bd.bitdelta_attention(state["batch"], state["q"], state["k_pages"],
                                         state["v_pages"])
        return {"out": out, "lse": lse}
    return {"norm": _plain_norm, "append": _plain_append, "attention": _plain_attention}[op](state)


def _plain_norm(st):
    def rms(v):
        return v / torch.sqrt((v * v).mean(dim=1, keepdim=True) + EPS)

    rows = st["y"].shape[0]
    slot = torch.zeros(rows, dtype=torch.int64, device="cuda")
    if st["seg_offsets"] is not None:
        row = torch.arange(rows, device="cuda")
        seg = (row[:, None] >= st["seg_offsets"][None, 1:]).sum(dim=1)
        slot = st["seg_variant"][seg].long()
    b = st["y"].float()
    if st["post"] is not None:
        b = rms(b) * st["post"].float()[slot]
    if st["gate"] is not None:
        b = b * st["gate"].float()
    h = st["residual"].float() + st["scale"] * b
    x = rms(h) * st["pre"].float()[slot]
    return {"h": h.to(st["residual"].dtype), "x": x.to(torch.bfloat16)}


def _token_places(st):
    """Sequence and position of every token of the batch."""
    off = st["seq_offsets"].long()
    tok = torch.arange(st["tokens"], device="cuda")
    seq = (tok[:, None] >= off[None, 1:]).sum(dim=1)
    pos = st["kv_len"].long()[seq] - (off[seq + 1] - tok)
    return seq, pos


def _plain_append(st):
    c = st["case"]
    hq, hkv, dim, rot, page = c["hq"], c["hkv"], c["dim"], c["rot"], c["page"]
    seq, pos = _token_places(st)
    heads = st["qkv"].view(st["tokens"], hq + 2 * hkv, dim)
    x = heads[:, :hq + hkv].float()
    cos = st["rope"][pos, :rot // 2][:, None]
    sin = st["rope"][pos, rot // 2:][:, None]
    r, keep = x[..., :rot], x[..., rot:]
    if c["interleaved"]:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    x = torch.cat([r, keep], dim=-1).to(torch.bfloat16)
    place = st["page_table"].long()[seq, pos // page]
    st["k_pages"][place, :, pos % page] = x[:, hq:]
    st["v_pages"][place, :, pos % page] = heads[:, hq + hkv:]
    return {"q": x[:, :hq].contiguous(), "k_pages": st["k_pages"], "v_pages": st["v_pages"]}


def _plain_attention(st):
    c = st["case"]
    out = torch.empty_like(st["q"])
    lse = torch.empty((st["tokens"], c["hq"]), dtype=torch.float32, device="cuda")
    n_short, t_short = c["short"], c["short"] * c["q_short"]
    if n_short:
        _plain_runs(st, slice(0, n_short), slice(0, t_short), c["q_short"], out, lse)
    if c["long"]:
        _plain_runs(st, slice(n_short, None), slice(t_short, None), c["q_long"], out, lse)
    return {"out": out, "lse": lse}


def _plain_runs(st, seqs, toks, q_len, out, lse):
    """Attention of sequences with q_len query tokens each, keys padded to the longest."""
    c = st["case"]
    hkv, dim, g = c["hkv"], c["dim"], c["hq"] // c["hkv"]
    kv_len = st["kv_len"][seqs].long()
    table = st["page_table"][seqs].long()
    n = table.shape[0]

    def keys(pages):
        return pages[table].transpose(1, 2).reshape(n, hkv, -1, dim).float()

    q = st["q"][toks].view(n, q_len, hkv, g, dim).permute(0, 2, 1, 3, 4).float()
    s = torch.matmul(q.reshape(n, hkv, q_len * g, dim), keys(st["k_pages"]).transpose(2, 3))
    s = s.view(n, hkv, q_len, g, -1) * (1.0 / math.sqrt(dim))
    key = torch.arange(s.shape[-1], device="cuda")
    pos = kv_len[:, None] - q_len + torch.arange(q_len, device="cuda")[None]
    seen = key[None, None] <= pos[..., None]
    s = torch.where(seen[:, None, :, None], s, -math.inf)
    top = s.amax(dim=-1, keepdim=True)
    p = torch.exp(s - top)
    del s
    total = p.sum(dim=-1, keepdim=True)
    live = (key[None] < kv_len[:, None])[:, None, :, None]
    v = torch.where(live, keys(st["v_pages"]), 0.0)
    o = torch.matmul(p.view(n, hkv, q_len * g, -1), v).view(n, hkv, q_len, g, dim) / total
    out[toks] = o.permute(0, 2, 1, 3, 4).reshape(n * q_len, hkv * g, dim).to(torch.bfloat16)
    m = (top + torch.log(total)).squeeze(-1)
    lse[toks] = m.permute(0, 2, 1, 3).reshape(n * q_len, hkv * g)


# ------------------------------------------------------------------ in 64 bits


def exact(case, seed):
    """The outputs from the operators' definitions in 64 bits, row by row or head by head."""
    st = prepare(case, seed)
    return {"norm": _exact_norm, "append": _exact_append, "attention": _exact_attention}[case["op"]](st)


def _exact_norm(st):
    y, res = st["y"].double(), st["residual"].double()
    h, x = torch.empty_like(res), torch.empty_like(res)
    cuts = [0, y.shape[0]] if st["seg_offsets"] is None else st["seg_offsets"].tolist()
    ids = [0] if st["seg_variant"] is None else st["seg_variant"].tolist()
    for lo, hi, v in zip(cuts[:-1], cuts[1:], ids):
        b = y[lo:hi]
        if st["post"] is not None:
            b = b * (b.pow(2).mean(1, keepdim=True) + EPS).rsqrt() * st["post"][v].double()
        if st["gate"] is not None:
            b = b * (st["gate"] if st["gate"].dim() == 1 else st["gate"][lo:hi]).double()
        h[lo:hi] = res[lo:hi] + st["scale"] * b
        x[lo:hi] = h[lo:hi] * (h[lo:hi].pow(2).mean(1, keepdim=True) + EPS).rsqrt() * st["pre"][v].double()
    return {"h": h, "x": x}


def _exact_append(st):
    c = st["case"]
    hq, hkv, dim, rot, page = c["hq"], c["hkv"], c["dim"], c["rot"], c["page"]
    half = rot // 2
    x = st["qkv"].double().view(-1, hq + 2 * hkv, dim)
    kp, vp = st["k_pages"].double(), st["v_pages"].double()
    q = torch.empty((st["tokens"], hq, dim), dtype=torch.float64, device="cuda")
    first = torch.arange(half, device="cuda") * (2 if c["interleaved"] else 1)
    second = first + (1 if c["interleaved"] else half)
    off, lens = st["seq_offsets"].tolist(), st["kv_len"].tolist()
    for s in range(len(lens)):
        lo, hi = off[s], off[s + 1]
        pos = torch.arange(lens[s] - (hi - lo), lens[s], device="cuda")
        w = torch.complex(st["rope"][pos, :half].double(), st["rope"][pos, half:].double())[:, None]
        z = torch.complex(x[lo:hi, :hq + hkv][..., first], x[lo:hi, :hq + hkv][..., second]) * w
        r = x[lo:hi, :hq + hkv].clone()
        r[..., first], r[..., second] = z.real, z.imag
        q[lo:hi] = r[:, :hq]
        at = st["page_table"][s].long()[pos // page]
        kp[at, :, pos % page] = r[:, hq:]
        vp[at, :, pos % page] = x[lo:hi, hq + hkv:]
    return {"q": q, "k_pages": kp, "v_pages": vp}


def _exact_attention(st):
    c = st["case"]
    hq, hkv, dim, page = c["hq"], c["hkv"], c["dim"], c["page"]
    g = hq // hkv
    if work(c)["flops"] > 4e12:
        return None
    out = torch.empty((st["tokens"], hq, dim), dtype=torch.float64, device="cuda")
    lse = torch.empty((st["tokens"], hq), dtype=torch.float64, device="cuda")
    off, lens = st["seq_offsets"].tolist(), st["kv_len"].tolist()
    for s in range(len(lens)):
        lo, hi, n = off[s], off[s + 1], lens[s]
        rows = st["page_table"][s, :-(-n // page)].long()
        later = torch.ones((hi - lo, n), dtype=torch.bool, device="cuda").triu(n - (hi - lo) + 1)
        for h in range(hkv):
            k = st["k_pages"][rows, h].reshape(-1, dim)[:n].double()
            v = st["v_pages"][rows, h].reshape(-1, dim)[:n].double()
            for j in range(h * g, (h + 1) * g):
                a = (st["q"][lo:hi, j].double() @ k.T) / math.sqrt(dim)
                a.masked_fill_(later, -math.inf)
                lse[lo:hi, j] = torch.logsumexp(a, 1)
                out[lo:hi, j] = torch.exp(a - lse[lo:hi, j, None]) @ v
    return {"out": out, "lse": lse}
