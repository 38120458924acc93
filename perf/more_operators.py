"""The operators at the end of a serving step, as cases that can be timed.

Three operators beside the decoder block's:

  sample   a token per row of logits by temperature, top-k, top-p and min-p, from
           one given random number a row
  weigh    the attention weight that each cached key got from a step's queries,
           added to a table that lies beside the paged cache
  evict    a cache cut to a budget: per key head the protected and the heaviest
           keys stay, and those past the new length move into the freed slots

`run` computes each either in its plain form (elementary torch operations, in 32
bits or, for the sums that a choice hangs on, in 64) or, where `own` is true, by the
calls a user makes.
"""
import math

import numpy as np
import torch

own = False


def listed():
    return [
        # the next token of one conversation
        _sample("sample_1", 1, 32000, 0, "chat"),
        # a decode batch whose requests bring settings of their own, greedy ones among them
        _sample("sample_64", 64, 128000, 0, "mixed"),
        # a large batch without cuts, from logits padded to a multiple of 64 columns
        _sample("sample_500", 500, 99991, 9, "plain"),
        # a decode step of 8 short conversations: latency
        _weigh("weigh_8", 8, 1, 0, 0, 120, 1000, 64, 8, 128, 16),
        # a full decode batch with ragged contexts
        _weigh("weigh_64", 64, 1, 0, 0, 500, 8000, 64, 8, 128, 64),
        # one conversation with a very long context: few rows, one long axis
        _weigh("weigh_1_long", 1, 1, 0, 0, 131071, 131071, 64, 8, 128, 16),
        # 64 requests in two groups, each behind its own long system prompt
        _weigh("weigh_shared_64", 64, 1, 0, 0, 8192 + 37, 8192 + 700, 64, 8, 128, 64, prefix=8192,
               group=32),
        # a long prompt, weighed by its last 64 tokens
        _weigh("weigh_prompt_window", 0, 1, 1, 8192, 8192, 8192, 64, 8, 128, 64, window=64),
        # a prompt weighed by all of its tokens
        _weigh("weigh_prompt", 0, 1, 1, 2048, 2048, 2048, 64, 8, 128, 16),
        # a decode batch back to its budget: the tokens of the last 64 steps at most
        _evict("evict_64", 64, 4097, 4160, 4096, 256, 4, 8, 128, 64),
        # four prompts cut to an eighth
        _evict("evict_prompts", 4, 8192, 8192, 1024, 64, 4, 8, 128, 16),
        # half of a very long context
        _evict("evict_1_long", 1, 131071, 131071, 65536, 1024, 4, 8, 128, 16),
    ]


def _sample(name, rows, vocab, pad, settings):
    return {"name": name, "op": "sample", "rows": rows, "vocab": vocab, "pad": pad,
            "settings": settings}


def _weigh(name, short, q_short, long, q_long, kv_lo, kv_hi, hq, hkv, dim, page, window=0,
           prefix=0, group=0):
    return {"name": name, "op": "weigh", "short": short, "q_short": q_short, "long": long,
            "q_long": q_long, "kv_lo": kv_lo, "kv_hi": kv_hi, "hq": hq, "hkv": hkv, "dim": dim,
            "page": page, "window": window, "prefix": prefix, "group": group}


def _evict(name, seqs, kv_lo, kv_hi, keep, recent, sink, hkv, dim, page):
    return {"name": name, "op": "evict", "short": seqs, "q_short": 1, "long": 0, "q_long": 0,
            "kv_lo": kv_lo, "kv_hi": kv_hi, "keep": keep, "recent": recent, "sink": sink,
            "hq": hkv, "hkv": hkv, "dim": dim, "page": page, "window": 0, "prefix": 0, "group": 0}


def draw(rng):
    def size(lo, hi):  # spread over the logarithm
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    kind = rng.choice(["sample", "sample", "decode", "shared", "mixed", "prompt", "evict", "evict"])
    if kind == "sample":
        vocab = rng.choice([32000, 50257, 64000, 128000, size(300, 260000), size(300, 260000)])
        rows = size(1, max(2, min(2048, 48_000_000 // vocab)))
        c = _sample("", rows, vocab, rng.choice([0, 0, 1, 9, 64]),
                    rng.choice(["chat", "mixed", "plain"]))
        c.pop("name")
        return c
    hq, hkv = rng.choice([(64, 8), (32, 8), (40, 8), (24, 8), (32, 4), (16, 16), (16, 2), (28, 4)])
    dim, page = rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128])
    most = 270000 * 1024 // (hkv * dim)  # keys in all: no more bytes than the largest case
    if kind == "decode":
        n = size(1, 256)
        kv_hi = size(16, max(32, min(131071, most // n)))
        c = _weigh("", n, rng.choice([1, 1, 1, 2]), 0, 0, max(2, kv_hi // rng.choice([1, 3, 10])),
                   kv_hi, hq, hkv, dim, page)
    elif kind == "shared":
        group = rng.choice([2, 8, 16, 33, 64])
        n = group * rng.choice([1, 2, 3])
        prefix = page * max(1, size(256, 16384) // page)
        own_lo = size(1, 200) + 1
        c = _weigh("", n, 1, 0, 0, prefix + own_lo, prefix + own_lo + size(1, 800), hq, hkv, dim,
                   page, prefix=prefix, group=group)
    elif kind == "mixed":
        long, q_long = rng.choice([1, 2, 4]), size(40, 600)
        kv_lo = q_long + size(1, 600)
        c = _weigh("", size(1, 64), 1, long, q_long, kv_lo, kv_lo + size(1, 1500), hq, hkv, dim,
                   page, window=rng.choice([0, 0, 32]))
    elif kind == "prompt":
        q_long, window = size(33, 8192), rng.choice([16, 32, 64, 128])
        if rng.random() < 0.5:
            q_long, window = size(33, 2000), 0
        c = _weigh("", 0, 1, rng.choice([1, 2, 4]) if q_long < 1024 else 1, q_long, q_long,
                   q_long + rng.choice([0, 0, size(1, 2000)]), hq, hkv, dim, page, window=window)
    else:
        n = size(1, 128)
        keep = size(64, max(128, min(65536, most // n // 2)))
        kv_lo = keep + size(1, keep)
        kv_hi = min(131071, kv_lo + rng.choice([0, size(1, 64), keep // 2]))
        c = _evict("", n, min(kv_lo, kv_hi), kv_hi, keep, rng.choice([0, keep // 16, keep // 4]),
                   rng.choice([0, 4, 16]), hkv, dim, page)
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
    if c["op"] == "sample":
        return {"bytes": c["rows"] * (2 * c["vocab"] + 20 + 8), "flops": 4 * c["rows"] * c["vocab"]}
    q, kv = _lengths(c)
    hq, hkv, dim = c["hq"], c["hkv"], c["dim"]
    tables = 4 * (2 * len(q) + 1) + sum(4 * -(-k // c["page"]) for k in kv)
    if c["op"] == "evict":
        keep = [min(c["keep"], k) for k in kv]
        # of the slots past the new length, as many move as the weights' even spread says;
        # those of the last tokens all do
        moved = 0.0
        for k, n in zip(kv, keep):
            late = min(c["recent"], k - n)
            moved += late + (k - n - late) * max(0, n - c["recent"] - c["sink"]) / max(
                1, k - c["recent"] - c["sink"])
        return {"bytes": hkv * (8 * sum(kv) + 8 * sum(keep) + int(moved) * 8 * dim) + tables,
                "flops": hkv * sum(kv)}
    groups = len(q) // c["group"] if c["prefix"] else 0
    keys = sum(kv) - (len(q) - groups) * c["prefix"]
    rows = [min(a, c["window"]) if c["window"] else a for a in q]
    seen = sum(r * (k - r) + r * (r + 1) // 2 for r, k in zip(rows, kv))
    return {"bytes": sum(rows) * hq * (2 * dim + 4) + keys * hkv * (2 * dim + 8) + tables,
            "flops": 2 * seen * hq * dim}


# ------------------------------------------------------------------ inputs


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    def uniform(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    if c["op"] == "sample":
        return _prepare_sample(c, normal, uniform)
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
        # tokens that earlier evictions took from the sequences
        "pos_offset": torch.from_numpy(rng.integers(0, 5000, n).astype(np.int32)).cuda(),
        # every page holds values: a recycled cache is full of earlier tokens
        "k_pages": normal(n_pages, hkv, page, dim, std=1.2),
        # sums of softmax weights: a few heavy keys, many that hardly count, some never looked at
        "weights": torch.relu(torch.exp(2.0 * torch.randn(
            (n_pages, hkv, page), generator=g, device="cuda") - 3.0) - 0.01),
    }
    at = state["pos_offset"].long()[:, None] + torch.arange(
        table.shape[1] * page, device="cuda").view(1, -1)
    state["positions"] = torch.zeros((n_pages, hkv, page), dtype=torch.int32, device="cuda")
    if c["op"] == "evict":
        state["v_pages"] = normal(n_pages, hkv, page, dim)
        state["keep"] = torch.full((n,), c["keep"], dtype=torch.int32, device="cuda")
        # positions in the order of the slots, as after a prompt, the first ones low
        at = torch.where(torch.arange(at.shape[1], device="cuda") < c["sink"],
                         at - state["pos_offset"].long()[:, None], at)
        live = torch.arange(table.shape[1], device="cuda") * page < state["kv_len"][:, None]
        state["positions"][state["page_table"].long()[live]] = at.view(
            n, -1, page)[live][:, None].to(torch.int32)
        # the tables after the eviction: a server keeps the old ones until its step is through
        state["weights_out"] = torch.zeros_like(state["weights"])
        state["positions_out"] = torch.zeros_like(state["positions"])
    else:
        state["q"] = normal(tokens, hq, dim, std=1.5)
        # what the attention left of its softmax; rows outside of the window are not looked at
        state["lse"] = torch.full((tokens, hq), 12.0, device="cuda")
        for toks, seqs, q_rows in _runs(c):
            s, _ = _scores(state, toks, seqs, q_rows)
            top = s.amax(dim=-1)
            lse = top + torch.log(torch.exp(s - top[..., None]).sum(dim=-1))
            del s
            state["lse"][toks] = lse.permute(0, 2, 1, 3).reshape(-1, hq)
        if prefix:
            state["group_offsets"] = torch.arange(0, n + 1, c["group"], device="cuda",
                                                  dtype=torch.int32)
            state["prefix_len"] = torch.full((n // c["group"],), prefix, device="cuda",
                                             dtype=torch.int32)
    if own:  # a serving loop keeps the batch for all layers of a step
        import bit_weight_delta_gb300 as bd
        state["batch"] = bd.AttentionBatch(
            state["seq_offsets"], state["kv_len"], state["page_table"], n_tokens=tokens,
            max_q_len=int(q_len.max()), max_kv_len=int(kv_len.max()), n_q_heads=hq,
            n_kv_heads=hkv, head_dim=dim, page_size=page,
            group_offsets=state.get("group_offsets"), prefix_len=state.get("prefix_len"))
    return state


def _prepare_sample(c, normal, uniform):
    rows, vocab = c["rows"], c["vocab"]
    # rows of a language model's head: a broad bulk, some rows sharper than others, a few
    # candidates well above it
    spread = 1.5 + 2.0 * uniform(rows, 1)
    logits = normal(rows, vocab + c["pad"], dtype=torch.float32) * spread
    place = (uniform(rows, 8) * vocab).long()
    logits.scatter_add_(1, place, 4.0 + 10.0 * uniform(rows, 8))
    # every eighth row is held to a grammar: nine tenths of its tokens are masked
    masked = (torch.arange(rows, device="cuda") % 8 == 5)[:, None] & (
        uniform(rows, vocab + c["pad"]) < 0.9)
    logits = torch.where(masked, -math.inf, logits).to(torch.bfloat16)
    state = {"case": c, "logits": logits[:, :vocab], "u": uniform(rows), "temperature": None,
             "top_k": None, "top_p": None, "min_p": None}
    if c["settings"] == "chat":
        state["temperature"] = torch.full((rows,), 0.8, device="cuda")
        state["top_k"] = torch.full((rows,), 50, dtype=torch.int32, device="cuda")
        state["top_p"] = torch.full((rows,), 0.95, device="cuda")
    elif c["settings"] == "mixed":
        t = 0.5 + uniform(rows)
        state["temperature"] = torch.where(uniform(rows) < 0.2, 0.0, t)
        k = (1.0 + 100.0 * uniform(rows)).to(torch.int32)
        state["top_k"] = torch.where(uniform(rows) < 0.5, 0, k).to(torch.int32)
        p = 0.5 + 0.5 * uniform(rows)
        state["top_p"] = torch.where(uniform(rows) < 0.4, 1.0, p)
        state["min_p"] = torch.where(uniform(rows) < 0.6, 0.0, 0.1 * uniform(rows))
    return state


# ------------------------------------------------------------------ one pass


def run(state):
    op = state["case"]["op"]
    if own:
        import bit_weight_delta_gb300 as bd
        if op == "sample":
            tokens, prob = bd.bitdelta_sample(
                state["logits"], state["u"], temperature=state["temperature"],
                top_k=state["top_k"], top_p=state["top_p"], min_p=state["min_p"])
            return {"tokens": tokens, "prob": prob}
        if op == "weigh":
            weights, positions = bd.bitdelta_kv_weigh(
                state["batch"], state["q"], state["lse"], state["k_pages"], state["weights"],
                state["positions"], window=state["case"]["window"],
                pos_offset=state["pos_offset"])
            return {"weights": weights, "positions": positions}
        weights, positions = bd.bitdelta_kv_evict(
            state["batch"], state["keep"], state["k_pages"], state["v_pages"], state["weights"],
            state["positions"], recent=state["case"]["recent"], sink=state["case"]["sink"],
            pos_offset=state["pos_offset"], weights_out=state["weights_out"],
            positions_out=state["positions_out"])
        return {"weights": weights, "positions": positions, "k_pages": state["k_pages"],
                "v_pages": state["v_pages"]}
    return {"sample": _plain_sample, "weigh": _plain_weigh, "evict": _plain_evict}[op](state)


def _plain_sample(st):
    """In 64 bits: a choice hangs on sums over the whole row."""
    x = st["logits"].double()
    rows, vocab = x.shape
    one = torch.ones(rows, device="cuda", dtype=torch.float64)
    t = one if st["temperature"] is None else st["temperature"].double()
    k = torch.full((rows,), vocab, device="cuda")
    if st["top_k"] is not None:
        k = torch.where(st["top_k"] > 0, st["top_k"].long().clamp(max=vocab), k)
    k = torch.where(t > 0, k, 1)
    top_p = one if st["top_p"] is None else st["top_p"].double()
    min_p = 0.0 * one if st["min_p"] is None else st["min_p"].double()
    value, order = torch.sort(x, dim=1, descending=True, stable=True)
    w = torch.exp((value - value[:, :1]) / torch.where(t > 0, t, 1.0)[:, None])
    total = torch.cumsum(w, dim=1)
    at_k = total.gather(1, k[:, None] - 1)
    n_p = (total < top_p[:, None] * at_k).sum(dim=1) + 1
    n = torch.minimum(k, torch.where(top_p < 1.0, n_p, vocab))
    n = torch.minimum(n, (w >= min_p[:, None]).sum(dim=1))
    kept = total.gather(1, n[:, None] - 1)
    pick = (total <= st["u"].double()[:, None] * kept).sum(dim=1)
    pick = torch.minimum(pick, n - 1)[:, None]
    return {"tokens": order.gather(1, pick)[:, 0].to(torch.int32),
            "prob": (w.gather(1, pick) / kept)[:, 0].float()}


def _runs(c):
    """Token and sequence ranges of the short and the long sequences, and the query tokens that
    count of each."""
    ns, ts = c["short"], c["short"] * c["q_short"]
    runs = []
    if ns:
        runs.append((slice(0, ts), slice(0, ns), c["q_short"]))
    if c["long"]:
        runs.append((slice(ts, None), slice(ns, None), c["q_long"]))
    out = []
    for toks, seqs, q_len in runs:
        rows = min(q_len, c["window"]) if c["window"] else q_len
        n = c["short"] if seqs.stop is not None else c["long"]
        t = torch.arange(toks.start, toks.start + n * q_len, device="cuda").view(n, q_len)
        out.append((t[:, q_len - rows:].reshape(-1), seqs, rows))
    return out


def _scores(st, toks, seqs, rows, key_dtype=torch.float32):
    """Scaled scores [n, hkv, rows, g, keys] of sequences with `rows` query tokens each that
    count, minus infinity where a query does not see the key, and their page tables."""
    c = st["case"]
    hkv, dim, g = c["hkv"], c["dim"], c["hq"] // c["hkv"]
    kv_len, table = st["kv_len"][seqs].long(), st["page_table"][seqs].long()
    n = table.shape[0]
    k = st["k_pages"][table].transpose(1, 2).reshape(n, hkv, -1, dim).to(key_dtype)
    q = st["q"][toks].view(n, rows, hkv, g, dim).permute(0, 2, 1, 3, 4).to(key_dtype)
    s = torch.matmul(q.reshape(n, hkv, rows * g, dim), k.transpose(2, 3))
    s = s.view(n, hkv, rows, g, -1) * (1.0 / math.sqrt(dim))
    key = torch.arange(s.shape[-1], device="cuda")
    pos = kv_len[:, None] - rows + torch.arange(rows, device="cuda")[None]
    seen = key[None, None] <= pos[..., None]
    return torch.where(seen[:, None, :, None], s, -math.inf), table


def _plain_weigh(st):
    c = st["case"]
    page, hkv, g = c["page"], c["hkv"], c["hq"] // c["hkv"]
    off = st["seq_offsets"].long()
    # the step's own tokens: their slots begin at zero, and get their positions
    tok = torch.arange(st["tokens"], device="cuda")
    seq = (tok[:, None] >= off[None, 1:]).sum(dim=1)
    slot = st["kv_len"].long()[seq] - (off[seq + 1] - tok)
    place = st["page_table"].long()[seq, slot // page]
    st["weights"][place, :, slot % page] = 0.0
    st["positions"][place, :, slot % page] = (slot + st["pos_offset"].long()[seq]).to(
        torch.int32)[:, None]
    for toks, seqs, rows in _runs(c):
        s, table = _scores(st, toks, seqs, rows)
        n, keys = table.shape[0], s.shape[-1]
        lse = st["lse"][toks].view(n, rows, hkv, g).transpose(1, 2)
        got = torch.exp(s - lse[..., None]).sum(dim=(2, 3))
        del s
        key = torch.arange(keys, device="cuda")
        live = key[None] < st["kv_len"][seqs].long()[:, None]
        where = (table[:, key // page] * page + key % page)[live]
        flat = st["weights"].transpose(1, 2).reshape(-1, hkv)
        flat.index_put_((where,), got.transpose(1, 2)[live], accumulate=True)
        st["weights"].copy_(flat.view(-1, page, hkv).transpose(1, 2))
    return {"weights": st["weights"], "positions": st["positions"]}


def _plain_evict(st):
    c = st["case"]
    page, hkv = c["page"], c["hkv"]
    table, kv = st["page_table"].long(), st["kv_len"].long()
    n, slots = table.shape[0], table.shape[1] * page
    keep = torch.minimum(st["keep"].long(), kv)[:, None, None]
    slot = torch.arange(slots, device="cuda").expand(n, hkv, slots)

    def rows(pages):  # [n, hkv, slots] of a table beside the cache
        return pages[table].transpose(1, 2).reshape(n, hkv, slots)

    weight, position = rows(st["weights"]), rows(st["positions"])
    live = slot < kv[:, None, None]
    late = (kv + st["pos_offset"].long())[:, None, None] - c["recent"]
    held = (position >= late) | (position < c["sink"])
    rank = torch.where(held, math.inf, weight)
    rank = torch.where(live, rank, -1.0)
    order = torch.sort(rank, dim=2, descending=True, stable=True)[1]
    kept = torch.zeros_like(live).scatter_(2, order, slot < keep)
    hole = (slot < keep) & ~kept
    mover = (slot >= keep) & kept
    # the i-th mover's slot, and for each hole its own number
    number = torch.cumsum(mover, dim=2) - 1
    source = torch.zeros((n, hkv, slots), dtype=torch.int64, device="cuda")
    source.scatter_(2, torch.where(mover, number, slots - 1), torch.where(mover, slot, 0))
    source = torch.where(hole, source.gather(2, (torch.cumsum(hole, dim=2) - 1).clamp(min=0)), slot)
    seq = torch.arange(n, device="cuda")[:, None, None].expand(n, hkv, slots)
    head = torch.arange(hkv, device="cuda")[None, :, None].expand(n, hkv, slots)
    out = (slot < keep).nonzero(as_tuple=True)
    s, h, to, src = seq[out], head[out], slot[out], source[out]
    place, frm = (table[s, to // page], h, to % page), (table[s, src // page], h, src % page)
    st["weights_out"][place] = st["weights"][frm]
    st["positions_out"][place] = st["positions"][frm]
    moved = to != src
    place, frm = (tuple(i[moved] for i in p) for p in (place, frm))
    st["k_pages"][place] = st["k_pages"][frm]
    st["v_pages"][place] = st["v_pages"][frm]
    return {"weights": st["weights_out"], "positions": st["positions_out"],
            "k_pages": st["k_pages"], "v_pages": st["v_pages"]}


# ------------------------------------------------------------------ in 64 bits


def exact(case, seed):
    """The outputs from the operators' definitions in 64 bits, row by row or head by head."""
    st = prepare(case, seed)
    return {"sample": _exact_sample, "weigh": _exact_weigh, "evict": _exact_evict}[case["op"]](st)


def _exact_sample(st):
    rows, vocab = st["logits"].shape
    tokens = torch.zeros(rows, dtype=torch.int32, device="cuda")
    prob = torch.zeros(rows, dtype=torch.float64, device="cuda")

    def setting(name, row, default):
        return default if st[name] is None else st[name][row].item()

    for r in range(rows):
        x = st["logits"][r].double()
        t = setting("temperature", r, 1.0)
        if t == 0.0:
            tokens[r], prob[r] = int((x == x.max()).nonzero()[0]), 1.0
            continue
        order = torch.argsort(-x, stable=True)
        w = torch.exp((x[order] - x.max()) / t)
        k = setting("top_k", r, 0)
        if k > 0:
            w[k:] = 0.0
        p = setting("top_p", r, 1.0)
        if p < 1.0:  # a token stays while those before it have not reached p
            before = torch.cumsum(w, 0) - w
            w[before >= p * w.sum()] = 0.0
        w[w < setting("min_p", r, 0.0)] = 0.0
        total = torch.cumsum(w, 0)
        i = int(torch.searchsorted(total, total[-1] * st["u"][r].item(), right=True))
        i = min(i, int((w > 0).sum()) - 1)
        tokens[r], prob[r] = int(order[i]), w[i] / total[-1]
    return {"tokens": tokens, "prob": prob}


def _exact_weigh(st):
    c = st["case"]
    hkv, dim, page, g = c["hkv"], c["dim"], c["page"], c["hq"] // c["hkv"]
    weights, positions = st["weights"].double(), st["positions"].clone()
    off, kv, shift = (st[n].tolist() for n in ("seq_offsets", "kv_len", "pos_offset"))
    for s, n in enumerate(kv):  # new slots first: a shared page may hold another's sums
        slot = torch.arange(n - (off[s + 1] - off[s]), n, device="cuda")
        place = st["page_table"][s].long()[slot // page]
        weights[place, :, slot % page] = 0.0
        positions[place, :, slot % page] = (slot + shift[s]).to(torch.int32)[:, None]
    for s, n in enumerate(kv):
        lo, hi = off[s], off[s + 1]
        if c["window"]:
            lo = max(lo, hi - c["window"])
        slot = torch.arange(n, device="cuda")
        place = st["page_table"][s].long()[slot // page]
        seen = slot[None] <= torch.arange(n - (hi - lo), n, device="cuda")[:, None]
        for h in range(hkv):
            k = st["k_pages"][place, h, slot % page].double()
            got = torch.zeros(n, dtype=torch.float64, device="cuda")
            for i in range(h * g, (h + 1) * g):
                a = st["q"][lo:hi, i].double() @ k.T / math.sqrt(dim)
                a = torch.exp(a - st["lse"][lo:hi, i].double()[:, None])
                got += torch.where(seen, a, 0.0).sum(0)
            weights[place, h, slot % page] += got
    return {"weights": weights, "positions": positions}


def _exact_evict(st):
    c = st["case"]
    page = c["page"]
    w_in, p_in = st["weights"].cpu().numpy(), st["positions"].cpu().numpy()
    table, kv, shift = (st[n].cpu().numpy() for n in ("page_table", "kv_len", "pos_offset"))
    frm, to = [], []
    for s in range(len(kv)):
        slot = np.arange(kv[s])
        place = table[s][slot // page].astype(np.int64)
        keep = min(c["keep"], int(kv[s]))
        for h in range(c["hkv"]):
            w, p = w_in[place, h, slot % page], p_in[place, h, slot % page]
            held = (p >= kv[s] + shift[s] - c["recent"]) | (p < c["sink"])
            stay = np.sort(np.lexsort((slot, -w.astype(np.float64), ~held))[:keep])
            src = np.arange(keep)
            src[np.setdiff1d(src, stay)] = stay[stay >= keep]
            frm.append((place[src] * c["hkv"] + h) * page + src % page)
            to.append((place[:keep] * c["hkv"] + h) * page + np.arange(keep) % page)
    frm, to = (torch.from_numpy(np.concatenate(v)).cuda() for v in (frm, to))
    out = {}
    for name, table_out in (("weights", "weights_out"), ("positions", "positions_out"),
                            ("k_pages", "k_pages"), ("v_pages", "v_pages")):
        flat = st[name].reshape(-1, c["dim"]) if name.endswith("pages") else st[name].reshape(-1)
        new = st[table_out].reshape(flat.shape).clone()
        new[to] = flat[frm]
        new = new.view(st[name].shape)
        out[name] = new.double() if new.is_floating_point() else new
    return out
