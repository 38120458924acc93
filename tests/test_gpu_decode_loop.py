"""The decode loop's parts together (examples/decode_loop.py): a prompt, single tokens,
weights and evictions over several rounds, against the same loop in 64 bits that keeps
every token and leaves out what the cache dropped.

The positions table says which tokens a key head still has.  With those, the attention
is the one of bitdelta_attention's own test, (2^-8 + 2^-18·s_max)·Σ w|v| plus 2^-8 of the value, on the
same bf16 queries, keys and values.  A weight is a sum of at most 200 softmax weights,
each within 2^-17 relative (2^-19·s_max + 2^-21·(1 + s_max + |lse|) with s_max and |lse| below
8, and lse's own 2^-16·(1 + |lse|)): 2^-12 of the sum is allowed.  What is kept has to be heavier than what is dropped, but for that."""
import math
import os
import sys

import pytest
import torch

import bit_weight_delta_gb300 as bd

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))
import decode_loop as ex  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hkv,dim,page", [(8, 2, 64, 16), (8, 1, 128, 32)])
def test_rounds_of_steps_and_evictions(hq, hkv, dim, page):
    prompts, budget, slack, recent, sink = [60, 33, 90], 40, 6, 8, 4
    n, g = len(prompts), hq // hkv
    seqs = ex.Sequences(n, budget, slack, hq, hkv, dim, page)
    cache = ex.LayerCache(seqs.room(max(prompts) + 1), hkv, page, dim)
    for t in (cache.k, cache.v, cache.weights):
        t.fill_(float("nan"))                 # recycled pages
    cache.positions.fill_(-1)
    rope = ex.rope_table(200, dim)
    gen = torch.Generator(device="cuda").manual_seed(dim)
    keys, vals = [None] * n, [None] * n       # of every token ever, [tokens, hkv, dim]
    weight = [torch.zeros((hkv, 0), dtype=torch.float64, device="cuda") for _ in range(n)]
    cuts = 0
    for step in range(30):
        q_len = prompts if step == 0 else [1] * n
        batch = seqs.batch(q_len)
        tokens = sum(q_len)
        qkv = torch.randn((tokens, (hq + 2 * hkv) * dim), generator=gen, device="cuda").to(torch.bfloat16)
        # (append once by itself, for the rotated queries and keys)
        q = bd.bitdelta_kv_append(batch, qkv, rope, cache.k, cache.v, pos_offset=seqs.pos_offset)
        out = cache.attend(batch, qkv, rope, seqs.pos_offset)
        off = [sum(q_len[:i]) for i in range(n + 1)]
        shift = seqs.pos_offset.tolist()
        for s in range(n):
            lo, hi, kv = off[s], off[s + 1], seqs.lens[s]
            first = 0 if keys[s] is None else keys[s].shape[0]
            new = torch.arange(kv - (hi - lo), kv, device="cuda")
            pg = seqs.page_table[s].long()[new // page]
            k, v = cache.k[pg, :, new % page], cache.v[pg, :, new % page]
            # the rotation is that of the token's own position
            x = qkv[lo:hi].view(hi - lo, -1, dim)[:, hq:hq + hkv].double()
            c, sn = rope[first:first + hi - lo].double()[:, None].chunk(2, -1)
            a, b = x.chunk(2, -1)
            want = torch.cat([a * c - b * sn, b * c + a * sn], -1)
            mag = torch.cat([a.abs() + b.abs()] * 2, -1)
            assert ((k.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -22 * mag).all()
            keys[s] = k if first == 0 else torch.cat([keys[s], k])
            vals[s] = v if first == 0 else torch.cat([vals[s], v])
            weight[s] = torch.cat([weight[s], torch.zeros((hkv, hi - lo), dtype=torch.float64,
                                                          device="cuda")], 1)
            slots = torch.arange(kv, device="cuda")
            place = seqs.page_table[s].long()[slots // page]
            for h in range(hkv):
                pos = cache.positions[place, h, slots % page].long()
                assert pos.unique().numel() == kv and int(pos.min()) >= 0
                assert int(pos.max()) == first + hi - lo - 1 == kv + shift[s] - 1
                kk, vv = keys[s][pos, h].double(), vals[s][pos, h].double()
                qq = q[lo:hi, h * g:(h + 1) * g].double().transpose(0, 1)
                a = qq @ kk.T / math.sqrt(dim)
                seen = pos[None] <= torch.arange(first, first + hi - lo, device="cuda")[:, None]
                w = torch.softmax(torch.where(seen, a, -math.inf), -1)
                ref = w @ vv
                s_max = (qq.abs() @ kk.abs().T / math.sqrt(dim)).amax()
                tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -18 * s_max) * (w @ vv.abs())
                got = out[lo:hi, h * g:(h + 1) * g].double().transpose(0, 1)
                assert ((got - ref).abs() <= tol).all(), (step, s, h)
                weight[s][h, pos] += w.sum((0, 1))
                table = cache.weights[place, h, slots % page].double()
                assert ((table - weight[s][h, pos]).abs() <= 2.0 ** -12 * weight[s][h, pos]).all()
        had = [[cache.positions[seqs.page_table[s].long()[torch.arange(seqs.lens[s], device="cuda") // page],
                                h, torch.arange(seqs.lens[s], device="cuda") % page].long()
                for h in range(hkv)] for s in range(n)]
        lens = list(seqs.lens)
        if seqs.cut(batch, [cache], recent, sink):
            cuts += 1
            assert seqs.kv_len.tolist() == seqs.lens == [min(x, budget) for x in lens]
            for s in range(n):
                slots = torch.arange(seqs.lens[s], device="cuda")
                place = seqs.page_table[s].long()[slots // page]
                for h in range(hkv):
                    pos = cache.positions[place, h, slots % page].long()
                    assert pos.unique().numel() == seqs.lens[s]
                    gone = [p for p in had[s][h].tolist() if p not in set(pos.tolist())]
                    assert len(gone) == lens[s] - seqs.lens[s]
                    if not gone:
                        continue
                    total = keys[s].shape[0]
                    assert all(sink <= p < total - recent for p in gone)
                    free = [p for p in pos.tolist() if sink <= p < total - recent]
                    if free:
                        least = weight[s][h, free].min()
                        assert (weight[s][h, gone] <= least * (1 + 2.0 ** -11)).all()
    assert cuts >= 3
    assert bd.bitdelta_check_error() == 0


def test_the_example_runs(capsys):
    ex.main()
    assert "->" in capsys.readouterr().out
