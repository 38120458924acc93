"""bitdelta_attention against the softmax in 64 bits.

Tolerances (derived before the first run).  A score is an fp32 sum of head_dim
exact products: off by at most 2^-19 of s_max = scale·max_k Σ|q·k|, which moves
each weight by that relative amount, and the normalised weights by twice it.
Weights are rounded to bf16 (half an ulp, 2^-9) for the product with v: with
the factor two for both effects' sums, out is within (2^-8 + 2^-18·s_max)·Σ w|v|
plus the output's own rounding, 2^-8 of the value.  The denominator is summed
in fp32 from unrounded weights: lse within 2^-18·s_max + 2^-16·(1 + |lse|)."""
import math

import numpy as np
import pytest
import torch

import bit_weight_delta_gb300 as bd

pytestmark = pytest.mark.gpu
NAN = float("nan")


class Case:
    """lens: (query tokens, keys) per sequence; groups: (sequences, shared prefix)."""

    def __init__(self, lens, hq=8, hkv=2, dim=128, page=16, groups=(), seed=0, std=1.0,
                 extra_tokens=0, spare=3):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.hq, self.hkv, self.dim, self.page = lens, hq, hkv, dim, page
        n = len(lens)
        self.off = np.concatenate([[0], np.cumsum([q for q, _ in lens])]).astype(np.int32)
        self.kv = np.array([k for _, k in lens], np.int32)
        need = [-(-int(k) // page) for k in self.kv]
        lead = {}                       # sequence -> (first member, shared pages)
        s0, offs, pre = 0, [0], []
        for cnt, prefix in groups:
            for s in range(s0 + 1, s0 + cnt):
                lead[s] = (s0, prefix // page)
            s0 += cnt
            offs.append(s0)
            pre.append(prefix)
        fresh = [need[s] - lead.get(s, (0, 0))[1] for s in range(n)]
        n_pages = sum(fresh) + spare
        order = rng.permutation(n_pages)
        self.table = np.full((n, max(need + [1]) + 1), 2 ** 30, np.int32)   # past kv_len: unread
        u = 0
        for s in range(n):
            first, sh = lead.get(s, (s, 0))
            self.table[s, :sh] = self.table[first, :sh]
            self.table[s, sh:need[s]] = order[u:u + fresh[s]]
            u += fresh[s]
        self.t = int(self.off[-1]) + extra_tokens

        def rn(*shape):
            return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)

        self.q = rn(self.t, hq, dim)
        self.kp = torch.full((n_pages, hkv, page, dim), NAN, dtype=torch.bfloat16, device="cuda")
        self.vp = self.kp.clone()
        for s in range(n):              # NaN stays wherever no key is
            for i in range(need[s]):
                m = min(page, int(self.kv[s]) - i * page)
                self.kp[self.table[s, i], :, :m] = rn(hkv, m, dim)
                self.vp[self.table[s, i], :, :m] = rn(hkv, m, dim)
        kw = {}
        if groups:
            kw = {"group_offsets": torch.tensor(offs, dtype=torch.int32).cuda(),
                  "prefix_len": torch.tensor(pre, dtype=torch.int32).cuda()}
        self.make = lambda **over: bd.AttentionBatch(
            torch.from_numpy(self.off).cuda(), torch.from_numpy(self.kv).cuda(),
            torch.from_numpy(self.table).cuda(), **{**dict(
                n_tokens=self.t, max_q_len=max([q for q, _ in lens], default=0),
                max_kv_len=int(self.kv.max(initial=0)), n_q_heads=hq, n_kv_heads=hkv,
                head_dim=dim, page_size=page), **kw, **over})
        self.batch = self.make()

    def run(self, **kw):
        return bd.bitdelta_attention(self.batch, self.q, self.kp, self.vp, **kw)

    def check(self, out, lse, scale=None, seqs=None):
        scale = 1.0 / math.sqrt(self.dim) if scale is None else scale
        g = self.hq // self.hkv
        assert torch.isfinite(out.float()).all()
        for s in range(len(self.lens)) if seqs is None else seqs:
            lo, hi, n = int(self.off[s]), int(self.off[s + 1]), int(self.kv[s])
            if hi == lo:
                continue
            o_got, l_got = out[lo:hi].double(), lse[lo:hi].double()
            ql = hi - lo
            keys = torch.arange(n, device="cuda")
            pos = n - ql + torch.arange(ql, device="cuda")
            seen = keys[None] <= pos[:, None]
            pages = torch.from_numpy(self.table[s, :-(-n // self.page)].astype(np.int64)).cuda()
            for h in range(self.hkv):
                k = self.kp[pages, h].reshape(-1, self.dim)[:n].double()
                v = self.vp[pages, h].reshape(-1, self.dim)[:n].double()
                q = self.q[lo:hi, h * g:(h + 1) * g].double().transpose(0, 1)
                a = torch.where(seen, q @ k.T * scale, -math.inf)
                s_max = (q.abs() @ k.abs().T * scale).amax(-1, keepdim=True) if n else 0.0
                ref_l = torch.logsumexp(a, -1, keepdim=True) if n else torch.full(
                    (g, ql, 1), -math.inf, device="cuda", dtype=torch.float64)
                w = torch.where(seen, torch.exp(a - ref_l), 0.0)
                ref = w @ v
                empty = ~torch.isfinite(ref_l)
                tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -18 * s_max) * (w @ v.abs())
                got = o_got[:, h * g:(h + 1) * g].transpose(0, 1)
                bad = (got - torch.where(empty, 0.0, ref)).abs() > torch.where(empty, 0.0, tol)
                assert not bad.any(), (s, h, int(bad.sum()), (got - ref).abs().max().item())
                got_l = l_got[:, h * g:(h + 1) * g].transpose(0, 1).unsqueeze(-1)
                assert (torch.isneginf(got_l) == empty).all()
                lerr = torch.where(empty, 0.0, (got_l - ref_l).abs())
                ltol = 2.0 ** -18 * s_max + 2.0 ** -16 * (1 + torch.where(empty, 0.0, ref_l).abs())
                assert (lerr <= ltol).all(), (s, h, lerr.max().item())
        # tokens of no sequence
        assert (out[int(self.off[-1]):] == 0).all()
        assert torch.isneginf(lse[int(self.off[-1]):]).all()
        assert bd.bitdelta_check_error() == 0


HEADS = [(8, 1, 128), (8, 8, 64), (6, 2, 128), (10, 2, 64), (32, 1, 128), (14, 2, 128)]


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("hq,hkv,dim", HEADS)
def test_single_tokens(hq, hkv, dim, page):
    lens = [(1, k) for k in (1, 2, 15, 16, 17, 31, 33, 64, 65, 127, 128, 129, 300, 1000)]
    c = Case(lens, hq, hkv, dim, page, seed=page)
    c.check(*c.run())


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("hq,hkv,dim", HEADS)
def test_prompts_from_their_start(hq, hkv, dim, page):
    lens = [(q, q) for q in (1, 2, 7, 16, 31, 33, 64, 100, 129, 257)]
    c = Case(lens, hq, hkv, dim, page, seed=page + 1)
    c.check(*c.run())


@pytest.mark.parametrize("page", [16, 32, 128])
@pytest.mark.parametrize("hq,hkv,dim", HEADS)
def test_chunks_behind_earlier_context(hq, hkv, dim, page):
    lens = [(33, 40), (2, 500), (100, 333), (1, 77), (64, 1024), (130, 131), (3, 3), (5, 260)]
    c = Case(lens, hq, hkv, dim, page, seed=page + 2)
    c.check(*c.run())


@pytest.mark.parametrize("hq,hkv,dim,page", [(8, 1, 128, 16), (8, 8, 64, 32), (6, 2, 128, 64),
                                             (16, 2, 128, 128), (32, 2, 64, 16)])
def test_shared_prefixes(hq, hkv, dim, page):
    """Groups of every size, prefixes from nothing to long ones, members of unlike
    query lengths, and sequences of no group behind them."""
    p1, p2, p3 = 256, 1024, 640
    lens = ([(1, p1 + i + 1) for i in range(40)] + [(1, p2 + 3), (90, p2 + 90), (2, p2 + 400)]
            + [(1, p3 + 1)] + [(1, 50), (1, 60)] + [(4, p1 + 37 * i + 4) for i in range(9)]
            + [(1, 5), (20, 300)])
    groups = [(40, p1), (3, p2), (1, p3), (2, 0), (9, p1)]
    c = Case(lens, hq, hkv, dim, page, groups=groups, seed=page + 3)
    c.check(*c.run())
    # the groups change how it is computed, not what
    plain = c.make(group_offsets=None, prefix_len=None)
    o2, l2 = bd.bitdelta_attention(plain, c.q, c.kp, c.vp)
    c.check(o2, l2)


@pytest.mark.parametrize("hq,hkv,dim", [(8, 1, 128), (16, 2, 64)])
def test_one_long_context(hq, hkv, dim):
    """Few rows and one long axis: the split over keys and its join."""
    c = Case([(1, 20011)], hq, hkv, dim, 64, seed=5)
    c.check(*c.run())
    c = Case([(40, 9000)], hq, hkv, dim, 32, seed=6)
    c.check(*c.run())


@pytest.mark.parametrize("hq,hkv,dim", [(32, 1, 128), (32, 1, 64), (20, 1, 128), (9, 1, 128)])
def test_one_long_context_of_many_heads(hq, hkv, dim):
    """Hundreds of parts per row, whose join is cut by rows as well."""
    c = Case([(1, 9001)], hq, hkv, dim, 64, seed=31)
    out, lse = c.run()
    c.check(out, lse)
    assert torch.equal(out, c.run()[0])


@pytest.mark.parametrize("hq,hkv,q", [(40, 2, 1), (16, 2, 4)])
def test_about_as_many_uneven_tiles_as_ctas(hq, hkv, q):
    """Tiles of 1 to 24 blocks, which are cut to half of a CTA's share."""
    c = Case([(q, 4 + 41 * s) for s in range(74)], hq, hkv, 128, 32, seed=32)
    c.check(*c.run())


def test_many_sequences():
    rng = np.random.default_rng(3)
    lens = [(1, int(k)) for k in rng.integers(1, 700, 300)]
    c = Case(lens, 8, 2, 64, 32, seed=7)
    c.check(*c.run())


def test_larger_scores_and_another_scale():
    c = Case([(1, 400), (70, 300), (5, 64)], 8, 2, 128, 16, seed=8, std=4.0)
    c.check(*c.run())
    c.check(*c.run(scale=0.01), scale=0.01)
    c.check(*c.run(scale=2.0), scale=2.0)


def test_rising_scores():
    """Each key scores higher than the last by a wide step, so the running maximum
    moves in every tile and the sums are rescaled each time."""
    c = Case([(1, 700), (64, 700)], 4, 1, 128, 16, seed=9)
    c.q.zero_()
    c.q[:, :, 0] = 8.0
    c.kp.nan_to_num_(0.0).mul_(0.0)
    for s in range(2):
        for k in range(700):
            c.kp[c.table[s, k // 16], 0, k % 16, 0] = k * 0.5
    c.check(*c.run())


def test_empty_rows():
    """Sequences without keys, tokens at negative positions, sequences without
    tokens, tokens of no sequence."""
    c = Case([(1, 0), (0, 10), (3, 2), (60, 20), (0, 0), (2, 2), (1, 40)], 8, 2, 128, 16, seed=10,
             extra_tokens=3)
    out, lse = c.run()
    c.check(out, lse)
    assert (out[0] == 0).all() and (out[1] == 0).all()       # 3 tokens, 2 keys: the first is empty


def test_nothing_to_do():
    c = Case([], 8, 2, 128, 16)
    out, lse = c.run()
    assert out.shape == (0, 8, 128) and lse.shape == (0, 8)


@pytest.mark.parametrize("max_q", [1, 64])
def test_tokens_without_any_sequence(max_q):
    """A batch of padding alone writes zeros, in either kernel."""
    c = Case([], 8, 2, 128, 16, extra_tokens=5)
    c.batch = c.make(max_q_len=max_q, max_kv_len=64)
    out = torch.full((5, 8, 128), NAN, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((5, 8), NAN, device="cuda")
    c.run(out=out, lse=lse)
    assert (out == 0).all() and torch.isneginf(lse).all()
    assert bd.bitdelta_check_error() == 0


def test_infinite_and_nan_keys_behind_the_mask():
    """Pages past kv_len and the last page's tail hold NaN in every test here; infinities
    behave the same."""
    c = Case([(1, 17), (50, 50), (1, 129)], 8, 2, 128, 64, seed=11)
    want = c.run()
    c.kp.nan_to_num_(nan=float("inf"))
    c.vp.nan_to_num_(nan=float("-inf"))
    got = c.run()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    c.check(*got)


def test_repeatable_on_streams_and_in_a_graph():
    lens = [(1, 900 + 16 * i) for i in range(40)] + [(100, 500)]
    c = Case(lens, 16, 2, 128, 16, groups=[(40, 512)], seed=12)
    o, l = c.run()
    for _ in range(3):
        o1, l1 = c.run()
        assert torch.equal(o, o1) and torch.equal(l, l1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o1, l1 = c.run(stream=s)
    s.synchronize()
    assert torch.equal(o, o1) and torch.equal(l, l1)
    o2, l2 = torch.zeros_like(o), torch.zeros_like(l)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.batch.plan()
        c.run(out=o2, lse=l2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(l, l2)


def test_new_lengths_in_the_same_batch():
    """plan() again after the lengths changed in place, as in a decode loop."""
    c = Case([(1, 300), (1, 200)], 8, 2, 128, 16, seed=13)
    c.check(*c.run())
    kv = c.batch._keep[1]
    kv.copy_(torch.tensor([250, 7], dtype=torch.int32))
    c.kv[:] = [250, 7]
    c.batch.plan()
    c.check(*c.run())


def test_a_cache_past_32_bits():
    hkv, page, dim = 8, 128, 128
    n_pages = (2 ** 32) // (hkv * page * dim) + 8
    c = Case([(1, 200), (40, 300)], 16, hkv, dim, page, seed=14)
    kp = torch.full((n_pages, hkv, page, dim), NAN, dtype=torch.bfloat16, device="cuda")
    vp = torch.full_like(kp, NAN)
    have = c.kp.shape[0]
    kp[-have:], vp[-have:] = c.kp, c.vp
    want = c.run()
    c.check(*want)
    c.table = np.where(c.table < have, c.table + n_pages - have, c.table).astype(np.int32)
    got = bd.bitdelta_attention(c.make(), c.q, kp, vp)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_bad_tables_are_reported():
    c = Case([(1, 100), (40, 64)], 8, 2, 128, 16, seed=15)
    c.table[0, 3] = c.kp.shape[0]                 # one page too far
    bd.bitdelta_attention(c.make(), c.q, c.kp, c.vp)
    assert bd.bitdelta_check_error() == 7
    c.table[0, 3] = -1
    bd.bitdelta_attention(c.make(), c.q, c.kp, c.vp)
    assert bd.bitdelta_check_error() == 7
    for over in (dict(max_q_len=39), dict(max_kv_len=99)):
        c.make(**over)
        assert bd.bitdelta_check_error() == 7
    c.off[1] = 50                                 # not sorted
    c.make()
    assert bd.bitdelta_check_error() == 7


@pytest.mark.parametrize("units", [33, 66, 132, 264, 528, 565, 607])
@pytest.mark.parametrize("hq,dim", [(24, 128), (8, 64)])
def test_groups_that_share_nothing(hq, dim, units):
    """A batch whose every prefix is empty has work for one of the two roles
    only: all CTAs and no more are that role's (152·x/x in 32 bits is a little
    above 152 for these numbers of 16-key units)."""
    c = Case([(1, 16 * units)], hq, 1, dim, 32, groups=[(1, 0)], seed=23)
    out, lse = c.run()
    c.check(out, lse)
    again, lse2 = c.run()
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    assert bd.bitdelta_check_error() == 0


def test_a_prefix_longer_than_a_member_is_cut():
    """prefix_len past a member's earlier context counts only as far as all members have it."""
    lens = [(1, 64 + 1 + i) for i in range(40)]
    c = Case(lens, 8, 1, 128, 16, groups=[(40, 64)], seed=16)
    batch = c.make(prefix_len=torch.tensor([4096], dtype=torch.int32).cuda())
    c.check(*bd.bitdelta_attention(batch, c.q, c.kp, c.vp))


def test_refusals():
    c = Case([(1, 30)], 8, 2, 128, 16)
    for kw in (dict(q=c.q.float()), dict(q=c.q[:, :4].contiguous()), dict(kp=c.kp.float()),
               dict(kp=c.kp[:, :1].contiguous()), dict(out=c.q.float()),
               dict(lse=torch.zeros((1, 4), device="cuda"))):
        a = {"q": c.q, "kp": c.kp, **kw}
        with pytest.raises(ValueError):
            bd.bitdelta_attention(c.batch, a["q"], a["kp"], c.vp, out=a.get("out"),
                                  lse=a.get("lse"))
    for scale in (0.0, -1.0, math.inf, NAN):
        with pytest.raises(bd.BitDeltaError):
            c.run(scale=scale)
    for over in (dict(page_size=8), dict(head_dim=96), dict(n_q_heads=7), dict(n_q_heads=66)):
        with pytest.raises(bd.BitDeltaError):
            c.make(**over)
    with pytest.raises(ValueError):
        c.make(prefix_len=torch.zeros(1, dtype=torch.int32).cuda())


def test_ranges_cut_in_every_way():
    """Very unlike lengths: runs that span many CTAs, runs that share one with others, and
    runs of one tile, in one batch; alone, and beside prompts in the same launch."""
    rng = np.random.default_rng(17)
    short = [(1, 30000)] + [(1, int(k)) for k in rng.integers(1, 40, 60)] + [(1, 9000), (2, 17),
                                                                            (1, 4096), (1, 1)]
    c = Case(short, 8, 2, 64, 64, seed=17)
    c.check(*c.run())
    c = Case(short[:40] + [(300, 700)] + short[40:], 8, 2, 64, 64, seed=18)
    c.check(*c.run())


@pytest.mark.parametrize("seed", range(16))
def test_random_batches(seed):
    """Random heads, pages, groups, query and key lengths."""
    rng = np.random.default_rng(1000 + seed)
    hq, hkv = [(8, 1), (8, 8), (6, 2), (10, 2), (12, 4), (32, 1), (28, 4), (24, 8)][seed % 8]
    dim, page = [64, 128][int(rng.integers(2))], [16, 32, 64, 128][int(rng.integers(4))]
    lens, groups = [], []
    for _ in range(int(rng.integers(0, 3))):
        prefix, n = page * int(rng.integers(0, 900 // page + 2)), int(rng.integers(1, 24))
        groups.append((n, prefix))
        for _ in range(n):
            q = int(rng.choice([1, 1, 1, 2, 5, 40]))
            lens.append((q, prefix + q + int(rng.integers(0, 300))))
    for _ in range(int(rng.integers(1, 30))):
        q = int(rng.choice([0, 1, 1, 1, 3, 17, 100, 260]))
        lens.append((q, max(0, q + int(rng.integers(-2, 900)))))
    c = Case(lens, hq, hkv, dim, page, groups=groups, seed=seed, std=float(rng.uniform(0.3, 2.5)),
             extra_tokens=int(rng.integers(0, 3)))
    c.check(*c.run())


def test_one_token_everywhere():
    """The smallest batch."""
    for dim in (64, 128):
        c = Case([(1, 1)], 1, 1, dim, 16, seed=19)
        out, lse = c.run()
        c.check(out, lse)
        want = c.vp[c.table[0, 0], 0, 0]
        assert torch.equal(out[0, 0], want)          # its own value, weight one


def test_a_dropped_batch_keeps_its_memory_while_another_stream_works():
    """The plan, the workspace and the tables belong to the stream that made them; a
    batch that another stream uses is dropped while that stream still works, and the
    first stream is not given their memory before it is done."""
    c = Case([(1, 900), (100, 500)], 16, 2, 128, 16, seed=40)
    want = c.run()
    kv = torch.from_numpy(c.kv).cuda()
    qkv = torch.zeros((c.t, 20 * 128), dtype=torch.bfloat16, device="cuda")
    k2, v2 = c.kp.clone(), c.vp.clone()
    # kernels loaded and outputs in hand: either would wait for the stream's work
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    q2 = bd.bitdelta_kv_append(c.batch, qkv, None, k2, v2)
    side = torch.cuda.Stream()
    for call in ("attention", "append"):
        batch = bd.AttentionBatch(
            torch.from_numpy(c.off).cuda(), kv.clone(), torch.from_numpy(c.table).cuda(),
            n_tokens=c.t, max_q_len=100, max_kv_len=900, n_q_heads=16, n_kv_heads=2, head_dim=128,
            page_size=16)
        used = {t.data_ptr() for t in batch._tensors}
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(1_000_000_000)               # about half a second
        if call == "attention":
            bd.bitdelta_attention(batch, c.q, c.kp, c.vp, out=out, lse=lse, stream=side)
        else:
            bd.bitdelta_kv_append(batch, qkv, None, k2, v2, out=q2, stream=side)
        done = side.record_event()
        del batch
        free = {b["address"] for seg in torch.cuda.memory_snapshot() for b in seg["blocks"]
                if b["state"] == "inactive"}
        assert not done.query(), "the stream was done too early to tell"
        assert not used & free
        side.synchronize()
        if call == "attention":
            assert torch.equal(want[0], out) and torch.equal(want[1], lse)
    assert bd.bitdelta_check_error() == 0


@pytest.mark.parametrize("dim", [64, 128])
def test_a_nan_query_gives_nan(dim):
    """Output and lse of its rows alone; an lse of minus infinity is for rows without a
    key.  Single tokens alone and in parts, prompts whole and cut, shared prefixes."""
    batches = [([(1, 40), (1, 20011), (1, 300)], ()), ([(100, 300), (1, 50), (40, 9000)], ()),
               ([(1, 512 + i) for i in range(1, 31)] + [(40, 600)], [(30, 512)])]
    for lens, groups in batches:
        c = Case(lens, 8, 2, dim, 16, groups=groups, seed=41)
        want, want_l = c.run()
        rows = [(int(c.off[s + 1]) - 1, 3 * s % 8) for s in range(len(lens))]
        hit = torch.zeros((c.t, 8), dtype=torch.bool, device="cuda")
        for t, h in rows:
            c.q[t, h, 5] = NAN
            hit[t, h] = True
        out, lse = c.run()
        assert out[hit].isnan().all() and lse[hit].isnan().all()
        # a row's neighbours share its exchanges but not its values
        ok = ~hit
        assert torch.isfinite(out[ok].float()).all()
        assert ((out[ok].float() - want[ok].float()).abs() <= 2.0 ** -7 * c.vp.float().nan_to_num(
            0.0).abs().max()).all()
        assert ((lse[ok] - want_l[ok]).abs() <= 2.0 ** -14 * (1 + want_l[ok].abs())).all()
        assert bd.bitdelta_check_error() == 0


@pytest.mark.parametrize("what", ["single", "groups", "prompts", "tiles"])
def test_more_sequences_and_tiles_than_the_plan_takes_at_once(what):
    """The plan walks sequences and tiles 1024 at a time and carries its sums over."""
    rng = np.random.default_rng(42)
    groups = []
    if what == "single":
        lens = [(1, int(k)) for k in rng.integers(0, 40, 2500)]
    elif what == "groups":
        groups = [(9, 32)] * 150
        lens = [(1, 33 + int(k)) for k in rng.integers(0, 40, 1350)]
        lens += [(1, int(k)) for k in rng.integers(0, 40, 200)]
    elif what == "prompts":
        lens = [(1, int(k)) for k in rng.integers(1, 40, 2100)]
        for s in (0, 1023, 1024, 1500, 2047, 2048, 2099):
            lens[s] = (int(rng.integers(20, 200)), 200)
    else:
        lens = [(int(q), 30 + int(q)) for q in rng.integers(5, 9, 2200)]    # a tile each
    n = len(lens)
    c = Case(lens, 4, 1 if what == "tiles" else 2, 64, 16, groups=groups, seed=43, extra_tokens=2)
    out, lse = c.run()
    near = {s for k in (0, 1024, 2048, n) for s in range(k - 5, k + 5) if 0 <= s < n}
    c.check(out, lse, seqs=sorted(near | set(range(0, n, 11))))
    again, lse2 = c.run()
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("lens", [[(1, 100), (1, 64)], [(1, 100), (40, 64)]])
@pytest.mark.parametrize("what", ["max_q_len", "max_kv_len", "not sorted", "past the tokens",
                                  "narrow table", "groups"])
def test_a_refused_table_writes_rows_without_keys(lens, what):
    """Every row, in either kernel: nothing of the outputs is left as it was."""
    groups = [(2, 16)] if what == "groups" else ()
    c = Case(lens, 8, 2, 128, 16, groups=groups, seed=44)
    over = {}
    if what == "max_q_len":
        over["max_q_len"] = max(q for q, _ in lens) - 1
    elif what == "max_kv_len":
        over["max_kv_len"] = 99
    elif what == "not sorted":
        c.off[1] = c.t + 1
    elif what == "past the tokens":
        c.off[2] += 1
        over["max_q_len"] = 64
    elif what == "narrow table":
        c.table = np.ascontiguousarray(c.table[:, :6])
    else:
        over["group_offsets"] = torch.tensor([2, 0], dtype=torch.int32).cuda()
    batch = c.make(**over)
    assert bd.bitdelta_check_error() == 7
    out = torch.full((c.t, 8, 128), NAN, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c.t, 8), NAN, device="cuda")
    bd.bitdelta_attention(batch, c.q, c.kp, c.vp, out=out, lse=lse)
    assert (out == 0).all() and torch.isneginf(lse).all()
    assert bd.bitdelta_check_error() == 0
