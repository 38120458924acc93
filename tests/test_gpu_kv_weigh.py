"""bitdelta_kv_weigh against the softmax weights in 64 bits.

Tolerances (derived before the first run).  A score is an fp32 sum of head_dim exact
products, off by at most 2^-19 of s_max = scale·max Σ|q·k| (as in the attention's tests); its product with log2 e,
the subtraction of the lse and the power add at most 2^-21·(1 + s_max + |lse|) to a weight,
relatively.  Sums in fp32 of n weights, in an order of the kernel's own, add at most
2^-24·n relatively, of positive terms (n <= 2^12 here: 2^-12 would be the worst case of a
serial sum; the rows pass through lanes of eight, so 2^-24·(n/8 + 8) bounds it), and the
sum with the table's value one rounding."""
import math

import numpy as np
import pytest
import torch

import bit_weight_delta_gb300 as bd

pytestmark = pytest.mark.gpu
INF, NAN = math.inf, math.nan


class Case:
    """lens: (query tokens, keys) per sequence; groups: (sequences, shared prefix)."""

    def __init__(self, lens, hq=8, hkv=2, dim=128, page=16, groups=(), window=0, seed=0, std=1.0,
                 extra_tokens=0, shift=True):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.hq, self.hkv, self.dim, self.page = lens, hq, hkv, dim, page
        self.window = window
        n = len(lens)
        self.off = np.concatenate([[0], np.cumsum([q for q, _ in lens])]).astype(np.int32)
        self.kv = np.array([k for _, k in lens], np.int32)
        need = [-(-int(k) // page) for k in self.kv]
        lead, s0, offs, pre = {}, 0, [0], []
        for cnt, prefix in groups:
            for s in range(s0 + 1, s0 + cnt):
                lead[s] = (s0, prefix // page)
            s0 += cnt
            offs.append(s0)
            pre.append(prefix)
        fresh = [need[s] - lead.get(s, (0, 0))[1] for s in range(n)]
        self.n_pages = sum(fresh) + 3
        order, u = rng.permutation(self.n_pages), 0
        self.table = np.full((n, max(need + [1]) + 1), 2 ** 30, np.int32)   # past kv_len: unread
        for s in range(n):
            first, sh = lead.get(s, (s, 0))
            self.table[s, :sh] = self.table[first, :sh]
            self.table[s, sh:need[s]] = order[u:u + fresh[s]]
            u += fresh[s]
        self.t = int(self.off[-1]) + extra_tokens
        self.shift = torch.from_numpy(rng.integers(0, 9999, n).astype(np.int32)).cuda() if shift else None

        def rn(*shape):
            return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)

        self.q = rn(self.t, hq, dim)
        self.kp = torch.full((self.n_pages, hkv, page, dim), NAN, dtype=torch.bfloat16, device="cuda")
        for s in range(n):              # NaN stays wherever no key is
            for i in range(need[s]):
                m = min(page, int(self.kv[s]) - i * page)
                self.kp[self.table[s, i], :, :m] = rn(hkv, m, dim)
        self.w = torch.rand((self.n_pages, hkv, page), generator=g, device="cuda")
        self.pos = torch.full((self.n_pages, hkv, page), -5, dtype=torch.int32, device="cuda")
        for s, (ql, kv) in enumerate(lens):     # a recycled page: what new slots held before
            for slot in range(max(0, kv - ql), kv):
                self.w[self.table[s, slot // page], :, slot % page] = NAN
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
        self.scale = 1.0 / math.sqrt(dim)
        self.lse = torch.full((self.t, hq), NAN, device="cuda")
        self.scores = {}
        for s in range(n):
            for h in range(hkv):
                sc, seen, _ = self.score(s, h)
                self.lse[self.off[s]:self.off[s + 1], h * (hq // hkv):(h + 1) * (hq // hkv)] = (
                    torch.logsumexp(torch.where(seen, sc, -INF), -1).T.float())

    def score(self, s, h):
        """Scaled scores [g, q_len, kv] in 64 bits, what is seen, and the largest Σ|q·k|."""
        g = self.hq // self.hkv
        lo, hi, n = int(self.off[s]), int(self.off[s + 1]), int(self.kv[s])
        slot = torch.arange(n, device="cuda")
        pg = torch.from_numpy(self.table[s, :-(-n // self.page)].astype(np.int64)).cuda()
        k = self.kp[pg, h].reshape(-1, self.dim)[:n].double()
        q = self.q[lo:hi, h * g:(h + 1) * g].double().transpose(0, 1)
        seen = slot[None] <= torch.arange(n - (hi - lo), n, device="cuda")[:, None]
        return q @ k.T * self.scale, seen, (
            q.abs() @ k.abs().T * self.scale).amax() if n and hi > lo else 0.0

    def want(self):
        """(weights, tolerances, positions) after the call."""
        w, pos = self.w.double(), self.pos.clone()
        tol = torch.zeros_like(w)
        g = self.hq // self.hkv
        for s, (ql, kv) in enumerate(self.lens):
            slot = torch.arange(max(0, kv - ql), kv, device="cuda")
            pg = torch.from_numpy(self.table[s].astype(np.int64)).cuda()[slot // self.page]
            if ql > 0:
                w[pg, :, slot % self.page] = 0.0
                shift = 0 if self.shift is None else int(self.shift[s])
                pos[pg, :, slot % self.page] = (slot + shift).to(torch.int32)[:, None]
        rows = {}
        for s, (ql, kv) in enumerate(self.lens):
            if ql == 0 or kv == 0:
                continue
            slot = torch.arange(kv, device="cuda")
            pg = torch.from_numpy(self.table[s].astype(np.int64)).cuda()[slot // self.page]
            first = max(0, ql - self.window) if self.window else 0
            lo, hi = int(self.off[s]), int(self.off[s + 1])
            for h in range(self.hkv):
                sc, seen, s_max = self.score(s, h)
                lse = self.lse[lo:hi, h * g:(h + 1) * g].double().T[..., None]
                a = torch.where(seen & torch.isfinite(lse), torch.exp(sc - lse), 0.0)[:, first:]
                l_max = torch.where(torch.isfinite(lse), lse.abs(), 0.0).amax()
                rel = 2.0 ** -19 * s_max + 2.0 ** -21 * (1 + s_max + l_max) + 2.0 ** -24 * (
                    a.shape[0] * a.shape[1] / 8 + 8)
                a = a.sum((0, 1))
                w[pg, h, slot % self.page] += a
                tol[pg, h, slot % self.page] += rel * a
        return w, tol + 2.0 ** -23 * w.abs(), pos

    def call(self, **kw):
        return bd.bitdelta_kv_weigh(self.batch, self.q, self.lse, self.kp, self.w, self.pos,
                                    window=self.window, pos_offset=self.shift, **kw)

    def check(self):
        want, tol, pos = self.want()
        got = self.call()
        assert got[0] is self.w and got[1] is self.pos
        assert bd.bitdelta_check_error() == 0
        bad = (self.w.double() - want).abs() > tol
        assert not bad.any(), (int(bad.sum()), (self.w.double() - want).abs().max().item())
        assert not torch.isnan(self.w).any()
        assert torch.equal(self.pos, pos)


HEADS = [(8, 1, 128), (8, 8, 64), (6, 2, 128), (10, 2, 64), (32, 1, 128), (14, 2, 128), (7, 1, 64)]


@pytest.mark.parametrize("hq,hkv,dim", HEADS)
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_mixed_lengths(hq, hkv, dim, page):
    Case([(1, 1), (1, 40), (5, 5), (3, 300), (1, 129), (0, 20), (40, 40), (70, 190)], hq, hkv, dim,
         page, seed=hq + page).check()


@pytest.mark.parametrize("kv", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 1000])
def test_single_tokens(kv):
    Case([(1, kv), (1, max(1, kv - 1)), (1, kv + 1)], hq=8, hkv=1, page=16, seed=kv).check()


@pytest.mark.parametrize("q", [2, 3, 8, 9, 16, 17, 31, 32, 33, 63, 64, 65, 128, 130, 257, 600])
@pytest.mark.parametrize("hq,hkv,dim", [(8, 1, 128), (4, 2, 64), (5, 1, 128)])
def test_prompts(q, hq, hkv, dim):
    Case([(q, q)], hq, hkv, dim, seed=q).check()
    Case([(q, q + 77), (1, 50), (q // 2, q)], hq, hkv, dim, page=32, seed=q).check()


@pytest.mark.parametrize("window", [1, 2, 16, 31, 64, 1000])
def test_windows(window):
    Case([(200, 200), (64, 300), (1, 77), (20, 20), (150, 151)], window=window, seed=window).check()


@pytest.mark.parametrize("window", [0, 1, 3, 20])
@pytest.mark.parametrize("lens", [
    [(1, 70), (1, 100), (1, 65)], [(2, 80), (5, 69), (1, 65), (0, 64)],
    [(40, 120), (1, 70), (33, 97)], [(1, 90)]])
def test_shared_prefixes(lens, window):
    Case(lens + [(1, 33), (9, 40)], groups=[(len(lens), 64)], window=window, seed=3).check()


def test_groups_of_many():
    lens = [(1, 256 + 1 + i) for i in range(70)] + [(2, 512 + 9 * i + 2) for i in range(33)]
    Case(lens, hq=16, hkv=2, groups=[(70, 256), (33, 512)], page=64, seed=4).check()


def test_a_group_without_a_prefix_or_members():
    Case([(1, 50), (3, 40), (1, 20)], groups=[(2, 0), (0, 16), (1, 16)], seed=5).check()


def test_many_sequences():
    rng = np.random.default_rng(6)
    lens = [(1, int(k)) for k in rng.integers(1, 300, 700)]
    Case(lens, hq=4, hkv=1, dim=64, seed=6).check()
    lens = [(int(q), int(q + k)) for q, k in zip(rng.integers(0, 5, 300), rng.integers(1, 60, 300))]
    Case(lens, hq=4, hkv=2, dim=64, seed=7).check()


def test_a_long_context():
    Case([(1, 40001)], hq=8, hkv=2, page=128, seed=8).check()
    Case([(1, 20000), (1, 3), (600, 9000)], hq=8, hkv=1, page=64, window=40, seed=9).check()


def test_tokens_of_no_sequence_and_padding():
    """Rows behind the last sequence, and a sequence with more query tokens than keys."""
    c = Case([(3, 50), (1, 20)], extra_tokens=5, seed=10)
    c.check()
    c = Case([(6, 4), (1, 20)], seed=11)
    c.check()
    c = Case([(2, 0), (1, 20)], seed=12)
    c.check()


def test_rows_whose_lse_is_not_finite_add_nothing():
    c = Case([(40, 90), (1, 30), (6, 70)], seed=13)
    c.lse[3, 1], c.lse[7, :], c.lse[40, 0], c.lse[42, 5] = NAN, -INF, INF, NAN
    c.q[42, 5] = NAN
    c.check()


def test_infinite_and_nan_keys_out_of_sight():
    """Keys that a causal mask hides from a row do not reach its sums."""
    c = Case([(70, 70)], hq=2, hkv=1, seed=14)
    c.kp[c.table[0, 4], 0, 5] = INF        # slot 69: the last row alone sees it
    c.lse[69] = NAN
    c.check()


def test_repeated_calls_accumulate():
    c = Case([(1, 100), (4, 60)], seed=15)
    c.check()
    base = c.w.clone()
    c.call()
    d = c.w.double() - base.double()
    assert torch.isfinite(c.w).all() and (d >= -1e-6).all()
    # a sequence's weights sum to one per row
    for s, (ql, kv) in enumerate(c.lens):
        for h in range(c.hkv):
            got = sum(d[c.table[s, p // 16], h, p % 16].item() for p in range(kv - ql))
            assert got <= ql * (c.hq // c.hkv) + 1e-3


def test_the_same_call_gives_the_same_bits():
    a = Case([(300, 300), (1, 5000), (1, 90)], hq=8, hkv=2, seed=16)
    start = a.w.clone()
    a.call()
    first = a.w.clone()
    for _ in range(3):
        a.w.copy_(start)
        a.call()
        assert torch.equal(a.w, first)


def test_after_the_attention():
    """With the lse that bitdelta_attention gives, a sequence's weights sum to its rows."""
    c = Case([(30, 200), (1, 77)], hq=8, hkv=2, seed=17)
    vp = torch.nan_to_num(c.kp)
    _, lse = bd.bitdelta_attention(c.batch, c.q, c.kp, vp)
    c.w.zero_()
    bd.bitdelta_kv_weigh(c.batch, c.q, lse, c.kp, c.w, c.pos)
    for s, (ql, kv) in enumerate(c.lens):
        slot = np.arange(kv)
        for h in range(c.hkv):
            got = c.w[c.table[s, slot // 16], h, slot % 16].double().sum().item()
            assert abs(got - ql * 4) <= ql * 4 * 2.0 ** -12
    assert bd.bitdelta_check_error() == 0


def test_scales():
    c = Case([(9, 60), (1, 33)], seed=18)
    for scale in (0.02, 0.5):
        c = Case([(9, 60), (1, 33)], seed=18)
        c.scale = scale
        for s in range(2):
            for h in range(c.hkv):
                sc, seen, _ = c.score(s, h)
                c.lse[c.off[s]:c.off[s + 1], 4 * h:4 * h + 4] = torch.logsumexp(
                    torch.where(seen, sc, -INF), -1).T.float()
        want, tol, _ = c.want()
        c.call(scale=scale)
        assert ((c.w.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("scale", [2.0 ** -100, 1e-20, 1e-3, 40.0])
@pytest.mark.parametrize("lens", [[(1, 90), (2, 33)], [(50, 300), (17, 17)]])
def test_scales_far_from_the_usual(scale, lens):
    c = Case(lens, hq=8, hkv=2, seed=30)
    c.scale = scale
    for s in range(len(lens)):
        for h in range(c.hkv):
            sc, seen, _ = c.score(s, h)
            c.lse[c.off[s]:c.off[s + 1], 4 * h:4 * h + 4] = torch.logsumexp(
                torch.where(seen, sc, -INF), -1).T.float()
    want, tol, pos = c.want()
    c.call(scale=scale)
    assert bd.bitdelta_check_error() == 0
    # a term below fp32's least normal number, 2^-126, may come out as 0; a key has at most
    # 50·4 < 2^8 terms
    tol += 2.0 ** -118
    assert ((c.w.double() - want).abs() <= tol).all() and torch.equal(c.pos, pos)


def test_a_cache_past_32_bits():
    """The same pages behind 65536 others, more than 2^31 elements into the cache."""
    c = Case([(1, 300), (60, 200), (3, 40), (1, 129), (1, 140)], hq=8, hkv=2, dim=128, page=128,
             seed=31)
    first, w, pos = 65536, c.w.clone(), c.pos.clone()
    c.call()
    kp = torch.zeros((first + c.n_pages, 2, 128, 128), dtype=torch.bfloat16, device="cuda")
    kp[first:] = c.kp
    far_w = torch.zeros(kp.shape[:3], device="cuda")
    far_w[first:] = w
    far_pos = torch.zeros(kp.shape[:3], dtype=torch.int32, device="cuda")
    far_pos[first:] = pos
    c.table = (np.minimum(c.table, 2 ** 29) + first).astype(np.int32)
    bd.bitdelta_kv_weigh(c.make(), c.q, c.lse, kp, far_w, far_pos, pos_offset=c.shift)
    assert bd.bitdelta_check_error() == 0
    assert torch.equal(far_w[first:].view(torch.int32), c.w.view(torch.int32))
    assert torch.equal(far_pos[first:], c.pos)
    assert not far_w[:first].any() and not far_pos[:first].any()


def test_a_graph_of_prompts_and_shared_prefixes():
    """Both kernels of a call captured, replayed twice over the same tables, and an eager call
    between."""
    c = Case([(1, 70), (5, 90), (1, 66), (130, 300), (1, 1000)], groups=[(3, 64)], seed=32)
    c.call()
    start, pos = torch.nan_to_num(c.w), c.pos.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.call()
    for _ in range(2):
        c.w.copy_(start)
        c.call()
        want = c.w.clone()
        c.w.copy_(start)
        graph.replay()
        assert torch.equal(c.w, want) and torch.equal(c.pos, pos)
    assert bd.bitdelta_check_error() == 0


@pytest.mark.parametrize("bad", ["kv", "order", "tokens", "prefix", "odd prefix", "table"])
def test_broken_tables_change_nothing(bad):
    c = Case([(1, 70), (2, 90), (1, 40)], groups=[(2, 64)], seed=19)
    if bad == "kv":
        c.kv[1] = 95
    elif bad == "order":
        c.off[1] = 4
    elif bad == "tokens":
        c.off[3] = 9
    elif bad == "table":
        c.kv[2] = 16 * c.table.shape[1] + 1
    over = {"max_kv_len": 90} if bad != "table" else {"max_kv_len": 10 ** 6}
    if bad == "prefix":
        over["prefix_len"] = torch.tensor([80], dtype=torch.int32, device="cuda")
    if bad == "odd prefix":
        over["prefix_len"] = torch.tensor([24], dtype=torch.int32, device="cuda")
    c.batch = c.make(**over)
    bd.bitdelta_check_error()        # the plan reports some of them as well
    w, pos = c.w.clone(), c.pos.clone()
    c.call()
    assert bd.bitdelta_check_error() == 7
    assert torch.equal(c.w.view(torch.int32), w.view(torch.int32)) and torch.equal(c.pos, pos)


@pytest.mark.parametrize("q", [1, 64])
def test_a_bad_page_is_reported_and_skipped(q):
    c = Case([(q, 200), (1, 50)], hq=8, hkv=2, seed=20)
    want, tol, pos = c.want()
    bad = int(c.table[0, 2])
    c.table[0, 2] = -1
    c.batch = c.make()
    w = c.w.clone()
    c.call()
    assert bd.bitdelta_check_error() == 7
    assert torch.equal(c.w[bad], w[bad])
    rest = torch.ones(c.n_pages, dtype=torch.bool, device="cuda")
    rest[bad] = False
    assert ((c.w.double() - want).abs() <= tol)[rest].all()


def test_a_graph_replays_with_new_lengths():
    c = Case([(1, 500), (1, 80), (1, 300)], seed=21)
    kv = torch.from_numpy(c.kv).cuda()
    batch = bd.AttentionBatch(torch.from_numpy(c.off).cuda(), kv, torch.from_numpy(c.table).cuda(), 3,
                              1, 500, 8, 2, 128, 16)
    start = c.w.clone()
    call = lambda: bd.bitdelta_kv_weigh(batch, c.q, c.lse, c.kp, c.w, c.pos, pos_offset=c.shift)
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for new in ([500, 80, 300], [100, 80, 299], [1, 16, 300]):
        c.kv[:] = new
        c.lens = [(1, k) for k in new]
        for s in range(3):
            for h in range(2):
                sc, seen, _ = c.score(s, h)
                c.lse[s, 4 * h:4 * h + 4] = torch.logsumexp(torch.where(seen, sc, -INF), -1).T.float()
        c.w.copy_(torch.nan_to_num(start))
        want, tol, _ = c.want()
        kv.copy_(torch.from_numpy(c.kv))
        graph.replay()
        assert ((c.w.double() - want).abs() <= tol).all()
    assert bd.bitdelta_check_error() == 0


def test_two_streams_at_once():
    cases = [Case([(1, 2000)] * 30 + [(60, 500)] * 2, seed=22 + i) for i in range(2)]
    wants = [c.want() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for c, s in zip(cases, streams):
        c.call(stream=s)
    torch.cuda.synchronize()
    for c, (want, tol, pos) in zip(cases, wants):
        assert ((c.w.double() - want).abs() <= tol).all() and torch.equal(c.pos, pos)


def test_refusals():
    c = Case([(1, 20)])
    args = [c.q, c.lse, c.kp, c.w, c.pos]
    for i, wrong in ((0, c.q.float()), (0, c.q[:0]), (1, c.lse.double()), (1, c.lse[:, :4]),
                     (2, c.kp[:, :1]), (2, c.kp.float()), (3, c.w[:1]), (3, c.w.half()),
                     (4, c.pos.long()), (4, c.pos.cpu()), (0, c.q.cpu()),
                     (3, c.w.transpose(1, 2))):
        with pytest.raises(ValueError):
            bd.bitdelta_kv_weigh(c.batch, *args[:i], wrong, *args[i + 1:])
    for kw in ({"window": -1}, {"window": 2 ** 31}, {"pos_offset": c.pos},
               {"pos_offset": torch.zeros(1, device="cuda")}):
        with pytest.raises(ValueError):
            bd.bitdelta_kv_weigh(c.batch, *args, **kw)
    for scale in (0.0, -1.0, NAN, INF):
        with pytest.raises(bd.BitDeltaError):
            bd.bitdelta_kv_weigh(c.batch, *args, scale=scale)


@pytest.mark.parametrize("grouped", [False, True])
def test_prompts_with_many_runs_between_them(grouped):
    """What a role waits for another does not grow by the runs without tiles between two that
    have some: all waits end within 5 ms, with 40000 single tokens of one key each there."""
    n, g, dim, page, q = 40000, 8, 64, 16, 2000
    lens = np.array([q] + [1] * n + [q])
    need = -(-lens // page)
    first = np.concatenate([[0], np.cumsum(need)])
    table = (first[:-1, None] + np.minimum(np.arange(need.max()), need[:, None] - 1)).astype(np.int32)
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    i32 = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()
    kw = {}
    if grouped:                            # pairs that share nothing
        kw = {"group_offsets": i32(np.arange(0, n + 3, 2)), "prefix_len": i32([0] * (n // 2 + 1))}
    batch = bd.AttentionBatch(i32(off), i32(lens), i32(table), int(off[-1]), q, q, g, 1, dim, page, **kw)
    gen = torch.Generator(device="cuda").manual_seed(36)
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)
    qs, kp = rn(int(off[-1]), g, dim), rn(int(first[-1]), 1, page, dim)
    _, lse = bd.bitdelta_attention(batch, qs, kp, kp)
    weights = torch.zeros((int(first[-1]), 1, page), device="cuda")
    positions = torch.full(weights.shape, -1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    bd.bitdelta_set_wait_limit_ns(5_000_000)
    try:
        bd.bitdelta_kv_weigh(batch, qs, lse, kp, weights, positions)
        assert bd.bitdelta_check_error() == 0
    finally:
        bd.bitdelta_set_wait_limit_ns(2_000_000_000)
    # every row's weights sum to one, within lse's own error, 2^-16·(1 + |lse|) at most with
    # |lse| below 10, and a score's, 2^-19 of less than 16
    w, pages = weights.view(-1).double(), int(need[0]) * page
    for part in (w[:pages], w[-pages:]):
        assert abs(part.sum().item() - q * g) <= q * g * 2.0 ** -12
    single = w[pages:-pages].view(n, page)
    assert ((single[:, 0] - g).abs() <= g * 2.0 ** -12).all() and not single[:, 1:].any()
    pos = positions.view(-1)
    for part in (pos[:pages], pos[-pages:]):
        assert torch.equal(part[:q], torch.arange(q, device="cuda", dtype=torch.int32))
    assert (pos[pages:-pages].view(n, page)[:, 0] == 0).all()


@pytest.mark.parametrize("at", [[0, 5, 639, 640, 641, 1279, 1280, 1499], [700], [1499], [3, 4]])
@pytest.mark.parametrize("window", [0, 20])
def test_prompts_spread_among_many_single_tokens(at, window):
    """More runs than a CTA of the tile kernel has threads, and than one of the short runs'."""
    rng = np.random.default_rng(33)
    lens = [(1, int(k)) for k in rng.integers(1, 60, 1500)]
    for i in at:
        lens[i] = (17 + i % 40, 60 + i % 300)
    Case(lens, hq=4, hkv=1, dim=64, window=window, seed=33).check()


@pytest.mark.parametrize("members,groups", [(3, 250), (2, 400), (5, 1)])
def test_groups_behind_many_sequences(members, groups):
    rng = np.random.default_rng(34)
    lens = [(1, int(k)) for k in rng.integers(65, 120, members * groups)]
    lens += [(1, int(k)) for k in rng.integers(1, 50, 900)]
    lens[-1], lens[-400] = (30, 70), (9, 300)
    Case(lens, hq=8, hkv=1, dim=64, seed=34,
         groups=[(members, 16 * (1 + g % 4)) for g in range(groups)]).check()


@pytest.mark.parametrize("lens,groups", [([(1, 100), (4, 60), (40, 130), (1, 7)], ()),
                                         ([(1, 70), (2, 90), (1, 101), (20, 80)], [(3, 64)])])
def test_each_further_call_adds_as_much(lens, groups):
    c = Case(lens, groups=groups, window=0, seed=35)
    for _ in range(3):
        c.check()


@pytest.mark.parametrize("at", [0, 1, 3])
@pytest.mark.parametrize("kv", [0, 5, 64])
@pytest.mark.parametrize("q", [1, 30])
def test_a_member_of_a_group_without_tokens(at, kv, q):
    """A server's empty place in a group: a prefix longer than its keys reaches into no query
    tokens of its own, and the others' weights are what they are without it."""
    lens = [(1, 70), (q, 110), (2, 90), (1, 65)]
    lens[at] = (0, 64)
    c = Case(lens + [(1, 40)], groups=[(4, 64)], seed=37)
    c.kv[at], c.lens[at] = kv, (0, kv)
    c.batch = c.make()
    vp = torch.nan_to_num(c.kp)
    bd.bitdelta_attention(c.batch, c.q, c.kp, vp)
    assert bd.bitdelta_check_error() == 0
    c.check()
