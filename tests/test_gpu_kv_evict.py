"""bitdelta_kv_evict and bitdelta_kv_evict_lengths against the choice made row by row on
the host.  An eviction compares and copies: every result is exact."""
import math

import numpy as np
import pytest
import torch

import bit_weight_delta_gb300 as bd

pytestmark = pytest.mark.gpu
INF, NAN = math.inf, math.nan


class Case:
    """kv: keys per sequence; groups: (sequences, shared keys)."""

    def __init__(self, kv, keep, hkv=2, dim=64, page=16, recent=0, sink=0, groups=(), seed=0,
                 spare=3, shift=None, ties=False, width=None):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.kv, self.keep = np.array(kv, np.int32), np.array(keep, np.int32)
        self.hkv, self.dim, self.page, self.recent, self.sink = hkv, dim, page, recent, sink
        n = len(kv)
        need = [-(-int(k) // page) for k in kv]
        self.prefix, lead, s0, offs, pre = [0] * n, {}, 0, [0], []
        for cnt, shared in groups:
            for s in range(s0, s0 + cnt):
                self.prefix[s] = shared
                if s > s0:
                    lead[s] = (s0, shared // page)
            s0 += cnt
            offs.append(s0)
            pre.append(shared)
        fresh = [need[s] - lead.get(s, (0, 0))[1] for s in range(n)]
        self.n_pages = sum(fresh) + spare
        order, u = rng.permutation(self.n_pages), 0
        self.table = np.full((n, width or max(need + [1]) + 1), 2 ** 30, np.int32)  # past kv: unread
        for s in range(n):
            first, sh = lead.get(s, (s, 0))
            self.table[s, :sh] = self.table[first, :sh]
            self.table[s, sh:need[s]] = order[u:u + fresh[s]]
            u += fresh[s]
        shape = (self.n_pages, hkv, page)
        self.k = torch.randn((*shape, dim), generator=g, device="cuda").to(torch.bfloat16)
        self.v = torch.randn((*shape, dim), generator=g, device="cuda").to(torch.bfloat16)
        w = torch.randn(shape, generator=g, device="cuda").exp() - 0.3
        self.w = (w * 2).round() if ties else torch.relu(w)
        # neither early nor late, and then as many of both as there are to be
        self.pos = torch.randint(sink, sink + 10, shape, generator=g, device="cuda",
                                 dtype=torch.int32)
        self.shift = np.array(shift if shift is not None else
                              rng.integers(0, 1000, n) + min(recent, 10 ** 6) + sink + 10, np.int32)
        for s in range(n):             # positions of a few are recent, of a few the first
            for h in range(hkv):
                some = rng.permutation(int(kv[s]))[:recent + sink]
                for i, slot in enumerate(some):
                    self.pos[self.table[s, slot // page], h, slot % page] = (
                        int(kv[s]) + int(self.shift[s]) - 1 - i if i < recent else i - recent)
        kw = {}
        if groups:
            kw = {"group_offsets": torch.tensor(offs, dtype=torch.int32).cuda(),
                  "prefix_len": torch.tensor(pre, dtype=torch.int32).cuda()}
        self.make = lambda **over: bd.AttentionBatch(
            torch.arange(n + 1, dtype=torch.int32, device="cuda"),
            torch.from_numpy(self.kv).cuda(), torch.from_numpy(self.table).cuda(), **{**dict(
                n_tokens=n, max_q_len=1, max_kv_len=int(self.kv.max(initial=0)), n_q_heads=hkv,
                n_kv_heads=hkv, head_dim=dim, page_size=page), **kw, **over})
        self.batch = self.make()

    def length(self, s):
        kv, keep = int(self.kv[s]), int(self.keep[s])
        return kv if keep < 0 or keep >= kv else max(keep, min(self.prefix[s], kv))

    def want(self, apart):
        """(k, v, weights, positions) after the call, from the tensors as they are."""
        k, v, w, pos = (t.clone().cpu() for t in (self.k, self.v, self.w, self.pos))
        w_in, p_in = self.w.cpu().numpy(), self.pos.cpu().numpy()
        if apart:
            w, pos = torch.full_like(w, -7.0), torch.full_like(pos, -7)
        src_k, src_v = self.k.cpu(), self.v.cpu()
        for s in range(len(self.kv)):
            n, new, first = int(self.kv[s]), self.length(s), min(self.prefix[s], int(self.kv[s]))
            place = lambda i: (self.table[s, i // self.page].astype(np.int64), i % self.page)
            for h in range(self.hkv):
                slots = np.arange(first, n)
                pg, at = place(slots)
                ww, pp = w_in[pg, h, at].astype(np.float64), p_in[pg, h, at].astype(np.int64)
                held = (pp >= n + int(self.shift[s]) - self.recent) | (pp < self.sink)
                ww = np.where(np.isnan(ww), -INF, ww)
                ww = np.where(held, 0.0, ww)        # protected ones are alike
                nan = np.isnan(w_in[pg, h, at])
                rank = np.lexsort((slots, nan & ~held, -ww, ~held))
                stay = np.sort(slots[rank[:new - first]])
                src = np.arange(new)
                holes = np.setdiff1d(np.arange(first, new), stay)
                src[holes] = stay[stay >= new]
                to, frm = place(np.arange(new)), place(src)
                if apart or (src != np.arange(new)).any():
                    w[to[0], h, to[1]] = torch.from_numpy(w_in[frm[0], h, frm[1]])
                    pos[to[0], h, to[1]] = torch.from_numpy(p_in[frm[0], h, frm[1]])
                k[to[0], h, to[1]] = src_k[frm[0], h, frm[1]]
                v[to[0], h, to[1]] = src_v[frm[0], h, frm[1]]
        return k, v, w, pos

    def call(self, apart=False, **kw):
        out = {}
        if apart:
            out = {"weights_out": torch.full_like(self.w, -7.0),
                   "positions_out": torch.full_like(self.pos, -7)}
        return bd.bitdelta_kv_evict(
            self.batch, torch.from_numpy(self.keep).cuda(), self.k, self.v, self.w, self.pos,
            recent=self.recent, sink=self.sink, pos_offset=torch.from_numpy(self.shift).cuda(),
            **out, **kw)

    def check(self, apart=False):
        want = self.want(apart)
        before = self.w.clone(), self.pos.clone()
        got = self.call(apart)
        assert bd.bitdelta_check_error() == 0
        for name, a, b in zip(("k", "v", "weights", "positions"), (self.k, self.v, *got), want):
            a, b = a.cpu(), b
            if a.dtype == torch.float32:
                a, b = a.view(torch.int32), b.view(torch.int32)
            if a.dtype == torch.bfloat16:
                a, b = a.view(torch.int16), b.view(torch.int16)
            assert torch.equal(a, b), (name, int((a != b).sum()))
        if apart:
            assert torch.equal(self.w.view(torch.int32), before[0].view(torch.int32))
            assert torch.equal(self.pos, before[1])


@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dim", [64, 128])
def test_pages_and_head_sizes(page, dim, apart):
    Case([300, 77, 1, 16, 0, 129], [100, 76, 1, 3, 5, 128], dim=dim, page=page, recent=5,
         sink=2).check(apart)


@pytest.mark.parametrize("kv", [2, 15, 16, 17, 31, 33, 511, 512, 513, 1025, 4160])
@pytest.mark.parametrize("share", ["one", "half", "all but one"])
def test_lengths(kv, share):
    keep = {"one": 1, "half": kv // 2, "all but one": kv - 1}[share]
    Case([kv, kv], [keep, keep], hkv=3, recent=min(2, keep), seed=kv).check()


@pytest.mark.parametrize("kv,keep", [(6000, 5000), (9001, 512), (20000, 19999), (33000, 16500),
                                     (70001, 30001)])
@pytest.mark.parametrize("apart", [False, True])
def test_one_long_sequence_over_a_cluster(kv, keep, apart):
    Case([kv], [keep], hkv=2, dim=64, page=128, recent=100, sink=4, seed=kv).check(apart)


def test_a_cache_past_32_bits():
    """The same pages behind 65536 others, more than 2^31 elements into the cache."""
    c = Case([300, 5000, 129], [100, 2000, 128], hkv=2, dim=128, page=128, recent=5, sink=2, seed=40)
    small = [t.clone() for t in (c.k, c.v, c.w, c.pos)]
    c.call()
    first, far = 65536, []
    for t in small:
        far.append(torch.zeros((first + c.n_pages, *t.shape[1:]), dtype=t.dtype, device="cuda"))
        far[-1][first:] = t
    near = (c.k, c.v, c.w, c.pos)
    c.k, c.v, c.w, c.pos = far
    c.table = (np.minimum(c.table, 2 ** 29) + first).astype(np.int32)
    c.batch = c.make()
    c.call()
    assert bd.bitdelta_check_error() == 0
    for a, b in zip(far, near):
        assert torch.equal(a[first:], b) and not a[:first].any()


@pytest.mark.parametrize("n", [40, 80, 160, 400])
def test_many_sequences(n):
    rng = np.random.default_rng(n)
    kv = rng.integers(1, 400, n)
    Case(kv, rng.integers(-1, 300, n), hkv=1, recent=3, sink=1, seed=n).check()


@pytest.mark.parametrize("others,kv", [(160, 700), (160, 5000), (160, 17000), (39, 9000), (30, 17000),
                                       (15, 33000), (3, 5000)])
@pytest.mark.parametrize("apart", [False, True])
def test_one_long_sequence_among_short_ones(others, kv, apart):
    """One to eight CTAs of every number of threads, most of them with next to nothing to do."""
    rng = np.random.default_rng(others)
    short = rng.integers(1, 60, others)
    at = others // 2
    Case([*short[:at], kv, *short[at:]], [*(short[:at] // 2), kv // 3, *(short[at:] - 1)], hkv=1,
         page=32, recent=2, sink=1, seed=kv).check(apart)


def test_equal_weights_go_by_their_slot():
    Case([1000, 257], [500, 100], ties=True, recent=10, sink=1, seed=3).check()
    c = Case([5000], [2000], hkv=1, seed=4)      # all alike: nothing moves
    c.w.fill_(1.5)
    c.check()
    c = Case([12000], [700], hkv=4, ties=True, seed=5)
    c.check()


def test_weights_of_every_kind():
    c = Case([600, 600], [200, 400], hkv=2, recent=20, seed=6)
    flat = c.w.view(-1)
    g = torch.Generator(device="cuda").manual_seed(1)
    for value, step in ((NAN, 3), (INF, 17), (-INF, 19), (0.0, 5), (-0.0, 4), (-1.0, 7), (1e-45, 11)):
        at = torch.randperm(flat.numel(), generator=g, device="cuda")[::step]
        flat[at] = value
    c.check()


def test_nothing_but_nan():
    c = Case([100], [40], hkv=1, seed=7)
    c.w.fill_(NAN)
    c.check()


def test_more_protected_than_kept():
    Case([200, 90], [50, 10], recent=100, sink=0, seed=8).check()
    c = Case([200, 90], [50, 10], recent=40, sink=40, seed=9)
    c.check()


def test_everything_protected():
    c = Case([300], [70], hkv=2, seed=10)
    c.recent = 2 ** 31 - 1
    c.check()


@pytest.mark.parametrize("keep", [-1, 0, 1, 63, 64, 65, 128, 200, 10 ** 9])
def test_budgets_around_a_shared_prefix(keep):
    c = Case([200, 150, 90, 64, 70], [keep] * 5, groups=[(4, 64)], recent=3, seed=11)
    c.check(apart=True)
    c = Case([200, 150, 90, 64, 70], [keep] * 5, groups=[(4, 64)], recent=3, seed=11)
    c.check()


def test_a_keep_of_nothing():
    c = Case([100, 30], [0, 0], seed=12)
    c.check()
    assert [c.length(s) for s in range(2)] == [0, 0]


def test_slots_past_the_new_length_and_other_pages_stay():
    c = Case([100, 60], [50, 60], seed=13, spare=5)
    k, w = c.k.clone(), c.w.clone()
    c.call()
    for s, new in ((0, 50), (1, 0)):
        for slot in range(new, int(c.kv[s])):
            pg, at = c.table[s, slot // c.page], slot % c.page
            assert torch.equal(c.k[pg, :, at], k[pg, :, at])
            assert torch.equal(c.w[pg, :, at], w[pg, :, at])
    used = set(c.table[0, :7].tolist()) | set(c.table[1, :4].tolist())
    for pg in set(range(c.n_pages)) - used:
        assert torch.equal(c.k[pg], k[pg]) and torch.equal(c.w[pg], w[pg])


def test_an_evicted_cache_is_cut_no_further():
    c = Case([900, 333], [400, 200], recent=30, sink=4, seed=14)
    c.check()
    kv, shift = torch.from_numpy(c.kv).cuda(), torch.from_numpy(c.shift).cuda()
    bd.bitdelta_kv_evict_lengths(c.batch, torch.from_numpy(c.keep).cuda(), kv, shift)
    assert kv.tolist() == [400, 200]
    assert shift.tolist() == [int(c.shift[0]) + 500, int(c.shift[1]) + 133]
    c.kv, c.shift = kv.cpu().numpy(), shift.cpu().numpy()
    c.batch = c.make()
    k = c.k.clone()
    c.check()
    assert torch.equal(c.k, k)


def test_lengths_in_place():
    kv = torch.tensor([50, 20, 70, 64, 33], dtype=torch.int32, device="cuda")
    table = torch.zeros((5, 5), dtype=torch.int32, device="cuda")
    batch = bd.AttentionBatch(torch.arange(6, dtype=torch.int32, device="cuda"), kv, table, 5, 1, 80,
                              2, 2, 64, 16,
                              group_offsets=torch.tensor([2, 4], dtype=torch.int32, device="cuda"),
                              prefix_len=torch.tensor([32], dtype=torch.int32, device="cuda"))
    shift = torch.tensor([0, 1, 2, 3, 4], dtype=torch.int32, device="cuda")
    keep = torch.tensor([10, 30, 5, 40, -1], dtype=torch.int32, device="cuda")
    out = bd.bitdelta_kv_evict_lengths(batch, keep, kv, shift)
    assert out[0] is kv and out[1] is shift
    assert kv.tolist() == [10, 20, 32, 40, 33] and shift.tolist() == [40, 1, 40, 27, 4]
    assert bd.bitdelta_check_error() == 0


def test_a_bad_page_is_reported_and_leaves_the_head_alone():
    c = Case([100, 100], [40, 40], seed=15)
    good = Case([100, 100], [40, 40], seed=15)
    c.table[0, 3] = c.n_pages
    c.batch = c.make()
    k, w = c.k.clone(), c.w.clone()
    want = good.want(False)
    c.call()
    assert bd.bitdelta_check_error() == 7
    for pg in (p for p in c.table[0, :7] if p < c.n_pages):
        assert torch.equal(c.k[pg], k[pg]) and torch.equal(c.w[pg], w[pg])
    for pg in c.table[1, :7]:
        assert torch.equal(c.k[pg].cpu().view(torch.int16), want[0][pg].view(torch.int16))


def test_lengths_past_the_bounds_are_reported():
    for max_kv, kv in ((50, [60, 20]), (100, [-3, 20]), (1000, [500, 20])):
        c = Case([60, 20], [10, 10], seed=16)
        c.kv = np.array(kv, np.int32)
        c.batch = c.make(max_kv_len=max_kv)
        k = c.k.clone()
        c.call()
        assert bd.bitdelta_check_error() == 7
        for pg in c.table[0, :4]:
            assert torch.equal(c.k[pg], k[pg])


def test_a_graph_of_a_step():
    c = Case([700, 300, 20], [256, 256, 256], recent=16, seed=17)
    keep, shift = torch.from_numpy(c.keep).cuda(), torch.from_numpy(c.shift).cuda()
    start = [t.clone() for t in (c.k, c.v, c.w, c.pos)]

    def step():
        bd.bitdelta_kv_evict(c.batch, keep, c.k, c.v, c.w, c.pos, recent=16, pos_offset=shift)

    want = c.want(False)
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(2):
        for t, s in zip((c.k, c.v, c.w, c.pos), start):
            t.copy_(s)
        graph.replay()
        for t, x in zip((c.k, c.v, c.w, c.pos), want):
            assert torch.equal(t.cpu(), x)


def test_two_streams_at_once():
    cases = [Case([3000 + i] * 20, [1000] * 20, hkv=2, recent=50, seed=20 + i) for i in range(2)]
    wants = [c.want(False) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for c, s in zip(cases, streams):
        c.call(stream=s)
    torch.cuda.synchronize()
    for c, want in zip(cases, wants):
        for t, x in zip((c.k, c.v, c.w, c.pos), want):
            assert torch.equal(t.cpu(), x)
    assert bd.bitdelta_check_error() == 0


def test_refusals():
    c = Case([40], [20])
    keep = torch.from_numpy(c.keep).cuda()
    for args in ((keep[:0], c.k, c.v, c.w, c.pos), (keep.long(), c.k, c.v, c.w, c.pos),
                 (keep, c.k, c.v[:-1], c.w, c.pos), (keep, c.k, c.v, c.w[:-1], c.pos),
                 (keep, c.k, c.v, c.w.double(), c.pos), (keep, c.k, c.v, c.w, c.pos.long()),
                 (keep, c.k, c.v, c.w, c.pos.transpose(0, 1).contiguous()),
                 (keep, c.k.cpu(), c.v, c.w, c.pos), (keep, c.k, c.v, c.w.cpu(), c.pos)):
        with pytest.raises(ValueError):
            bd.bitdelta_kv_evict(c.batch, *args)
    for kw in ({"recent": -1}, {"sink": -1}, {"recent": 2 ** 31}, {"pos_offset": keep[:0]},
               {"weights_out": c.w[:-1]}, {"positions_out": c.pos.float()}):
        with pytest.raises(ValueError):
            bd.bitdelta_kv_evict(c.batch, keep, c.k, c.v, c.w, c.pos, **kw)
    with pytest.raises(TypeError):
        bd.bitdelta_kv_evict(c.batch, keep, c.k, c.v, c.w, c.pos, recent=1.5)
    big = c.make(max_kv_len=344065)
    with pytest.raises(bd.BitDeltaError):
        bd.bitdelta_kv_evict(big, keep, c.k, c.v, c.w, c.pos)


def lengths_of(c):
    """(kv_len, pos_offset) after bitdelta_kv_evict_lengths into outputs of their own."""
    kv, shift = torch.full((len(c.kv),), 77, dtype=torch.int32, device="cuda"), torch.from_numpy(c.shift).cuda()
    bd.bitdelta_kv_evict_lengths(c.batch, torch.from_numpy(c.keep).cuda(), kv, shift)
    return kv.tolist(), (shift.cpu().numpy() - c.shift).tolist()


@pytest.mark.parametrize("max_kv,kv", [(50, 60), (100, -3), (1000, 500)])
def test_lengths_of_a_refused_sequence_stay(max_kv, kv):
    """Past the bound, negative, and past the page table's row (of 5 pages)."""
    c = Case([60, 20], [10, 10], seed=50)
    c.kv = np.array([kv, 20], np.int32)
    c.batch = c.make(max_kv_len=max_kv)
    bd.bitdelta_check_error()
    c.call()
    assert bd.bitdelta_check_error() == 7
    assert lengths_of(c) == ([kv, 10], [0, 10])
    assert bd.bitdelta_check_error() == 7
    own, shift = torch.from_numpy(c.kv).cuda(), torch.from_numpy(c.shift).cuda()
    batch = bd.AttentionBatch(torch.arange(3, dtype=torch.int32, device="cuda"), own,
                              torch.from_numpy(c.table).cuda(), 2, 1, max_kv, 2, 2, 64, 16)
    bd.bitdelta_kv_evict_lengths(batch, torch.from_numpy(c.keep).cuda(), own, shift)   # in place
    assert own.tolist() == [kv, 10] and (shift.cpu().numpy() - c.shift).tolist() == [0, 10]
    assert bd.bitdelta_check_error() == 7


@pytest.mark.parametrize("where", [0, 3, 6])
def test_lengths_of_a_sequence_with_a_bad_page_stay(where):
    """The eviction left it alone; once its table is right, it is cut like any other."""
    c, good = (Case([100, 100], [40, 40], seed=51) for _ in range(2))
    page, c.table[0, where] = c.table[0, where], c.n_pages
    c.batch = c.make()
    c.call()
    assert bd.bitdelta_check_error() == 7
    assert lengths_of(c) == ([100, 40], [0, 60])
    assert bd.bitdelta_check_error() == 7
    want = good.want(False)
    c.table[0, where], c.keep[1] = page, -1
    c.batch = c.make()
    c.call()
    assert lengths_of(c) == ([40, 100], [60, 0])
    assert bd.bitdelta_check_error() == 0
    for got, t in zip((c.k, c.v, c.w, c.pos), want):
        assert torch.equal(got.cpu(), t)


def test_lengths_with_a_bad_page_that_is_not_chosen_from():
    """In a shared prefix, behind the last key, or of a sequence that is not cut: none of
    them stops the eviction or the lengths."""
    c = Case([100, 90, 70], [64, 80, 70], groups=[(2, 32)], seed=52)
    c.table[0, 1] = -1
    c.table[1, 6] = c.n_pages
    c.table[2, 2] = -1
    c.batch = c.make()
    c.call()
    assert lengths_of(c) == ([64, 80, 70], [36, 10, 0])
    assert bd.bitdelta_check_error() == 0


def test_lengths_of_many_sequences_and_groups():
    n = 700
    rng = np.random.default_rng(53)
    kv = rng.integers(64, 400, n)
    keep = rng.integers(-1, 300, n)
    c = Case(kv, keep, hkv=1, groups=[(2, 16 * (1 + i % 4)) for i in range(300)], seed=53)
    c.call()
    want = [c.length(s) for s in range(n)]
    assert lengths_of(c) == (want, [int(k) - w for k, w in zip(kv, want)])
    assert bd.bitdelta_check_error() == 0
