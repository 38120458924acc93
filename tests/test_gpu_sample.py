"""bitdelta_sample against the definition in 64 bits.

The kernel's weights are off by about 2^-40 and its sums hold them exactly, so a
choice can differ from the one in 64 bits only where u lies within V·2^-40 (2^-21 at
most) of a border between two tokens; `choose` says how near u lies, and the random numbers are
drawn until none does.  prob is a quotient of such sums, rounded to fp32: 2^-24
relative for the rounding, 2^-21 at most for the sums' 2^-44 steps over a vocabulary of 2^19;
2^-20 is allowed."""
import math

import numpy as np
import pytest
import torch

import bit_weight_delta_gb300 as bd

pytestmark = pytest.mark.gpu
INF, NAN = math.inf, math.nan


def choose(x, u, t=1.0, k=0, p=1.0, m=0.0):
    """(token, prob, distance of u and of the cuts from the next border) of one row of values."""
    x = np.where(np.isnan(x), -INF, x.astype(np.float64))
    if not (x > -INF).any():
        return -1, 0.0, 1.0
    order = np.argsort(-x, kind="stable")
    v = x[order]
    n_all = int((v > -INF).sum())
    with np.errstate(all="ignore"):
        if v[0] == INF:
            w = (v == INF).astype(np.float64)
        elif t == 0:
            w = (v == v[0]).astype(np.float64)
        else:
            w = np.exp((v - v[0]) / t)
    if t == 0:
        return int(order[0]), 1.0, 1.0
    total = np.cumsum(w)
    n, near = n_all, 1.0
    if 0 < k < n:
        n = k
    if p < 1:
        want = max(p, 0.0) * total[n - 1]
        cut = int(np.searchsorted(total[:n], want, side="left")) + 1
        # The weight 1 is exact, another one off by 2^-40 of itself and its two roundings to
        # 2^-44 steps, half a step each: a nearness of len(x)·2^-40 is that of their sum.
        # (Sums of nothing but the largest are exact.)
        less = w[(w > 0) & (w < 1)]
        off = less.sum() * 2.0 ** -40 + len(less) * 2.0 ** -44
        if off > 0:
            near = min(near, np.abs(total[:n] - want).min() / off * len(x) * 2.0 ** -40)
    else:
        cut = n
    if m > 0:
        cut = min(cut, max(1, int((w >= m).sum())))
        # one weight's own error, not V of them: 2^-40 of the distance is enough
        near = min(near, np.abs(w[w < 1] - m).min(initial=1.0) * len(x))
    cut = max(1, min(cut, n))
    target = min(max(u, 0.0), 1.0) * total[cut - 1]
    i = min(int(np.searchsorted(total[:cut], target, side="right")), int((w[:cut] > 0).sum()) - 1)
    near = min(near, np.abs(total[:cut] - target).min() / total[cut - 1]) if u < 1 else near
    return int(order[i]), w[i] / total[cut - 1], near


def values(logits):
    return logits.float().cpu().numpy()


def check(logits, u, t=None, k=None, p=None, m=None, least=None, **kw):
    """The call against `choose`, row by row; rows too near a border are given another u."""
    rows, vocab = logits.shape
    x = values(logits)
    least = vocab * 2.0 ** -40 if least is None else least
    u = np.array(u, np.float32)
    rng = np.random.default_rng(99)
    sets = [np.full(rows, d, dt) if a is None else np.array(a, dt) for a, d, dt in (
        (t, 1.0, np.float32), (k, 0, np.int32), (p, 1.0, np.float32), (m, 0.0, np.float32))]
    want = []
    for r in range(rows):
        args = [float(sets[0][r]), int(sets[1][r]), float(sets[2][r]), float(sets[3][r])]
        got = choose(x[r], float(u[r]), *args)
        for _ in range(20):
            if got[2] > least:
                break
            u[r] = rng.random(dtype=np.float32)
            got = choose(x[r], float(u[r]), *args)
        assert got[2] > least, r
        want.append(got[:2])
    names = ("temperature", "top_k", "top_p", "min_p")
    given = {n: torch.from_numpy(s).cuda() for n, s, a in zip(names, sets, (t, k, p, m))
             if a is not None}
    tokens, prob = bd.bitdelta_sample(logits, torch.from_numpy(u).cuda(), **given, **kw)
    assert bd.bitdelta_check_error() == 0
    assert tokens.tolist() == [w[0] for w in want]
    ref = np.array([w[1] for w in want])
    assert (np.abs(prob.cpu().numpy() - ref) <= 2.0 ** -20 * ref).all()


def rand_logits(rows, vocab, std=2.5, seed=0, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((rows, vocab + pad), generator=g, device="cuda") * std
    return x.to(torch.bfloat16)[:, :vocab]


def rand_u(rows, seed=0):
    return np.random.default_rng(seed).random(rows, dtype=np.float32)


@pytest.mark.parametrize("vocab", [1, 2, 7, 8, 9, 31, 255, 1000, 8191, 32000, 65528, 65537, 131071,
                                   262144, 524032])
def test_vocabularies(vocab):
    rows = 3
    check(rand_logits(rows, vocab, seed=vocab), rand_u(rows, vocab))


@pytest.mark.parametrize("rows", [1, 2, 5, 18, 19, 37, 38, 76, 77, 153, 400])
def test_rows(rows):
    """Every number of CTAs per row, and more rows than run at once."""
    check(rand_logits(rows, 5003, seed=rows), rand_u(rows, rows))


@pytest.mark.parametrize("pad", [0, 1, 2, 3, 5, 8, 13])
def test_padded_rows(pad):
    check(rand_logits(6, 1001, pad=pad), rand_u(6, 3))


@pytest.mark.parametrize("start", range(1, 9))
def test_rows_off_alignment(start):
    check(rand_logits(4, 777 + start)[:, start:], rand_u(4, 5))


def test_settings_of_every_kind():
    rows = 96
    rng = np.random.default_rng(1)
    t = rng.choice([0.0, 0.05, 0.3, 0.7, 1.0, 2.0, 30.0, 1e4], rows)
    k = rng.choice([-1, 0, 1, 2, 5, 50, 1000, 100000], rows)
    p = rng.choice([-1.0, 0.0, 0.1, 0.5, 0.9, 0.999, 1.0, 2.0], rows)
    m = rng.choice([-1.0, 0.0, 1e-6, 0.01, 0.3, 1.0, 2.0], rows)
    check(rand_logits(rows, 4001, seed=2), rand_u(rows, 2), t, k, p, m)


@pytest.mark.parametrize("which", ["t", "k", "p", "m"])
def test_one_setting(which):
    rows = 24
    rng = np.random.default_rng(4)
    v = {"t": rng.uniform(0.2, 2, rows), "k": rng.integers(1, 200, rows),
         "p": rng.uniform(0.05, 1, rows), "m": rng.uniform(0.001, 0.5, rows)}[which]
    check(rand_logits(rows, 20011, seed=5), rand_u(rows, 6), **{which: v})


def test_equal_logits_go_by_their_index():
    """One value everywhere: token floor(u·kept); cuts at exact shares."""
    vocab = 100000
    x = torch.full((4, vocab), -1.25, dtype=torch.bfloat16, device="cuda")
    u = torch.tensor([0.0, 0.5, 0.25, 0.75], device="cuda")
    tokens, prob = bd.bitdelta_sample(x, u)
    assert tokens.tolist() == [0, 50000, 25000, 75000]
    assert prob.tolist() == [np.float32(1e-5)] * 4
    k = torch.tensor([1, 2, 4, 4], dtype=torch.int32, device="cuda")
    tokens, prob = bd.bitdelta_sample(x, u, top_k=k)
    assert tokens.tolist() == [0, 1, 1, 3] and prob.tolist() == [1.0, 0.5, 0.25, 0.25]
    p = torch.full((4,), 0.5, device="cuda")
    tokens, prob = bd.bitdelta_sample(x, u, top_k=k, top_p=p)
    assert tokens.tolist() == [0, 0, 0, 1] and prob.tolist() == [1.0, 1.0, 0.5, 0.5]


def test_both_zeros_are_one_value():
    x = torch.zeros((1, 16), dtype=torch.bfloat16, device="cuda")
    x[0, ::2] = -0.0
    for i in range(16):
        u = torch.tensor([(i + 0.5) / 16], device="cuda")
        assert bd.bitdelta_sample(x, u)[0].item() == i


def test_ends_of_u():
    x = rand_logits(5, 999, seed=8)
    low = bd.bitdelta_sample(x, torch.tensor([0.0, -1.0, 0.0, 0.0, 1e-45], device="cuda"))[0]
    assert low.tolist() == x.float().argmax(1).tolist()
    last = torch.argsort(x.float(), dim=1, descending=True, stable=True)[:, 6]
    k = torch.full((5,), 7, dtype=torch.int32, device="cuda")
    high = bd.bitdelta_sample(x, torch.tensor([1.0, 2.0, INF, 1.0, 1.0], device="cuda"), top_k=k)[0]
    assert high.tolist() == last.tolist()


def test_masked_rows():
    x = rand_logits(12, 3001, seed=9)
    x[0] = -INF
    x[1] = NAN
    x[2, :3000] = -INF
    x[3, 1:] = -INF
    x[4, ::2] = NAN
    x[5, 17] = INF
    x[6, 5:9] = INF
    x[7, :] = torch.finfo(torch.bfloat16).min
    x[8, 10:] = torch.finfo(torch.bfloat16).min
    x[9, 3] = torch.finfo(torch.bfloat16).max
    x[9, 4] = torch.finfo(torch.bfloat16).min
    x[10] = -NAN
    x[10, 99] = -INF
    x[11, ::3] = -INF
    check(x, rand_u(12, 10))
    check(x, rand_u(12, 11), t=[0.0] * 12)
    check(x, rand_u(12, 12), k=[3] * 12, p=[0.9] * 12, m=[0.01] * 12)


def test_extreme_values_and_temperatures():
    """Every finite bf16 value once, spread over all temperatures."""
    bits = torch.arange(65536, dtype=torch.int32)
    x = bits.to(torch.uint16).view(torch.bfloat16)
    x = x[torch.isfinite(x.float())].cuda()[None].repeat(6, 1)
    check(x, rand_u(6, 13), t=[1e-30, 1.0, 1e10, 1e37, 3e38, INF])


def test_tiny_and_huge_temperatures():
    check(rand_logits(6, 2000, seed=3), rand_u(6, 14), t=[1e-45, 1e-38, 1e-10, 1e6, 1e30, INF])


# bf16 neighbours around 2^16, −2^16, ±2^-40 and zero, where the counters of values end
LARGE = [49152.0, 65024.0, 65280.0, 65536.0, 66048.0, 131072.0]
SMALL = [2.0 ** e for e in (-39, -40, -41, -42, -126, -133)] + [2.0 ** -40 * 1.0078125,
                                                               2.0 ** -41 * 1.9921875, 0.0]


@pytest.mark.parametrize("vocab", [64, 20011])
@pytest.mark.parametrize("sign", [1.0, -1.0, 0.0])  # 0: of both signs
@pytest.mark.parametrize("values_of, t", [
    (LARGE[:3], 3000.0), (LARGE, 3000.0), (LARGE, 3e5), (LARGE, 1.0), (LARGE[3:], 4e4),
    (SMALL, 2.0 ** -40), (SMALL, 2.0 ** -42), (SMALL, 1.0), (SMALL[2:], 2.0 ** -42),
    (SMALL[:2], 2.0 ** -40), (LARGE[1:5] + SMALL, 2e3), (LARGE[:3] + [0.0, 8.0], 2e3)])
def test_values_at_the_ends_of_the_counters(values_of, t, sign, vocab):
    rows = 6
    rng = np.random.default_rng(len(values_of))
    x = rng.choice(np.array(values_of), (rows, vocab))
    x *= rng.choice([1.0, -1.0], x.shape) if sign == 0 else sign
    x[1, 5:] = -INF                       # few logits, the rest masked
    x[2, ::2] = -NAN
    x[3, 1:] = np.where(rng.random(vocab - 1) < 0.9, 1.0, x[3, 1:])
    logits = torch.from_numpy(x).to(torch.bfloat16).cuda()
    assert torch.equal(logits.double().cpu().nan_to_num(7.0), torch.from_numpy(x).nan_to_num(7.0))
    check(logits, rand_u(rows, 8), t=[t] * rows, k=[0, 0, 0, 0, vocab // 3, 0],
          p=[1, 1, 1, 1, 1, 0.7])


def test_far_values_count_at_high_temperatures():
    """−2^16 and below, with the largest 33 temperatures above them and less."""
    x = np.full((8, 5000), -65536.0)
    x[:, 100:200] = -70144.0
    x[:, 7] = [0.0, 0.0, 0.0, 0.0, -32768.0, -65280.0, 60160.0, -131072.0]
    t = [1e3, 1.9e3, 2.2e3, 1e5, 1e3, 1e3, 1e5, 1e4]
    for seed in range(3):
        check(torch.from_numpy(x).to(torch.bfloat16).cuda(), rand_u(8, seed), t=t)


def test_bad_parameters_are_reported():
    x, u = rand_logits(3, 50), torch.tensor([0.3, 0.3, 0.3], device="cuda")
    good = bd.bitdelta_sample(x, u)[0].tolist()
    for name, value in (("temperature", -1.0), ("temperature", NAN), ("top_p", NAN), ("min_p", NAN)):
        v = torch.tensor([1.0, value, 1.0] if name != "min_p" else [0.0, value, 0.0], device="cuda")
        tokens, prob = bd.bitdelta_sample(x, u, **{name: v})
        assert tokens.tolist() == [good[0], -1, good[2]] and prob[1] == 0
        assert bd.bitdelta_check_error() == 7
    tokens, _ = bd.bitdelta_sample(x, torch.tensor([0.3, NAN, 0.3], device="cuda"))
    assert tokens.tolist() == [good[0], -1, good[2]]
    assert bd.bitdelta_check_error() == 7


def test_outputs_of_the_callers_own_and_rows_behind_them():
    x, u = rand_logits(4, 333), torch.from_numpy(rand_u(4)).cuda()
    want = bd.bitdelta_sample(x, u)
    tokens = torch.full((6,), 77, dtype=torch.int32, device="cuda")
    prob = torch.full((6,), 0.5, device="cuda")
    bd.bitdelta_sample(x, u, tokens=tokens[1:5], prob=prob[1:5])
    assert tokens.tolist() == [77, *want[0].tolist(), 77]
    assert prob.tolist() == [0.5, *want[1].tolist(), 0.5]


def test_no_rows():
    x = torch.empty((0, 100), dtype=torch.bfloat16, device="cuda")
    tokens, prob = bd.bitdelta_sample(x, torch.empty(0, device="cuda"))
    assert tokens.shape == (0,) and prob.shape == (0,)


def test_a_graph_replays_with_new_inputs():
    x, u = rand_logits(9, 12345, seed=20), torch.from_numpy(rand_u(9, 20)).cuda()
    t = torch.full((9,), 0.7, device="cuda")
    bd.bitdelta_sample(x, u, temperature=t)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tokens, prob = bd.bitdelta_sample(x, u, temperature=t)
    for seed in range(3):
        x.copy_(rand_logits(9, 12345, seed=30 + seed))
        u.copy_(torch.from_numpy(rand_u(9, 30 + seed)))
        graph.replay()
        want = bd.bitdelta_sample(x, u, temperature=t)
        assert torch.equal(tokens, want[0]) and torch.equal(prob, want[1])


def test_two_streams_at_once():
    jobs = []
    for i in range(2):
        jobs.append((torch.cuda.Stream(), rand_logits(40, 30011, seed=40 + i),
                     torch.from_numpy(rand_u(40, 40 + i)).cuda()))
    want = [bd.bitdelta_sample(x, u) for _, x, u in jobs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, (s, x, u) in enumerate(jobs):
            got[i].append(bd.bitdelta_sample(x, u, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert torch.equal(g[0], want[i][0]) and torch.equal(g[1], want[i][1])


def test_the_draw_follows_the_distribution():
    """Equally spaced u: each token's share of them is its probability, to one draw."""
    n = 4096
    x = rand_logits(1, 300, std=1.5, seed=50).expand(n, 300).contiguous()
    u = (torch.arange(n, device="cuda") + 0.5) / n
    tokens, _ = bd.bitdelta_sample(x, u)
    share = torch.bincount(tokens.long(), minlength=300).double()
    prob = torch.softmax(x[0].double(), 0) * n
    assert (share - prob).abs().max() <= 1.0 + 1e-6


@pytest.mark.parametrize("wrong", [
    lambda x, u: (x.float(), u), lambda x, u: (x[0], u), lambda x, u: (x, u[:-1]),
    lambda x, u: (x, u.double()), lambda x, u: (x.cpu(), u), lambda x, u: (x, u.cpu()),
    lambda x, u: (x.t(), u[:1].expand(10).contiguous()), lambda x, u: (x[:, :0], u),
    lambda x, u: (x[:1].expand(4, 10), u)])
def test_refusals(wrong):
    x, u = rand_logits(4, 10), torch.zeros(4, device="cuda")
    with pytest.raises(ValueError):
        bd.bitdelta_sample(*wrong(x, u))


def test_refused_settings():
    x, u = rand_logits(4, 10), torch.zeros(4, device="cuda")
    for name, v in (("temperature", torch.ones(3)), ("temperature", torch.ones(4).half()),
                    ("top_k", torch.ones(4)), ("top_k", torch.ones(4, dtype=torch.int64)),
                    ("top_p", torch.ones(5)), ("min_p", torch.ones(4, 1)),
                    ("tokens", torch.ones(4)), ("prob", torch.ones(2))):
        with pytest.raises(ValueError):
            bd.bitdelta_sample(x, u, **{name: v.cuda()})
    with pytest.raises(bd.BitDeltaError):
        bd.bitdelta_sample(torch.zeros((1, 524033), dtype=torch.bfloat16, device="cuda"), u[:1])


@pytest.mark.parametrize("value", [0.0, 1.5, -1.5, 2.0 ** 20, -2.0 ** 20])
def test_one_value_over_the_largest_vocabulary(value):
    """The largest sum that a row can have, 524032 weights of 2^44 in one bin."""
    x = torch.full((4, 524032), value, dtype=torch.bfloat16, device="cuda")
    check(x, rand_u(4, 60), k=[0, 0, 400001, 1000], p=[1.0, 0.3, 0.7, 0.5], m=[0.0, 0.5, 1.0, 0.0])
