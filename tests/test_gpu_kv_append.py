"""bitdelta_kv_append against the rotation in 64 bits.

Rotated values are one fp32 product-sum rounded once to bf16: within 2^-8 of
the value plus 2^-22 of |a| + |b|.  Everything that is not rotated, and every
cache row that is not a new token's, is bit-exact."""
import numpy as np
import pytest
import torch

import bit_weight_delta_gb300 as bd

pytestmark = pytest.mark.gpu


def make(lens, hq, hkv, dim, page, seed=0, width=None, spare=2, rope_rows=None, rot=None):
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    off = np.concatenate([[0], np.cumsum([q for q, _ in lens])]).astype(np.int32)
    kv = np.array([k for _, k in lens], np.int32)
    need = [-(-int(k) // page) for k in kv]
    n_pages = sum(need) + spare
    order = rng.permutation(n_pages)
    table = np.full((len(lens), width or max(max(need), 1)), -12345, np.int32)  # never read
    u = 0
    for s, n in enumerate(need):
        table[s, :n] = order[u:u + n]
        u += n
    t = int(off[-1])

    def rn(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

    batch = bd.AttentionBatch(
        torch.from_numpy(off).cuda(), torch.from_numpy(kv).cuda(), torch.from_numpy(table).cuda(),
        n_tokens=t, max_q_len=max([q for q, _ in lens], default=0),
        max_kv_len=int(kv.max(initial=0)), n_q_heads=hq, n_kv_heads=hkv, head_dim=dim,
        page_size=page)
    rot = dim if rot is None else rot
    rows = int(kv.max(initial=0)) if rope_rows is None else rope_rows
    ang = np.arange(rows)[:, None] * 10000.0 ** (-2.0 * np.arange(rot // 2) / max(rot, 1))
    rope = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)).cuda()
    return (batch, off, kv, table, rn(t, (hq + 2 * hkv) * dim), rope,
            rn(n_pages, hkv, page, dim), rn(n_pages, hkv, page, dim))


def reference(off, kv, table, qkv, rope, kp, vp, hq, hkv, dim, page, pairs):
    """Values in float64 and the magnitudes |a| + |b| of what was summed."""
    rot = rope.shape[1]
    x = qkv.double().cpu().numpy().reshape(-1, hq + 2 * hkv, dim)
    rp = rope.double().cpu().numpy()
    q = np.zeros((x.shape[0], hq, dim))
    kr, vr = kp.double().cpu().numpy(), vp.double().cpu().numpy()
    mag_q, mag_k = np.zeros_like(q), np.zeros_like(kr)
    a_i = np.arange(0, rot, 2) if pairs else np.arange(rot // 2)
    b_i = a_i + (1 if pairs else rot // 2)
    for s in range(len(kv)):
        for t in range(off[s], off[s + 1]):
            pos = int(kv[s]) - (off[s + 1] - t)
            if pos < 0:
                continue
            c, sn = rp[pos, :rot // 2], rp[pos, rot // 2:]
            y, m = x[t].copy(), np.zeros_like(x[t])
            a, b = x[t][:hq + hkv][:, a_i], x[t][:hq + hkv][:, b_i]
            y[:hq + hkv, a_i] = a * c - b * sn
            y[:hq + hkv, b_i] = b * c + a * sn
            m[:hq + hkv, a_i] = m[:hq + hkv, b_i] = np.abs(a) + np.abs(b)
            q[t], mag_q[t] = y[:hq], m[:hq]
            pg = table[s, pos // page]
            kr[pg, :, pos % page], mag_k[pg, :, pos % page] = y[hq:hq + hkv], m[hq:hq + hkv]
            vr[pg, :, pos % page] = x[t, hq + hkv:]
    return q, kr, vr, mag_q, mag_k


def close(got, ref, mag, what):
    err = np.abs(got.double().cpu().numpy() - ref)
    tol = np.where(mag > 0, 2.0 ** -8 * np.abs(ref) + 2.0 ** -22 * mag, 0.0)
    assert (err <= tol).all(), (what, err.max())


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("hq,hkv,dim,page,rot", [(8, 2, 128, 16, 128), (6, 6, 64, 32, 64),
                                                 (5, 1, 128, 128, 64), (64, 8, 128, 64, 16),
                                                 (3, 1, 64, 16, 48), (4, 2, 64, 16, 0)])
def test_append(hq, hkv, dim, page, rot, pairs):
    lens = [(1, 1), (1, 17), (5, 5), (3, 130), (40, 64), (1, 16), (0, 9), (7, 3)]
    batch, off, kv, table, qkv, rope, kp, vp = make(lens, hq, hkv, dim, page, seed=rot, rot=rot)
    ref = reference(off, kv, table, qkv, rope, kp, vp, hq, hkv, dim, page, pairs)
    q = bd.bitdelta_kv_append(batch, qkv, rope, kp, vp, interleaved=pairs)
    close(q, ref[0], ref[3], "q")
    close(kp, ref[1], ref[4], "k")
    assert np.array_equal(vp.double().cpu().numpy(), ref[2])
    assert bd.bitdelta_check_error() == 0
    # the same call again writes the same values
    k1, v1 = kp.clone(), vp.clone()
    q1 = bd.bitdelta_kv_append(batch, qkv, rope, kp, vp, interleaved=pairs)
    assert torch.equal(q, q1) and torch.equal(kp, k1) and torch.equal(vp, v1)


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("hq,hkv,dim,page,rot", [(6, 2, 128, 16, 128), (3, 1, 64, 64, 32)])
def test_more_tokens_than_run_at_once(hq, hkv, dim, page, rot, pairs):
    """Several rounds of CTAs, whose rows are fetched ahead; the last rows end
    at the tensor's end."""
    lens = [(1, 40), (1400, 1401), (1, 7), (131, 500)]
    batch, off, kv, table, qkv, rope, kp, vp = make(lens, hq, hkv, dim, page, seed=rot, rot=rot)
    ref = reference(off, kv, table, qkv, rope, kp, vp, hq, hkv, dim, page, pairs)
    q = bd.bitdelta_kv_append(batch, qkv, rope, kp, vp, interleaved=pairs)
    close(q, ref[0], ref[3], "q")
    close(kp, ref[1], ref[4], "k")
    assert np.array_equal(vp.double().cpu().numpy(), ref[2])
    assert bd.bitdelta_check_error() == 0


def test_no_rope_copies():
    batch, off, kv, table, qkv, rope, kp, vp = make([(2, 2), (1, 40)], 4, 2, 128, 16)
    q = bd.bitdelta_kv_append(batch, qkv, None, kp, vp)
    assert torch.equal(q.view(3, -1), qkv[:, :4 * 128])
    assert torch.equal(kp[table[1, 2], :, 7], qkv[2, 4 * 128:6 * 128].view(2, 128))


def test_tokens_without_any_sequence():
    """A batch of padding alone: zero queries, nothing appended."""
    empty = torch.zeros(0, dtype=torch.int32, device="cuda")
    batch = bd.AttentionBatch(torch.zeros(1, dtype=torch.int32, device="cuda"), empty,
                              empty.view(0, 4), 3, 1, 64, 4, 2, 64, 16)
    qkv = torch.randn(3, 8 * 64, device="cuda").to(torch.bfloat16)
    kp = torch.randn(2, 2, 16, 64, device="cuda").to(torch.bfloat16)
    vp, k0 = kp.clone(), kp.clone()
    q = torch.full((3, 4, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    bd.bitdelta_kv_append(batch, qkv, None, kp, vp, out=q)
    assert (q == 0).all() and torch.equal(kp, k0) and torch.equal(vp, k0)
    assert bd.bitdelta_check_error() == 0


def test_places_outside_are_reported_and_left_alone():
    batch, off, kv, table, qkv, rope, kp, vp = make([(2, 20), (1, 5)], 4, 2, 64, 16, rope_rows=19)
    k0, v0 = kp.clone(), vp.clone()
    q = bd.bitdelta_kv_append(batch, qkv, rope, kp, vp)    # position 19 has no rope row
    assert bd.bitdelta_check_error() == 7
    assert (q[1] == 0).all() and (q[0] != 0).any() and (q[2] != 0).any()
    pg = table[0, 1]
    assert torch.equal(kp[pg, :, 3], k0[pg, :, 3]) and torch.equal(vp[pg, :, 3], v0[pg, :, 3])
    bad = torch.full((1, 1), kp.shape[0], dtype=torch.int32).cuda()   # one page too far
    b2 = bd.AttentionBatch(torch.tensor([0, 1], dtype=torch.int32).cuda(),
                           torch.tensor([1], dtype=torch.int32).cuda(), bad, 1, 1, 1, 4, 2, 64, 16)
    k1 = kp.clone()
    q = bd.bitdelta_kv_append(b2, qkv[:1].contiguous(), rope, kp, vp)
    assert bd.bitdelta_check_error() == 7
    assert (q == 0).all() and torch.equal(kp, k1)


def test_cache_offsets_past_32_bits():
    """A cache whose element offsets pass 2^32: the last page is written."""
    hkv, page, dim = 8, 128, 128
    n_pages = (2 ** 32) // (hkv * page * dim) + 8
    kp = torch.zeros((n_pages, hkv, page, dim), dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    table = torch.tensor([[n_pages - 1]], dtype=torch.int32).cuda()
    batch = bd.AttentionBatch(torch.tensor([0, 1], dtype=torch.int32).cuda(),
                              torch.tensor([128], dtype=torch.int32).cuda(), table, 1, 1, 128, 8,
                              hkv, dim, page)
    qkv = torch.ones((1, 24 * dim), dtype=torch.bfloat16, device="cuda")
    bd.bitdelta_kv_append(batch, qkv, None, kp, vp)
    assert (kp[-1, :, 127] == 1).all() and (vp[-1, :, 127] == 1).all()
    assert kp[-1].sum().item() == hkv * dim and (kp[0] == 0).all() and (kp[7] == 0).all()
    assert bd.bitdelta_check_error() == 0


def test_refusals():
    batch, off, kv, table, qkv, rope, kp, vp = make([(2, 20)], 4, 2, 64, 16)
    for kw in (dict(qkv=qkv[:1]), dict(qkv=qkv.float()), dict(rope=rope.double()),
               dict(kp=kp[:, :1].contiguous()), dict(vp=vp[:, :, :8].contiguous()),
               dict(kp=kp.transpose(1, 2))):
        a = {"qkv": qkv, "rope": rope, "kp": kp, "vp": vp, **kw}
        with pytest.raises(ValueError):
            bd.bitdelta_kv_append(batch, a["qkv"], a["rope"], a["kp"], a["vp"])
    with pytest.raises(bd.BitDeltaError):     # rot_dim not a multiple of 16
        bd.bitdelta_kv_append(batch, qkv, rope[:, :24].contiguous(), kp, vp)
    with pytest.raises(bd.BitDeltaError):     # rot_dim above head_dim
        bd.bitdelta_kv_append(batch, qkv, torch.cat([rope, rope], 1), kp, vp)


@pytest.mark.parametrize("what", ["not sorted", "past the tokens", "negative offset", "max_q_len",
                                  "max_kv_len", "negative length"])
def test_lengths_that_break_the_batch_are_reported(what):
    """As the batch says of all its calls: queries of zeros, nothing appended."""
    batch, off, kv, table, qkv, rope, kp, vp = make([(2, 20), (1, 5), (4, 9)], 4, 2, 64, 16)
    k0, v0 = kp.clone(), vp.clone()
    offs, lens, most_q, most_kv = off.copy(), kv.copy(), 4, 20
    if what == "not sorted":
        offs[1:3] = [5, 3]                       # tokens 3 and 4 in two sequences
    elif what == "past the tokens":
        offs[3] = 8
    elif what == "negative offset":
        offs[0] = -1
    elif what == "max_q_len":
        most_q = 3
    elif what == "max_kv_len":
        most_kv = 19
    else:
        lens[1] = -5
    b = bd.AttentionBatch(torch.from_numpy(offs).cuda(), torch.from_numpy(lens).cuda(),
                          torch.from_numpy(table).cuda(), 7, most_q, most_kv, 4, 2, 64, 16)
    assert bd.bitdelta_check_error() == 7        # of the plan
    q = torch.full((7, 4, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    bd.bitdelta_kv_append(b, qkv, rope, kp, vp, out=q)
    assert bd.bitdelta_check_error() == 7
    assert (q == 0).all() and torch.equal(kp, k0) and torch.equal(vp, v0)
