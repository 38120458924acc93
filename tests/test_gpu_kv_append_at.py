"""bitdelta_kv_append with positions that go on after an eviction: a token's slot is its
place in the shortened cache, its angle that of slot + pos_offset.  The same arithmetic
on other rows of the same table: results are those of a call with that table's rows
moved, bit for bit."""
import pytest
import torch

import bit_weight_delta_gb300 as bd

pytestmark = pytest.mark.gpu
HQ, HKV, DIM, PAGE = 6, 2, 64, 16


def make(lens, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = len(lens)
    off = [sum(q for q, _ in lens[:i]) for i in range(n + 1)]
    width = -(-max(k for _, k in lens) // PAGE)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    batch = bd.AttentionBatch(i32(off), i32([k for _, k in lens]),
                              i32([[s * width + i for i in range(width)] for s in range(n)]),
                              off[-1], max(q for q, _ in lens), max(k for _, k in lens), HQ, HKV, DIM,
                              PAGE)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
    pages = rn(n * width, HKV, PAGE, DIM)
    rope = torch.randn((500, DIM), generator=g, device="cuda")
    return batch, off, rn(off[-1], (HQ + 2 * HKV) * DIM), pages, pages * 2, rope, i32


@pytest.mark.parametrize("pairs", [False, True])
def test_positions_are_shifted(pairs):
    lens, shift = [(1, 40), (5, 5), (17, 90), (1, 1)], [100, 0, 409, 3]
    batch, off, qkv, kp, vp, rope, i32 = make(lens)
    k, v = kp.clone(), vp.clone()
    q = bd.bitdelta_kv_append(batch, qkv, rope, k, v, interleaved=pairs, pos_offset=i32(shift))
    assert bd.bitdelta_check_error() == 0
    for s, add in enumerate(shift):     # the whole batch by this sequence's rows
        k2, v2 = kp.clone(), vp.clone()
        moved = torch.cat([rope[add:], rope[:add]])
        q2 = bd.bitdelta_kv_append(batch, qkv, moved, k2, v2, interleaved=pairs)
        assert torch.equal(q[off[s]:off[s + 1]], q2[off[s]:off[s + 1]])
        width = kp.shape[0] // len(lens)
        for a, b in ((k, k2), (v, v2)):
            assert torch.equal(a[s * width:(s + 1) * width], b[s * width:(s + 1) * width])


def test_no_offset_is_an_offset_of_zero():
    batch, _, qkv, kp, vp, rope, i32 = make([(3, 50), (1, 7)], seed=1)
    a, b = (kp.clone(), vp.clone()), (kp.clone(), vp.clone())
    qa = bd.bitdelta_kv_append(batch, qkv, rope, *a)
    qb = bd.bitdelta_kv_append(batch, qkv, rope, *b, pos_offset=i32([0, 0]))
    assert torch.equal(qa, qb) and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("shift", [-50, 460, 2 ** 31 - 1, -2 ** 31])
def test_positions_outside_of_the_table_are_reported(shift):
    batch, off, qkv, kp, vp, rope, i32 = make([(2, 45), (2, 30)], seed=2)
    k = kp.clone()
    q = bd.bitdelta_kv_append(batch, qkv, rope, k, vp, pos_offset=i32([shift, 5]))
    assert bd.bitdelta_check_error() == 7
    assert (q[:2] == 0).all() and (q[2:] != 0).any()
    assert torch.equal(k[:3], kp[:3])


def test_without_a_table_positions_do_not_matter():
    batch, _, qkv, kp, vp, _, i32 = make([(2, 45)], seed=3)
    a, b = (kp.clone(), vp.clone()), (kp.clone(), vp.clone())
    qa = bd.bitdelta_kv_append(batch, qkv, None, *a)
    qb = bd.bitdelta_kv_append(batch, qkv, None, *b, pos_offset=i32([-7000]))
    assert bd.bitdelta_check_error() == 0
    assert torch.equal(qa, qb) and torch.equal(a[0], b[0])


def test_refusals():
    batch, _, qkv, kp, vp, rope, i32 = make([(2, 45), (1, 3)], seed=4)
    for bad in (i32([1]), i32([1, 2]).long(), i32([1, 2]).float(), i32([1, 2]).cpu(),
                i32([[1, 2]])):
        with pytest.raises(ValueError):
            bd.bitdelta_kv_append(batch, qkv, rope, kp, vp, pos_offset=bad)
