"""bitdelta_add_norm against the formula in 64 bits.

Tolerances (derived before the first run): h is one fp32 sum, so within 2^-20
of the terms' magnitudes plus, for a bf16 residual, half an ulp (2^-9 of the
value, 2^-8 allowed).  x multiplies h by an inverse root of an fp32 mean (d
additions in a tree, 2^-18 allowed) and a weight, and is rounded once to bf16."""
import numpy as np
import pytest
import torch

import bit_weight_delta_gb300 as bd

pytestmark = pytest.mark.gpu
EPS = 1e-5


def rand(g, *shape, std=1.0, mean=0.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dtype)


def reference(y, res, pre, post, gate, scale, slots):
    y, pre = y.double().cpu(), pre.double().cpu()
    b = y
    if post is not None:
        b = y / torch.sqrt((y * y).mean(1, keepdim=True) + EPS) * post.double().cpu()[slots]
    if gate is not None:
        b = b * gate.double().cpu()
    r = torch.zeros_like(y) if res is None else res.double().cpu()
    h = r + scale * b
    x = h / torch.sqrt((h * h).mean(1, keepdim=True) + EPS) * pre[slots]
    return h, x, r.abs() + abs(scale) * b.abs()


def check(h, x, href, xref, mag, rtype):
    h, x = h.double().cpu(), x.double().cpu()
    tol = 2.0 ** -20 * mag + 2.0 ** -18 * mag * 0.25
    if rtype is torch.bfloat16:
        tol = tol + 2.0 ** -8 * href.abs()
    assert ((h - href).abs() <= tol).all(), (h - href).abs().max()
    # h's error reaches x through the same factor x/h
    factor = torch.where(href != 0, (xref / href).abs(), torch.zeros_like(href))
    xtol = 2.0 ** -8 * xref.abs() + 2.0 ** -17 * xref.abs() + factor * (2.0 ** -18 * mag) + 1e-30
    assert ((x - xref).abs() <= xtol).all(), (x - xref).abs().max()


@pytest.mark.parametrize("rtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,d", [(1, 8), (3, 264), (8, 8192), (130, 4096), (5, 1000),
                                    (2, 16384), (2, 32776), (1, 65536), (700, 1024)])
def test_plain_residual(rows, d, rtype):
    g = torch.Generator(device="cuda").manual_seed(rows * d)
    y, res = rand(g, rows, d), rand(g, rows, d, std=3.0, dtype=rtype)
    pre = rand(g, 1, d, std=0.1, mean=1.0)
    h, x = bd.bitdelta_add_norm(y, res, bd.norm_table(list(pre)), eps=EPS)
    check(h, x, *reference(y, res, pre, None, None, 1.0, [0] * rows), rtype)
    assert bd.bitdelta_check_error() == 0


@pytest.mark.parametrize("rows,d", [(609, 8192), (700, 6152), (308, 16384), (305, 32776)])
@pytest.mark.parametrize("residual", ["none", "other", "same"])
def test_more_rows_than_run_at_once(rows, d, residual):
    """Wide bf16 rows in several rounds of CTAs, which are fetched ahead; the
    residual absent, of its own, or updated in place."""
    g = torch.Generator(device="cuda").manual_seed(rows + d)
    y, pre = rand(g, rows, d), rand(g, 1, d, std=0.1, mean=1.0)
    res = None if residual == "none" else rand(g, rows, d, std=2.0)
    ref = reference(y, res, pre, None, None, 1.0, [0] * rows)
    h, x = bd.bitdelta_add_norm(y, res, bd.norm_table(list(pre)), eps=EPS,
                                residual_out=res if residual == "same" else None)
    check(h, x, *ref, torch.bfloat16)
    assert bd.bitdelta_check_error() == 0


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", ["none", "channel", "row"])
@pytest.mark.parametrize("rtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,d", [(5, 512), (67, 2056), (33, 9000)])
def test_segments_gate_and_post_norm(rows, d, rtype, gate, post):
    g = torch.Generator(device="cuda").manual_seed(d)
    n_tab = 4
    y, res = rand(g, rows, d), rand(g, rows, d, std=2.0, dtype=rtype)
    pre, pw = rand(g, n_tab, d, std=0.2, mean=1.0), rand(g, n_tab, d, std=0.2, mean=0.5)
    gt = {"none": None, "channel": rand(g, d), "row": rand(g, rows, d)}[gate]
    cuts = [0, 1, 2, 2, rows // 2, rows]       # an empty segment among them
    ids = [3, 0, 1, 2, 1]
    slots = [ids[s] for s in range(5) for _ in range(cuts[s + 1] - cuts[s])]
    h, x = bd.bitdelta_add_norm(
        y, res, bd.norm_table(list(pre)), post_table=bd.norm_table(list(pw)) if post else None,
        gate=gt, scale=-0.625, eps=EPS,
        seg_offsets=torch.tensor(cuts, dtype=torch.int32).cuda(),
        seg_variant=torch.tensor(ids, dtype=torch.int32).cuda())
    check(h, x, *reference(y, res, pre, pw if post else None, gt, -0.625, slots), rtype)
    assert bd.bitdelta_check_error() == 0


def test_in_place_residual_and_no_residual():
    g = torch.Generator(device="cuda").manual_seed(1)
    y, res = rand(g, 9, 4096), rand(g, 9, 4096, dtype=torch.float32)
    table = bd.norm_table(list(rand(g, 1, 4096)))
    h, x = bd.bitdelta_add_norm(y, res, table)
    r2 = res.clone()
    h2, x2 = bd.bitdelta_add_norm(y, r2, table, residual_out=r2)
    assert h2.data_ptr() == r2.data_ptr()
    assert torch.equal(h, h2) and torch.equal(x, x2)
    h3, _ = bd.bitdelta_add_norm(y, None, table)     # h = y
    assert torch.equal(h3, y)


def test_zero_rows_and_rows_of_zeros():
    table = bd.norm_table([torch.ones(64, dtype=torch.bfloat16, device="cuda")])
    y = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda")
    h, x = bd.bitdelta_add_norm(y, None, table)
    assert h.shape == x.shape == (0, 64)
    y = torch.zeros((3, 64), dtype=torch.bfloat16, device="cuda")
    h, x = bd.bitdelta_add_norm(y, None, table, post_table=table)
    assert (h == 0).all() and (x == 0).all()


def test_rows_outside_every_segment_are_left_alone():
    table = bd.norm_table([torch.ones(256, dtype=torch.bfloat16, device="cuda")])
    y = torch.ones((6, 256), dtype=torch.bfloat16, device="cuda")
    h = torch.full((6, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    x = h.clone()
    bd.bitdelta_add_norm(y, None, table, residual_out=h, out=x,
                         seg_offsets=torch.tensor([1, 4], dtype=torch.int32).cuda(),
                         seg_variant=torch.tensor([0], dtype=torch.int32).cuda())
    assert (h[1:4] == 1).all() and (h[[0, 4, 5]] == 7).all() and (x[[0, 4, 5]] == 7).all()


def test_a_bad_variant_id_is_reported():
    table = bd.norm_table([torch.ones(256, dtype=torch.bfloat16, device="cuda")])
    y = torch.ones((2, 256), dtype=torch.bfloat16, device="cuda")
    h, x = bd.bitdelta_add_norm(y, None, table,
                                seg_offsets=torch.tensor([0, 2], dtype=torch.int32).cuda(),
                                seg_variant=torch.tensor([5], dtype=torch.int32).cuda())
    assert bd.bitdelta_check_error() == 7
    assert (h == 1).all()
    assert bd.bitdelta_check_error() == 0


def test_another_stream_and_a_graph():
    g = torch.Generator(device="cuda").manual_seed(2)
    y, res = rand(g, 64, 4096), rand(g, 64, 4096)
    table = bd.norm_table(list(rand(g, 1, 4096)))
    h, x = bd.bitdelta_add_norm(y, res, table)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    h1, x1 = bd.bitdelta_add_norm(y, res, table, stream=s)
    s.synchronize()
    assert torch.equal(h, h1) and torch.equal(x, x1)
    h2, x2 = torch.empty_like(h), torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bd.bitdelta_add_norm(y, res, table, residual_out=h2, out=x2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(h, h2) and torch.equal(x, x2)


def test_refusals():
    y = torch.ones((2, 256), dtype=torch.bfloat16, device="cuda")
    table = bd.norm_table([torch.ones(256, dtype=torch.bfloat16, device="cuda")])
    with pytest.raises(ValueError):
        bd.bitdelta_add_norm(y)
    with pytest.raises(ValueError):
        bd.bitdelta_add_norm(y.float(), None, table)
    with pytest.raises(ValueError):
        bd.bitdelta_add_norm(y, y.half(), table)
    with pytest.raises(ValueError):
        bd.bitdelta_add_norm(y, y[:1], table)
    with pytest.raises(ValueError):
        bd.bitdelta_add_norm(y, None, table, gate=y[:1].reshape(-1)[:128])
    with pytest.raises(ValueError):
        bd.bitdelta_add_norm(y.t(), None, table)
    with pytest.raises(ValueError):
        bd.bitdelta_add_norm(y, None, table, seg_variant=torch.zeros(1, dtype=torch.int32).cuda())
    with pytest.raises(bd.BitDeltaError):
        bd.bitdelta_add_norm(torch.ones((2, 12), dtype=torch.bfloat16, device="cuda"), None, table)


def test_weights_shorter_than_a_row_are_refused():
    ones = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    y = torch.ones((2, 256), dtype=torch.bfloat16, device="cuda")
    right, short, long = (bd.norm_table([w, w]) for w in (ones, ones[:128], torch.cat([ones, ones])))
    for pre, post in ((short, None), (right, short)):
        with pytest.raises(ValueError):
            bd.bitdelta_add_norm(y, None, pre, post_table=post)
    with pytest.raises(ValueError):
        bd.norm_table([ones, ones[:128]])
    with pytest.raises(ValueError):
        bd.norm_table([])
    for table in (long, right.clone()):      # their first 256 elements; the caller's own pointers
        h, x = bd.bitdelta_add_norm(y, None, table)
        assert (h == 1).all()
    assert bd.bitdelta_check_error() == 0


@pytest.mark.parametrize("cuts", [[0, 4, 2, 6], [0, 2, 4, 7], [-1, 2, 4, 6], [3, 2, 1, 0]])
def test_malformed_segments_are_reported_and_write_nothing(cuts):
    """Overlapping segments, one past the rows, one before them."""
    table = bd.norm_table([torch.full((256,), i + 1.0, dtype=torch.bfloat16, device="cuda")
                           for i in range(3)])
    y = torch.ones((6, 256), dtype=torch.bfloat16, device="cuda")
    h = torch.full((6, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    x = h.clone()
    bd.bitdelta_add_norm(y, None, table, residual_out=h, out=x,
                         seg_offsets=torch.tensor(cuts, dtype=torch.int32).cuda(),
                         seg_variant=torch.tensor([0, 1, 2], dtype=torch.int32).cuda())
    assert bd.bitdelta_check_error() == 7
    assert (h == 7).all() and (x == 7).all()


def test_a_table_of_no_segments_writes_nothing():
    """As in the grouped linear: not a refusal, and not the whole batch on slot 0."""
    table = bd.norm_table([torch.ones(256, dtype=torch.bfloat16, device="cuda")])
    y = torch.ones((6, 256), dtype=torch.bfloat16, device="cuda")
    h = torch.full((6, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    x = h.clone()
    bd.bitdelta_add_norm(y, None, table, residual_out=h, out=x,
                         seg_offsets=torch.zeros(1, dtype=torch.int32).cuda(),
                         seg_variant=torch.zeros(0, dtype=torch.int32).cuda())
    assert (h == 7).all() and (x == 7).all()
    assert bd.bitdelta_check_error() == 0
