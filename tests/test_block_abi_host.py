"""The decoder-block entry points are exported as declared and reject bad
arguments on the host before touching the GPU (no GPU needed)."""
import ctypes
import os
import re
import subprocess

import pytest

import bit_weight_delta_gb300 as bd

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, SHAPE, MISALIGNED, WORKSPACE = 0, 1, 2, 3, 4
GOOD, BAD = 0x100000, 0x100008        # never dereferenced; BAD is off 16 bytes
HUGE = 1 << 40


@pytest.fixture(scope="module")
def lib():
    return bd.load()


def batch(**kw):
    a = dict(n_tokens=4, n_seq=2, max_q_len=2, max_kv_len=64, n_q_heads=8, n_kv_heads=2,
             head_dim=128, page_size=16, n_pages=10, table_stride=4, seq_offsets=GOOD,
             kv_len=GOOD, page_table=GOOD, n_group=0, group_offsets=None, prefix_len=None)
    a.update(kw)
    return bd._AttentionBatch(**a)


def test_declared_and_exported():
    text = open(os.path.join(ROOT, "include", "bitdelta_block.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    declared = set(re.findall(r"\b(bitdelta_\w+)\s*\(", text))
    out = subprocess.run(["nm", "-D", "--defined-only", bd.library_path()], capture_output=True,
                         text=True, check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if line.strip()}
    assert declared and declared <= exported
    assert set(bd.BLOCK_EXPORTED) == declared


def test_the_struct_matches_the_header(tmp_path):
    """Size and field offsets of the batch struct as the C compiler lays it out."""
    names = [n for n, _ in bd._AttentionBatch._fields_]
    src = tmp_path / "t.c"
    src.write_text('#include <stdio.h>\n#include "bitdelta_block.h"\nint main(void) {'
                   + "".join(f'printf("%zu ", offsetof(bd_attention_batch, {n}));' for n in names)
                   + 'printf("%zu", sizeof(bd_attention_batch)); return 0; }')
    exe = tmp_path / "t"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True,
                                          check=True).stdout.split()]
    assert got == [getattr(bd._AttentionBatch, n).offset for n in names] + [
        ctypes.sizeof(bd._AttentionBatch)]


def test_add_norm(lib):
    base = dict(y=GOOD, M=4, d=64, res=GOOD, res_out=GOOD, rtype=0, gate=None, gs=0, pre=GOOD,
                post=None, n_tab=1, so=None, sv=None, n_seg=0, x=GOOD)

    def call(**kw):
        a = {**base, **kw}
        return lib.bitdelta_add_norm(a["y"], a["M"], a["d"], a["res"], a["res_out"], a["rtype"],
                                     a["gate"], a["gs"], 1.0, 1e-5, a["pre"], a["post"],
                                     a["n_tab"], a["so"], a["sv"], a["n_seg"], a["x"], None)

    assert call(M=-1) == INVALID
    assert call(d=0) == INVALID
    assert call(y=None) == INVALID
    assert call(rtype=2) == INVALID
    assert call(gate=GOOD, gs=8) == INVALID
    assert call(so=GOOD) == INVALID
    assert call(n_seg=3) == INVALID
    assert call(pre=None) == INVALID
    assert call(n_tab=0) == INVALID
    assert call(x=None, res_out=None) == INVALID
    assert call(d=12) == SHAPE
    assert call(d=65544) == SHAPE
    assert call(M=HUGE) == SHAPE
    for name in ("y", "res", "res_out", "x"):
        assert call(**{name: BAD}) == MISALIGNED
    assert call(gate=BAD) == MISALIGNED
    assert call(M=0, y=None) == OK
    assert call(so=GOOD, sv=GOOD, n_seg=0) == OK


@pytest.mark.parametrize("bad,status", [
    (dict(n_tokens=-1), INVALID), (dict(n_seq=-1), INVALID), (dict(n_q_heads=0), INVALID),
    (dict(n_kv_heads=0), INVALID), (dict(n_q_heads=9), SHAPE), (dict(n_q_heads=66), SHAPE),
    (dict(head_dim=96), SHAPE), (dict(page_size=24), SHAPE), (dict(page_size=256), SHAPE),
    (dict(n_pages=1 << 31), SHAPE), (dict(n_group=3), SHAPE), (dict(seq_offsets=None), INVALID),
    (dict(kv_len=None), INVALID), (dict(page_table=None), INVALID), (dict(n_group=1), INVALID),
    (dict(kv_len=0x100002), MISALIGNED)])
def test_batch(lib, bad, status):
    b = batch(**bad)
    ref = ctypes.addressof(b)
    assert lib.bitdelta_attention_plan(ref, GOOD, HUGE, None) == status
    assert lib.bitdelta_attention(ref, GOOD, HUGE, GOOD, GOOD, GOOD, 1.0, GOOD, None, GOOD, HUGE,
                                  None) == status
    assert lib.bitdelta_kv_append(ref, GOOD, GOOD, 64, 64, 0, GOOD, GOOD, GOOD, None) == status
    assert lib.bitdelta_attention_plan_bytes(ref) == 0


def test_kv_append(lib):
    b = batch()
    base = dict(b=ctypes.addressof(b), qkv=GOOD, rope=GOOD, rows=64, rot=128, style=0, k=GOOD,
                v=GOOD, q=GOOD)

    def call(**kw):
        a = {**base, **kw}
        return lib.bitdelta_kv_append(a["b"], a["qkv"], a["rope"], a["rows"], a["rot"],
                                      a["style"], a["k"], a["v"], a["q"], None)

    assert call(b=None) == INVALID
    assert call(style=2) == INVALID
    assert call(rot=-16) == INVALID
    assert call(rows=-1) == INVALID
    assert call(rope=None) == INVALID
    assert call(rot=24) == SHAPE
    assert call(rot=144) == SHAPE
    for name in ("qkv", "k", "v", "q"):
        assert call(**{name: None}) == INVALID
        assert call(**{name: BAD}) == MISALIGNED
    empty = batch(n_tokens=0)
    assert call(b=ctypes.addressof(empty), qkv=None) == OK


def test_attention(lib):
    b = batch(n_group=1, group_offsets=GOOD, prefix_len=GOOD)
    base = dict(b=ctypes.addressof(b), plan=GOOD, pb=HUGE, q=GOOD, k=GOOD, v=GOOD, scale=1.0,
                out=GOOD, lse=None, ws=GOOD, wb=HUGE)

    def call(**kw):
        a = {**base, **kw}
        return lib.bitdelta_attention(a["b"], a["plan"], a["pb"], a["q"], a["k"], a["v"],
                                      a["scale"], a["out"], a["lse"], a["ws"], a["wb"], None)

    assert call(b=None) == INVALID
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert call(scale=scale) == INVALID
    for name in ("q", "k", "v", "out"):
        assert call(**{name: None}) == INVALID
        assert call(**{name: BAD}) == MISALIGNED
    assert call(plan=None) == WORKSPACE
    assert call(pb=16) == WORKSPACE
    assert call(plan=0x100010) == MISALIGNED
    assert call(ws=0x100010) == MISALIGNED
    assert lib.bitdelta_attention_plan(base["b"], None, HUGE, None) == WORKSPACE
    assert lib.bitdelta_attention_plan(base["b"], 0x100010, HUGE, None) == MISALIGNED


def test_attention_refuses_a_scale_that_overflows_in_base_2(lib):
    """Scores are scaled by scale·log2(e) in fp32: infinite times a zero score is no number."""
    b = batch()
    for scale, status in ((2.0 ** 127, None), (3e38, INVALID), (2.5e38, INVALID)):
        st = lib.bitdelta_attention(ctypes.addressof(b), GOOD, 16, GOOD, GOOD, GOOD, scale, GOOD,
                                    None, GOOD, HUGE, None)
        assert st == (WORKSPACE if status is None else status)    # 16 bytes hold no plan
