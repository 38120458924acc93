"""The entry points of include/bitdelta_decode.h are exported as declared and reject bad
arguments on the host before touching the GPU (no GPU needed)."""
import ctypes
import os
import re
import subprocess

import pytest

import bit_weight_delta_gb300 as bd

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, SHAPE, MISALIGNED, WORKSPACE = 0, 1, 2, 3, 4
GOOD, BAD, ODD = 0x100000, 0x100008, 0x100002     # never dereferenced
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
    text = open(os.path.join(ROOT, "include", "bitdelta_decode.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    declared = set(re.findall(r"\b(bitdelta_\w+)\s*\(", text))
    out = subprocess.run(["nm", "-D", "--defined-only", bd.library_path()], capture_output=True,
                         text=True, check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if line.strip()}
    assert declared and declared <= exported
    assert set(bd.DECODE_EXPORTED) == declared


def test_the_header_compiles_as_c(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "bitdelta_decode.h"\nint main(void) { return 0; }')
    subprocess.run(["gcc", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-c", str(src), "-o",
                    str(tmp_path / "t.o")], check=True)


def test_sample(lib):
    base = dict(x=GOOD, M=4, V=100, stride=100, u=GOOD, t=None, k=None, p=None, m=None, tok=GOOD,
                prob=None)

    def call(**kw):
        a = {**base, **kw}
        return lib.bitdelta_sample(a["x"], a["M"], a["V"], a["stride"], a["u"], a["t"], a["k"],
                                   a["p"], a["m"], a["tok"], a["prob"], None)

    assert call(M=-1) == INVALID
    assert call(V=0) == INVALID
    assert call(stride=99) == INVALID
    assert call(V=524033, stride=HUGE) == SHAPE
    assert call(M=HUGE) == SHAPE
    assert call(stride=HUGE) == SHAPE
    for name in ("x", "u", "tok"):
        assert call(**{name: None}) == INVALID
    assert call(x=0x100001) == MISALIGNED
    for name in ("u", "t", "k", "p", "m", "tok", "prob"):
        assert call(**{name: ODD}) == MISALIGNED
    assert call(M=0, x=None, u=None, tok=None) == OK


@pytest.mark.parametrize("bad,status", [
    (dict(n_tokens=-1), INVALID), (dict(n_q_heads=0), INVALID), (dict(n_q_heads=9), SHAPE),
    (dict(head_dim=96), SHAPE), (dict(page_size=24), SHAPE), (dict(n_pages=1 << 31), SHAPE),
    (dict(n_group=3), SHAPE), (dict(kv_len=None), INVALID), (dict(n_group=1), INVALID),
    (dict(kv_len=ODD), MISALIGNED)])
def test_batch(lib, bad, status):
    b = batch(**bad)
    ref = ctypes.addressof(b)
    assert lib.bitdelta_kv_append_at(ref, GOOD, GOOD, GOOD, 64, 64, 0, GOOD, GOOD, GOOD, None) == status
    assert lib.bitdelta_kv_weigh(ref, GOOD, GOOD, GOOD, 1.0, 0, None, GOOD, GOOD, GOOD, HUGE,
                                 None) == status
    assert lib.bitdelta_kv_evict(ref, GOOD, 0, 0, None, GOOD, GOOD, GOOD, GOOD, GOOD, GOOD,
                                 None) == status
    assert lib.bitdelta_kv_evict_lengths(ref, GOOD, GOOD, GOOD, None) == status
    assert lib.bitdelta_kv_weigh_workspace_bytes(ref) == 0


def test_kv_append_at(lib):
    b = batch()
    base = dict(b=ctypes.addressof(b), off=GOOD, qkv=GOOD, rope=GOOD, rows=64, rot=128, style=0, k=GOOD,
                v=GOOD, q=GOOD)

    def call(**kw):
        a = {**base, **kw}
        return lib.bitdelta_kv_append_at(a["b"], a["off"], a["qkv"], a["rope"], a["rows"], a["rot"],
                                         a["style"], a["k"], a["v"], a["q"], None)

    assert call(b=None) == INVALID
    assert call(off=ODD) == MISALIGNED
    assert call(rot=24) == SHAPE
    assert call(rope=None) == INVALID
    for name in ("qkv", "k", "v", "q"):
        assert call(**{name: None}) == INVALID
        assert call(**{name: BAD}) == MISALIGNED


def test_kv_weigh(lib):
    b = batch()
    base = dict(b=ctypes.addressof(b), q=GOOD, lse=GOOD, k=GOOD, scale=1.0, window=0, off=None, w=GOOD,
                pos=GOOD, ws=GOOD, wb=HUGE)

    def call(**kw):
        a = {**base, **kw}
        return lib.bitdelta_kv_weigh(a["b"], a["q"], a["lse"], a["k"], a["scale"], a["window"],
                                     a["off"], a["w"], a["pos"], a["ws"], a["wb"], None)

    assert call(b=None) == INVALID
    for scale in (0.0, -1.0, float("inf"), float("nan"), 3e38):
        assert call(scale=scale) == INVALID
    assert call(scale=2.0 ** -101) == INVALID
    assert call(window=-1) == INVALID
    for name in ("q", "lse", "k", "w", "pos"):
        assert call(**{name: None}) == INVALID
    for name in ("q", "k"):
        assert call(**{name: BAD}) == MISALIGNED
    for name in ("lse", "w", "pos", "off"):
        assert call(**{name: ODD}) == MISALIGNED
    assert call(ws=None) == WORKSPACE
    assert call(wb=100) == WORKSPACE
    assert call(ws=0x100010) == MISALIGNED
    for empty in (batch(n_tokens=0), batch(n_seq=0)):
        assert call(b=ctypes.addressof(empty), q=None) == OK
    assert call(b=ctypes.addressof(batch(n_pages=0))) == INVALID
    # the joined blocks' parts: 2 per SM
    assert lib.bitdelta_kv_weigh_workspace_bytes(base["b"]) >= 2 * 1024


def test_kv_evict(lib):
    b = batch()
    base = dict(b=ctypes.addressof(b), keep=GOOD, recent=0, sink=0, off=None, k=GOOD, v=GOOD, w=GOOD,
                pos=GOOD, wo=GOOD, po=GOOD)

    def call(**kw):
        a = {**base, **kw}
        return lib.bitdelta_kv_evict(a["b"], a["keep"], a["recent"], a["sink"], a["off"], a["k"],
                                     a["v"], a["w"], a["pos"], a["wo"], a["po"], None)

    assert call(b=None) == INVALID
    assert call(recent=-1) == INVALID
    assert call(sink=-1) == INVALID
    for name in ("keep", "k", "v", "w", "pos", "wo", "po"):
        assert call(**{name: None}) == INVALID
    for name in ("k", "v", "w", "pos", "wo", "po"):
        assert call(**{name: BAD}) == MISALIGNED
    for name in ("keep", "off"):
        assert call(**{name: ODD}) == MISALIGNED
    assert call(b=ctypes.addressof(batch(page_table=None, n_tokens=0))) == INVALID
    assert call(b=ctypes.addressof(batch(max_kv_len=344065))) == SHAPE
    assert call(b=ctypes.addressof(batch(n_seq=1 << 20, n_q_heads=1024, n_kv_heads=1024, n_pages=1))) == SHAPE
    assert call(b=ctypes.addressof(batch(n_seq=0)), keep=None) == OK


def test_kv_evict_lengths(lib):
    b = batch()
    ref = ctypes.addressof(b)
    assert lib.bitdelta_kv_evict_lengths(None, GOOD, GOOD, GOOD, None) == INVALID
    assert lib.bitdelta_kv_evict_lengths(ref, None, GOOD, GOOD, None) == INVALID
    assert lib.bitdelta_kv_evict_lengths(ref, GOOD, None, GOOD, None) == INVALID
    assert lib.bitdelta_kv_evict_lengths(ref, GOOD, GOOD, None, None) == INVALID
    assert lib.bitdelta_kv_evict_lengths(ref, GOOD, ODD, GOOD, None) == MISALIGNED
    assert lib.bitdelta_kv_evict_lengths(ref, GOOD, GOOD, ODD, None) == MISALIGNED
    empty = batch(n_seq=0)
    assert lib.bitdelta_kv_evict_lengths(ctypes.addressof(empty), None, None, None, None) == OK


def test_lengths_refuse_the_batches_that_the_eviction_refuses(lib):
    for bad in (dict(max_kv_len=344065),
                dict(n_seq=1 << 20, n_q_heads=1024, n_kv_heads=1024, n_pages=1)):
        ref = batch(**bad)
        assert lib.bitdelta_kv_evict(ctypes.addressof(ref), GOOD, 0, 0, None, GOOD, GOOD, GOOD, GOOD,
                                     GOOD, GOOD, None) == SHAPE
        assert lib.bitdelta_kv_evict_lengths(ctypes.addressof(ref), GOOD, GOOD, GOOD, None) == SHAPE
    odd = batch(n_tokens=0, page_table=ODD)
    assert lib.bitdelta_kv_evict_lengths(ctypes.addressof(odd), GOOD, GOOD, GOOD, None) == MISALIGNED
