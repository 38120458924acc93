"""The decoder-block calls run on their tensors' device, whichever is current,
and refuse tensors of several devices before any launch (no GPU needed: the
tensors, the library and the device guard are stand-ins)."""
import contextlib
import ctypes

import numpy as np
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import bit_weight_delta_gb300 as bd

BF16, F32, I32, I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64


class Tensor:
    """An int32 CUDA tensor as AttentionBatch looks at it."""
    is_cuda, dtype = True, torch.int32

    def __init__(self, *shape, device=1):
        self.shape, self.device = shape, torch.device("cuda", device)
        self.recorded = []         # streams

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x100000


class Stream:
    def __init__(self, handle, device):
        self.cuda_stream, self.device = handle, torch.device("cuda", device)


class World:
    """The current device and streams, and what the library was called with under which."""

    def __init__(self, monkeypatch):
        self.current, self.streams, self.calls = 0, {0: 0x66, 1: 0x77}, []

        @contextlib.contextmanager
        def guard(device):
            before, self.current = self.current, torch.device(device).index
            yield
            self.current = before

        @contextlib.contextmanager
        def on(stream):
            with guard(stream.device):
                before = self.streams[self.current]
                self.streams[self.current] = stream.cuda_stream
                yield
                self.streams[self.current] = before

        def call(name, result):
            def f(*args):
                self.calls.append((name, self.current, args[-1]))
                return result
            return f

        def used_by_current_stream(ref, tensors):
            stream = self.streams[bd._BatchState.from_address(ref).device]
            for t in tensors:
                t.recorded.append(stream)
            return stream

        self.lib = type("Lib", (), {})()
        self.lib.bitdelta_attention_plan_bytes = call("plan_bytes", 512)
        self.lib.bitdelta_attention_workspace_bytes = call("workspace_bytes", 1024)
        self.lib.bitdelta_attention_plan = call("plan", 0)
        native = type("Native", (), {})()
        native.used_by_current_stream = used_by_current_stream
        monkeypatch.setattr(bd, "load", lambda *a: self.lib)
        monkeypatch.setattr(bd, "_native", native)
        monkeypatch.setattr(torch, "empty",
                            lambda n, dtype, device: Tensor(n, device=device.index))
        monkeypatch.setattr(torch.cuda, "device", guard)
        monkeypatch.setattr(torch.cuda, "stream", on)


@pytest.fixture
def world(monkeypatch):
    return World(monkeypatch)


def batch(**over):
    a = dict(seq_offsets=Tensor(3), kv_len=Tensor(2), page_table=Tensor(2, 4), **over)
    return bd.AttentionBatch(a.pop("seq_offsets"), a.pop("kv_len"), a.pop("page_table"), 4, 2, 64,
                             8, 2, 128, 16, **a)


def test_sizes_and_plan_on_the_tensors_device(world):
    b = batch()
    assert [(n, d) for n, d, _ in world.calls] == [("plan_bytes", 1), ("workspace_bytes", 1),
                                                   ("plan", 1)]
    assert world.calls[-1][2] == 0x77                # that device's current stream
    assert b._plan.device.index == b._ws.device.index == 1
    b.plan(Stream(0x99, 1))
    assert world.calls[-1] == ("plan", 1, 0x99)
    assert world.current == 0


@pytest.mark.parametrize("name", ["group_offsets", "prefix_len"])
def test_batch_tensors_of_two_devices(world, name):
    groups = {"group_offsets": Tensor(2), "prefix_len": Tensor(1)}
    batch(**groups)
    groups[name].device = torch.device("cuda", 0)
    with pytest.raises(ValueError, match="one device"):
        batch(**groups)
    with pytest.raises(ValueError, match="one device"):
        bd.AttentionBatch(Tensor(3, device=0), Tensor(2), Tensor(2, 4), 4, 2, 64, 8, 2, 128, 16)


def test_a_stream_of_another_device(world):
    with pytest.raises(ValueError, match="stream"):
        batch(stream=Stream(0x99, 0))
    b = batch()
    with pytest.raises(ValueError, match="stream"):
        b.plan(Stream(0x99, 0))
    for f in (lambda s: bd.bitdelta_add_norm(Tensor(4, 64), stream=s),
              lambda s: bd.bitdelta_kv_append(b, Tensor(4, 64), None, None, None, stream=s),
              lambda s: bd.bitdelta_attention(b, Tensor(4, 64), None, None, stream=s)):
        with pytest.raises(ValueError, match="stream"):
            f(Stream(0x99, 0))


def test_the_plans_stream_is_recorded(world):
    """On every tensor of the batch: its memory outlives the work on that stream."""
    lengths = dict(seq_offsets=Tensor(3), kv_len=Tensor(2), page_table=Tensor(2, 4),
                   group_offsets=Tensor(2), prefix_len=Tensor(1))
    b = bd.AttentionBatch(**lengths, n_tokens=4, max_q_len=2, max_kv_len=64, n_q_heads=8,
                          n_kv_heads=2, head_dim=128, page_size=16)
    every = [b._plan, b._ws, *lengths.values()]
    assert len(b._tensors) == len(every) and all(x is y for x, y in zip(b._tensors, every))
    assert all(t.recorded == [0x77] for t in every)
    b.plan(Stream(0x99, 1))
    assert all(t.recorded == [0x77, 0x99] for t in every)
    b = batch(stream=Stream(0x55, 1))
    assert all(t.recorded == [0x55] for t in b._tensors)


def test_bounds_that_do_not_fit_the_struct(world):
    """2^32 + 64 keys would be 64 of them to the library."""
    sizes = [4, 2, 64, 8, 2, 128, 16]
    for i in range(1, len(sizes)):
        wrapped = sizes[:i] + [sizes[i] + 2 ** 32] + sizes[i + 1:]
        with pytest.raises(ValueError, match="32 bits"):
            bd.AttentionBatch(Tensor(3), Tensor(2), Tensor(2, 4), *wrapped)
    assert world.calls == []


def fake(dtype, *shape, device=0):
    return torch.empty(shape, dtype=dtype, device=f"cuda:{device}")


def test_add_norm_refuses_another_device():
    with FakeTensorMode():
        args = dict(y=fake(BF16, 4, 64), residual=fake(F32, 4, 64), pre_table=fake(I64, 2),
                    post_table=fake(I64, 2), gate=fake(BF16, 64), seg_offsets=fake(I32, 2),
                    seg_variant=fake(I32, 1), residual_out=fake(F32, 4, 64), out=fake(BF16, 4, 64))
        for name, t in args.items():
            other = torch.empty(t.shape, dtype=t.dtype, device="cuda:1")
            with pytest.raises(ValueError, match="another device"):
                bd.bitdelta_add_norm(**{**args, name: other})


class Batch:
    """A batch whose tables, plan and workspace lie on a device."""

    def __init__(self, device):
        self._state = bd._BatchState(bd._AttentionBatch(4, 2, 2, 64, 8, 2, 128, 16, 0, 4), device)
        self._ref = ctypes.addressof(self._state)
        self._tensors = ()
        self._args = (self._ref, (), 0x100000, 1 << 40, 0x100000, 1 << 40)


def test_append_and_attention_refuse_another_device():
    with FakeTensorMode():
        append = dict(qkv=fake(BF16, 4, 12 * 128), rope=fake(F32, 64, 128),
                      k_pages=fake(BF16, 3, 2, 16, 128), v_pages=fake(BF16, 3, 2, 16, 128),
                      out=fake(BF16, 4, 8, 128))
        attention = dict(q=fake(BF16, 4, 8, 128), k_pages=append["k_pages"],
                         v_pages=append["v_pages"], out=append["out"], lse=fake(F32, 4, 8))
        for call, args in ((bd.bitdelta_kv_append, append), (bd.bitdelta_attention, attention)):
            for name, t in args.items():
                other = torch.empty(t.shape, dtype=t.dtype, device="cuda:1")
                with pytest.raises(ValueError, match="another device"):
                    call(Batch(0), **{**args, name: other})
            with pytest.raises(ValueError, match="another device"):
                call(Batch(1), **args)               # all but the batch on device 0


def test_norm_weights_shorter_than_a_row_are_refused():
    """norm_table's length travels with the table; weights shorter than a row would be
    read past their end."""
    class Weight(Tensor):
        dtype = torch.bfloat16

    for weights in ([], [Weight(64), Weight(32)], [Weight(64), Weight(64, device=0)]):
        with pytest.raises(ValueError):
            bd.norm_table(weights)
    with FakeTensorMode():
        y, short, right = fake(BF16, 4, 64), fake(I64, 2), fake(I64, 2)
        short.norm_width, right.norm_width = 32, 64
        for kw in (dict(pre_table=short), dict(pre_table=right, post_table=short)):
            with pytest.raises(ValueError, match="shorter"):
                bd.bitdelta_add_norm(y, **kw)


def test_an_argument_without_a_truth_value():
    """Its own error, not a call that succeeds with an error set."""
    with FakeTensorMode():
        cache = fake(BF16, 3, 2, 16, 128)
        with pytest.raises(ValueError, match="truth value"):
            bd.bitdelta_kv_append(Batch(0), fake(BF16, 4, 12 * 128), None, cache, cache,
                                  interleaved=np.zeros(2))
