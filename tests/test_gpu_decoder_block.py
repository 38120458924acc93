"""The block example end to end: prompts and single tokens of the base model and
two variants in one batch, two steps over one cache, against the same block in
64 bits.  The bound is on the 2-norm: eight bf16 roundings lie on the path (each
2^-9 relative), the projections' share of the residual is of its own size, so
the streams agree within 2^-6."""
import os
import sys

import pytest
import torch

import bit_weight_delta_gb300 as bd

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))
import decoder_block as ex  # noqa: E402

pytestmark = pytest.mark.gpu


class Reference:
    """The block in float64 on whole sequences, keys and values kept per sequence."""

    def __init__(self, block, n_seq):
        self.b = block
        self.w = {}
        for name, (base, packs, _) in block.linears.items():
            self.w[name] = [base.double()]
            for packed, alpha in packs:
                self.w[name].append(bd.bitdelta_reconstruct(base, packed, alpha, per_row=True).double())
        self.k, self.v = [None] * n_seq, [None] * n_seq

    def norm(self, name, h, v):
        return h / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-5) * self.b.norms[name][0][v].double()

    def step(self, s, variant, h, rope):
        b, t = self.b, h.shape[0]
        qkv = (self.norm("attn", h, variant) @ self.w["qkv"][variant].T).view(t, -1, b.dim)
        start = 0 if self.k[s] is None else self.k[s].shape[0]
        cos, sin = rope[start:start + t].double()[:, None].chunk(2, dim=-1)
        x, y = qkv[:, :b.hq + b.hkv].chunk(2, dim=-1)
        rot = torch.cat([x * cos - y * sin, y * cos + x * sin], -1)
        k, v = rot[:, b.hq:], qkv[:, b.hq + b.hkv:]
        self.k[s] = k if start == 0 else torch.cat([self.k[s], k])
        self.v[s] = v if start == 0 else torch.cat([self.v[s], v])
        g = b.hq // b.hkv
        keys = self.k[s].repeat_interleave(g, 1).transpose(0, 1)
        vals = self.v[s].repeat_interleave(g, 1).transpose(0, 1)
        a = rot[:, :b.hq].transpose(0, 1) @ keys.transpose(1, 2) / b.dim ** 0.5
        later = torch.ones_like(a[0], dtype=torch.bool).triu(start + 1)
        o = torch.softmax(a.masked_fill(later, float("-inf")), -1) @ vals
        h = h + o.transpose(0, 1).reshape(t, -1) @ self.w["o"][variant].T
        gate, up = (self.norm("mlp", h, variant) @ self.w["gate_up"][variant].T).chunk(2, 1)
        h = h + (torch.nn.functional.silu(gate) * up) @ self.w["down"][variant].T
        return h, self.norm("next", h, variant)


def test_prompt_and_decode_steps():
    hidden, ffn, hq, hkv, dim, page = 512, 1024, 8, 2, 64, 16
    block = ex.Block(hidden, ffn, hq, hkv, dim, variants=2, seed=3)
    variant, prompts = [0, 1, 2, 1, 0], [70, 1, 33, 129, 5]
    width = 12
    perm = torch.randperm(len(prompts) * width, generator=torch.Generator().manual_seed(0))
    table = perm.view(len(prompts), width).to(torch.int32).cuda()
    kp = torch.full((len(prompts) * width, hkv, page, dim), float("nan"), dtype=torch.bfloat16,
                    device="cuda")
    vp = kp.clone()
    rope = ex.rope_table(width * page, dim)
    ref = Reference(block, len(prompts))
    g = torch.Generator(device="cuda").manual_seed(1)
    lens = [0] * len(prompts)
    for q_len in (prompts, [1] * 5, [1, 40, 1, 2, 1], [1] * 5):
        lens = [a + b for a, b in zip(lens, q_len)]
        offs = [sum(q_len[:i]) for i in range(len(q_len) + 1)]
        seg = (ex.int32(offs), ex.int32(variant), max(q_len))
        batch = bd.AttentionBatch(seg[0], ex.int32(lens), table, offs[-1], max(q_len), max(lens), hq,
                                  hkv, dim, page)
        h = torch.randn((offs[-1], hidden), generator=g, device="cuda")
        h1, x1 = block.forward(h, seg, batch, rope, kp, vp)
        assert bd.bitdelta_check_error() == 0
        for s, v in enumerate(variant):
            want_h, want_x = ref.step(s, v, h[offs[s]:offs[s + 1]].double(), rope)
            for got, want in ((h1, want_h), (x1, want_x)):
                err = (got[offs[s]:offs[s + 1]].double() - want).norm() / want.norm()
                assert err <= 2.0 ** -6, (s, err.item())
