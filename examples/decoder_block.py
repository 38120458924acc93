"""One decoder block of a served model, for a batch that mixes the base model and
its variants, prompts and single tokens:

    x      = norm(h)                        bitdelta_add_norm
    qkv    = QKV projection                 bitdelta_linear_grouped
    q      = rotary positions, cache append bitdelta_kv_append
    o      = attention over the cache       bitdelta_attention
    a      = O projection                   bitdelta_linear_grouped
    h, x   = h + a, norm                    bitdelta_add_norm
    f      = gate+up projection             bitdelta_linear_grouped
    d      = down projection of silu(g)·u   bitdelta_linear_grouped
    h, x   = h + d, the next block's norm   bitdelta_add_norm

A variant is W_base + α·sign(Δ) in the four projections and has norm weights of
its own.  `python examples/decoder_block.py` runs a prompt step and decode steps
on a GPU and prints what each took.
"""
import os
import sys

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import bit_weight_delta_gb300 as bd


class Block:
    """Random weights of one block: the base model's and `variants` compressed ones."""

    def __init__(self, hidden, ffn, hq, hkv, dim, variants, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.hq, self.hkv, self.dim, self.variants = hq, hkv, dim, variants

        def normal(*shape, std, mean=0.0):
            return (torch.randn(shape, generator=g, device=device) * std + mean).to(torch.bfloat16)

        self.linears = {}
        for name, d_out, d_in in (("qkv", (hq + 2 * hkv) * dim, hidden), ("o", hidden, hq * dim),
                                  ("gate_up", 2 * ffn, hidden), ("down", hidden, ffn)):
            base = normal(d_out, d_in, std=d_in ** -0.5)
            packs = []
            for _ in range(variants):
                delta = normal(d_out, d_in, std=0.05 * d_in ** -0.5)
                tuned = (base.float() + delta).to(torch.bfloat16)
                packs.append(bd.bitdelta_compress(base, tuned, per_row=True))
            self.linears[name] = (base, packs, bd.variant_tables(
                [p for p, _ in packs], [a for _, a in packs], device))
        self.norms = {}
        for name in ("attn", "mlp", "next"):
            weights = [normal(hidden, std=0.1, mean=1.0) for _ in range(variants + 1)]
            self.norms[name] = (weights, bd.norm_table(weights))

    def linear(self, name, x, seg):
        base, _, (packed, alpha) = self.linears[name]
        return bd.bitdelta_linear_grouped(x, seg[0], seg[1], base, packed, alpha, self.variants,
                                          seg[2])

    def norm(self, name, y, h, seg):
        """(h + y, its norm)."""
        return bd.bitdelta_add_norm(y, h, self.norms[name][1], seg_offsets=seg[0],
                                    seg_variant=seg[1])

    def forward(self, h, seg, batch, rope, k_pages, v_pages):
        """h: the residual stream [tokens, hidden] (fp32).  seg: (seg_offsets,
        seg_variant, longest segment): a sequence's tokens are one segment.
        Returns the residual stream and the next block's normed input."""
        zero = torch.zeros(h.shape, dtype=torch.bfloat16, device=h.device)
        _, x = self.norm("attn", zero, h, seg)
        q = bd.bitdelta_kv_append(batch, self.linear("qkv", x, seg), rope, k_pages, v_pages)
        o, _ = bd.bitdelta_attention(batch, q, k_pages, v_pages)
        h, x = self.norm("mlp", self.linear("o", o.view(h.shape[0], -1), seg), h, seg)
        gate, up = self.linear("gate_up", x, seg).chunk(2, dim=1)
        f = (torch.nn.functional.silu(gate.float()) * up.float()).to(torch.bfloat16)
        return self.norm("next", self.linear("down", f, seg), h, seg)


def rope_table(positions, dim, base=10000.0, device="cuda"):
    i = torch.arange(dim // 2, device=device, dtype=torch.float64)
    angle = torch.arange(positions, device=device)[:, None] * base ** (-2.0 * i / dim)
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def int32(values, device="cuda"):
    return torch.tensor(values, dtype=torch.int32, device=device)


def main():
    hidden, ffn, hq, hkv, dim, page = 4096, 14336, 32, 8, 128, 16
    block = Block(hidden, ffn, hq, hkv, dim, variants=2)
    prompts, steps, variant = [512, 300, 77, 1], 8, [0, 1, 2, 1]
    width = -(-(max(prompts) + steps) // page)
    table = int32([[s * width + i for i in range(width)] for s in range(len(prompts))])
    k_pages = torch.empty((len(prompts) * width, hkv, page, dim), dtype=torch.bfloat16,
                          device="cuda")
    v_pages = torch.empty_like(k_pages)
    rope = rope_table(max(prompts) + steps, dim)
    lens = list(prompts)
    for step in range(steps + 1):
        q_len = prompts if step == 0 else [1] * len(prompts)
        if step:
            lens = [n + 1 for n in lens]
        offsets = [sum(q_len[:i]) for i in range(len(q_len) + 1)]
        seg = (int32(offsets), int32(variant), max(q_len))
        batch = bd.AttentionBatch(seg[0], int32(lens), table, offsets[-1], max(q_len), max(lens),
                                  hq, hkv, dim, page)
        h = torch.randn((offsets[-1], hidden), device="cuda")
        block.forward(h, seg, batch, rope, k_pages, v_pages)          # warm
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        h, x = block.forward(h, seg, batch, rope, k_pages, v_pages)
        b.record()
        b.synchronize()
        what = "prompts" if step == 0 else "decode"
        print(f"step {step} ({what}, {offsets[-1]} tokens, contexts {lens}): "
              f"{a.elapsed_time(b) * 1e3:.0f} us, |h| {h.abs().mean().item():.3f}")
    code = bd.bitdelta_check_error()
    if code:
        raise bd.BitDeltaError("decoder block", code)


if __name__ == "__main__":
    main()
