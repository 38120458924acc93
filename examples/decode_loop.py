"""Generation with a cache held to a budget, for a batch of the base model and its
variants:

    prompt step, then per token
      block   as in decoder_block.py, and behind the attention
              what each cached key was looked at     bitdelta_kv_weigh
      head    logits                                 bitdelta_linear_grouped
      token   temperature, top-k, top-p, min-p       bitdelta_sample
    and whenever a sequence reaches the budget and its slack
      cut     the heaviest and the last keys stay    bitdelta_kv_evict, per layer
              the new lengths                        bitdelta_kv_evict_lengths

`python examples/decode_loop.py` generates a few tokens on a GPU and prints the
lengths and what the steps took.
"""
import os
import sys

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import bit_weight_delta_gb300 as bd
from decoder_block import Block, int32, rope_table


class LayerCache:
    """A layer's keys and values, and what the eviction goes by, beside them."""

    def __init__(self, n_pages, hkv, page, dim):
        self.k = torch.empty((n_pages, hkv, page, dim), dtype=torch.bfloat16, device="cuda")
        self.v = torch.empty_like(self.k)
        self.weights = torch.empty((n_pages, hkv, page), device="cuda")
        self.positions = torch.empty((n_pages, hkv, page), dtype=torch.int32, device="cuda")

    def attend(self, batch, qkv, rope, pos_offset, window=0):
        """Appends qkv's keys and values, and returns the attention of its queries."""
        q = bd.bitdelta_kv_append(batch, qkv, rope, self.k, self.v, pos_offset=pos_offset)
        o, lse = bd.bitdelta_attention(batch, q, self.k, self.v)
        bd.bitdelta_kv_weigh(batch, q, lse, self.k, self.weights, self.positions, window=window,
                             pos_offset=pos_offset)
        return o

    def cut(self, batch, keep, recent, sink, pos_offset):
        bd.bitdelta_kv_evict(batch, keep, self.k, self.v, self.weights, self.positions,
                             recent=recent, sink=sink, pos_offset=pos_offset)


class Sequences:
    """The lengths and pages of a batch of sequences, on the device and here."""

    def __init__(self, n, budget, slack, hq, hkv, dim, page):
        self.n, self.budget, self.slack = n, budget, slack
        self.heads = (hq, hkv, dim, page)
        self.lens = [0] * n
        self.kv_len = int32([0] * n)
        self.pos_offset = int32([0] * n)
        self.page_table = None

    def room(self, longest):
        """Pages for sequences of up to `longest` keys."""
        page = self.heads[3]
        width = -(-max(longest, self.budget + self.slack) // page)
        self.page_table = int32([[s * width + i for i in range(width)] for s in range(self.n)])
        return self.n * width

    def batch(self, q_len):
        """The next step's batch, of q_len new tokens per sequence."""
        self.lens = [a + b for a, b in zip(self.lens, q_len)]
        self.kv_len.copy_(int32(self.lens))
        offsets = [sum(q_len[:i]) for i in range(self.n + 1)]
        return bd.AttentionBatch(int32(offsets), self.kv_len, self.page_table, offsets[-1],
                                 max(q_len), max(self.lens), *self.heads)

    def cut(self, batch, layers, recent, sink=4):
        """Down to the budget, where a sequence has used up its slack.  True if one had."""
        if max(self.lens) < self.budget + self.slack:
            return False
        keep = int32([self.budget] * self.n)
        for layer in layers:
            layer.cut(batch, keep, recent, sink, self.pos_offset)
        bd.bitdelta_kv_evict_lengths(batch, keep, self.kv_len, self.pos_offset)
        self.lens = [min(n, self.budget) for n in self.lens]
        return True


class Layer(Block):
    def forward(self, h, seg, batch, rope, cache, pos_offset, window):
        zero = torch.zeros(h.shape, dtype=torch.bfloat16, device=h.device)
        _, x = self.norm("attn", zero, h, seg)
        o = cache.attend(batch, self.linear("qkv", x, seg), rope, pos_offset, window)
        h, x = self.norm("mlp", self.linear("o", o.view(h.shape[0], -1), seg), h, seg)
        gate, up = self.linear("gate_up", x, seg).chunk(2, dim=1)
        f = (torch.nn.functional.silu(gate.float()) * up.float()).to(torch.bfloat16)
        return self.norm("next", self.linear("down", f, seg), h, seg)


def bd_head(vocab, hidden, g):
    """The head's base weight and two variants' deltas, as bitdelta_linear_grouped takes them."""
    rn = lambda std: (torch.randn((vocab, hidden), generator=g, device="cuda") * std).to(torch.bfloat16)
    base = rn(3.0 * hidden ** -0.5)
    packs = [bd.bitdelta_compress(base, base + rn(0.1 * hidden ** -0.5), per_row=True)
             for _ in range(2)]
    return (base, *bd.variant_tables([p for p, _ in packs], [a for _, a in packs], "cuda"), packs)


def main():
    hidden, ffn, hq, hkv, dim, page, vocab = 2048, 5632, 16, 4, 128, 16, 32000
    variant, prompts, steps = [0, 1, 2, 1], [512, 300, 77, 600], 48
    budget, slack, n = 256, 32, 4
    layers = [Layer(hidden, ffn, hq, hkv, dim, variants=2, seed=i) for i in range(2)]
    g = torch.Generator(device="cuda").manual_seed(9)
    embed = torch.randn((vocab, hidden), generator=g, device="cuda").to(torch.bfloat16)
    head = bd_head(vocab, hidden, g)
    seqs = Sequences(n, budget, slack, hq, hkv, dim, page)
    pages = seqs.room(max(prompts) + 1)
    caches = [LayerCache(pages, hkv, page, dim) for _ in layers]
    rope = rope_table(max(prompts) + steps + 1, dim)
    temperature = torch.tensor([0.7, 0.0, 1.0, 0.9], device="cuda")
    top_k, top_p = int32([50, 0, 0, 200]), torch.tensor([0.95, 1.0, 0.9, 1.0], device="cuda")
    one_row = int32(range(n + 1))          # a sequence's last token is a segment
    tokens = torch.randint(0, vocab, (sum(prompts),), generator=g, device="cuda")
    for step in range(steps + 1):
        q_len = prompts if step == 0 else [1] * n
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        batch = seqs.batch(q_len)
        offsets = [sum(q_len[:i]) for i in range(n + 1)]
        seg = (int32(offsets), int32(variant), max(q_len))
        h = embed[tokens.long()].float()
        for layer, cache in zip(layers, caches):
            # a prompt is weighed by its last tokens
            h, x = layer.forward(h, seg, batch, rope, cache, seqs.pos_offset, window=64)
        last = x[[o - 1 for o in offsets[1:]]].contiguous()
        logits = bd.bitdelta_linear_grouped(last, one_row, int32(variant), *head[:3], 2, 1)
        tokens, _ = bd.bitdelta_sample(logits, torch.rand(n, generator=g, device="cuda"),
                                       temperature=temperature, top_k=top_k, top_p=top_p)
        before = list(seqs.lens)
        cut = seqs.cut(batch, caches, recent=64)
        b.record()
        b.synchronize()
        if step < 3 or cut:
            print(f"step {step}: {a.elapsed_time(b) * 1e3:.0f} us, tokens {tokens.tolist()}, "
                  f"keys {before}" + (f" -> {seqs.lens}" if cut else ""))
    code = bd.bitdelta_check_error()
    if code:
        raise bd.BitDeltaError("decode loop", code)


if __name__ == "__main__":
    main()
