"""A prompt through this library, with a small random decoder: 8-bit weights with
a scale for each 128 x 128 block (qkv, output, MLP, head) multiplied by chunks of
any number of rows, attention of a chunk over the 4-bit cache and itself, the
chunk's keys and values into the cache, and the log-probability of each token of
the prompt.

    python examples/prompt_chunks.py           # on an MI355X

Prints the prompt's score in chunks of several sizes, and what the decoder found
most likely at its last token.
"""

import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from quantized_weight_skinny_amd import decode_api as qd  # noqa: E402
from quantized_weight_skinny_amd import prompt_api as qp  # noqa: E402


class Decoder:
    """Random weights of a decoder without positions, enough to take a prompt in."""

    def __init__(self, hidden=512, heads=8, kv_heads=2, dim=64, ff=1024, vocab=1000, layers=2, pages=64, page_size=16,
                 seed=0, device="cuda"):
        self.heads, self.kv_heads, self.dim, self.vocab, self.device = heads, kv_heads, dim, vocab, device
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)

        def weight(n, k):
            return qp.BlockWeight.quantize(torch.randn((n, k), device=device, generator=gen) * k ** -0.5)

        self.blocks = [{"qkv": weight((heads + 2 * kv_heads) * dim, hidden), "out": weight(hidden, heads * dim),
                        "up": weight(2 * ff, hidden), "down": weight(hidden, ff)} for _ in range(layers)]
        self.head = weight(vocab, hidden)
        self.embed = torch.randn((vocab, hidden), device=device, generator=gen).bfloat16()
        self.cache = qd.KV4Cache(pages, page_size, kv_heads, dim, layers, k_scale=5.0 / 2688, v_scale=5.0 / 2688,
                                 device=device)
        self.pool = qd.PagePool(pages, page_size, track_writes=True)

    @staticmethod
    def norm(x):
        x = x.float()
        return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).bfloat16()

    def chunk(self, seqs, tokens):
        """Logits [all rows, vocab] of a chunk of new tokens of each sequence (lists of any lengths)."""
        before = [self.pool.length(s) for s in seqs]
        slots = [slot for s, t in zip(seqs, tokens) for slot in self.pool.extend(s, len(t))]
        copies = self.pool.take_copies()
        if copies:
            src, dst = (torch.tensor(p, dtype=torch.int32, device=self.device) for p in zip(*copies))
            qd.kv4_copy_pages(self.cache, src, dst)
        tables = [self.pool.table(s) for s in seqs]
        wide = max(len(t) for t in tables)
        as_ints = lambda x: torch.tensor(x, dtype=torch.int32, device=self.device)  # noqa: E731
        table, kv_len = as_ints([t + [-1] * (wide - len(t)) for t in tables]), as_ints(before)
        start = [0]
        for t in tokens:
            start.append(start[-1] + len(t))
        q_start, longest = as_ints(start), max(len(t) for t in tokens)
        slots = torch.tensor(slots, dtype=torch.int64, device=self.device)
        x = self.embed[torch.tensor([y for t in tokens for y in t], device=self.device)]
        rows, q_size, kv_size = start[-1], self.heads * self.dim, self.kv_heads * self.dim
        for i, w in enumerate(self.blocks):
            qkv = qp.fp8_block_linear(self.norm(x), w["qkv"])
            q = qkv[:, :q_size].view(rows, self.heads, self.dim)
            k = qkv[:, q_size:q_size + kv_size].view(rows, self.kv_heads, self.dim)
            v = qkv[:, q_size + kv_size:].view(rows, self.kv_heads, self.dim)
            a, _ = qp.kv4_chunk_attention(q, k, v, self.cache, table, kv_len, q_start=q_start, max_q_len=longest,
                                          max_kv_len=max(before), layer=i)
            qd.kv4_append(self.cache, k, v, slots, layer=i)
            x = x + qp.fp8_block_linear(a.view(rows, q_size), w["out"])
            gate, up = qp.fp8_block_linear(self.norm(x), w["up"]).float().chunk(2, 1)
            x = x + qp.fp8_block_linear((torch.nn.functional.silu(gate) * up).bfloat16(), w["down"])
        for s in seqs:
            self.pool.written(s)
        return qp.fp8_block_linear(self.norm(x), self.head, dtype=torch.float32)


def score(model, seq, prompt, size):
    """Log-probabilities of prompt[1:], taken in `size` tokens at a time, and the alternatives at the last of them."""
    logprobs = []
    for at in range(0, len(prompt) - 1, size):
        part = prompt[at:min(at + size, len(prompt) - 1)]
        logits = model.chunk([seq], [part])
        following = torch.tensor(prompt[at + 1:at + 1 + len(part)], dtype=torch.int32, device=model.device)
        logp, _, _, best, best_logp = qp.token_logprobs(logits, following, top=5)
        logprobs.append(logp)
    return torch.cat(logprobs), best[-1], best_logp[-1]


def main():
    model = Decoder()
    gen = torch.Generator().manual_seed(1)
    prompt = torch.randint(0, model.vocab, (300,), generator=gen).tolist()
    for size in (299, 128, 37):
        seq = model.pool.new()
        logprobs, best, best_logp = score(model, seq, prompt, size)
        print(f"chunks of {size}: mean log-probability {float(logprobs.mean()):.4f}; most likely at the last token:",
              [f"{t} ({p:.2f})" for t, p in zip(best.tolist(), best_logp.tolist())])
        model.pool.free(seq)
    assert model.pool.free_pages == model.pool.pages


if __name__ == "__main__":
    main()
