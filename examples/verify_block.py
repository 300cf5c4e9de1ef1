"""Speculative decoding on this library from end to end, with a small random
decoder: NVFP4 weights (qkv, output, MLP, head) through the skinny GEMM, keys
and values in the 4-bit paged cache, attention over it, and the verification
of drafted tokens. The drafts are looked up in the tokens so far.

    python examples/verify_block.py            # on an MI355X

Prints the tokens a step took, then forks the sequence: two continuations share
the prompt's pages, each writes its own.
"""

import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from quantized_weight_skinny_amd import decode_api as qd  # noqa: E402
from quantized_weight_skinny_amd import torch_api as qt  # noqa: E402


class Decoder:
    """Random weights of a decoder without positions, enough to run a step."""

    def __init__(self, hidden=512, heads=8, kv_heads=2, dim=64, ff=1024, vocab=1000, layers=2, pages=64, page_size=16,
                 seed=0, device="cuda"):
        self.heads, self.kv_heads, self.dim, self.vocab, self.layers, self.device = heads, kv_heads, dim, vocab, layers, device
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)

        def weight(n, k):
            w = torch.randn((n, k), device=device, generator=gen) * k ** -0.5
            return qt.pack_nvfp4(*qt.quantize_nvfp4(w), n, k)

        self.blocks = [{"qkv": weight((heads + 2 * kv_heads) * dim, hidden), "out": weight(hidden, heads * dim),
                        "up": weight(2 * ff, hidden), "down": weight(hidden, ff)} for _ in range(layers)]
        self.head = weight(vocab, hidden)
        self.embed = torch.randn((vocab, hidden), device=device, generator=gen).half()
        self.cache = qd.KV4Cache(pages, page_size, kv_heads, dim, layers, k_scale=5.0 / 2688, v_scale=5.0 / 2688,
                                 device=device)
        self.pool = qd.PagePool(pages, page_size, track_writes=True)

    @staticmethod
    def norm(x):
        x = x.float()
        return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).half()

    def step(self, seq, tokens):
        """Logits [len(tokens), vocab] of up to 16 tokens that follow the sequence's, whose keys and values enter
        the cache."""
        slots = torch.tensor(self.pool.extend(seq, len(tokens)), dtype=torch.int64, device=self.device)
        copies = self.pool.take_copies()
        if copies:
            src, dst = (torch.tensor(p, dtype=torch.int32, device=self.device) for p in zip(*copies))
            qd.kv4_copy_pages(self.cache, src, dst)
        length = self.pool.length(seq)
        table = torch.tensor([self.pool.table(seq)], dtype=torch.int32, device=self.device)
        kv_len = torch.tensor([length], dtype=torch.int32, device=self.device)
        x = self.embed[torch.tensor(tokens, device=self.device)]
        rows, q_size, kv_size = len(tokens), self.heads * self.dim, self.kv_heads * self.dim
        for i, w in enumerate(self.blocks):
            qkv = qt.gemm(self.norm(x), w["qkv"])
            q = qkv[:, :q_size].view(rows, self.heads, self.dim)
            k = qkv[:, q_size:q_size + kv_size].view(rows, self.kv_heads, self.dim)
            v = qkv[:, q_size + kv_size:].view(rows, self.kv_heads, self.dim)
            qd.kv4_append(self.cache, k, v, slots, layer=i)
            a, _ = qd.kv4_attention(q, self.cache, table, kv_len, layer=i)
            x = x + qt.gemm(a.view(rows, q_size), w["out"])
            x = x + qt.mlp(self.norm(x), w["up"], w["down"])[1]
        self.pool.written(seq)
        return qt.gemm(self.norm(x), self.head)


def lookup(history, count):
    """What followed the last occurrence of the final token earlier on: up to `count` drafts."""
    for at in range(len(history) - 2, -1, -1):
        if history[at] == history[-1]:
            return history[at + 1:at + 1 + count]
    return []


def generate(model, seq, history, new, drafts=7, temperature=0.0, seed=0, propose=lookup):
    """Extends `history` (whose last token is not yet in the cache) by at least `new` tokens; returns it and the
    tokens that each step took."""
    gen = torch.Generator(device=model.device)
    gen.manual_seed(seed)
    history, took = list(history), []
    temp = torch.tensor([temperature], device=model.device)
    while sum(took) < new:
        guess = propose(history, drafts)
        n = len(guess)
        logits = model.step(seq, [history[-1]] + guess)
        tokens, accepted, _ = qd.verify_drafts(
            logits.view(1, n + 1, model.vocab), torch.tensor([guess], dtype=torch.int32, device=model.device).view(1, n),
            torch.rand((1, n), device=model.device, generator=gen), torch.rand(1, device=model.device, generator=gen),
            temperature=temp)
        kept = accepted.item() + 1
        # the rejected drafts' keys and values leave; the picked token's are yet to come
        model.pool.truncate(seq, model.pool.length(seq) - (n + 1 - kept))
        history += tokens[0, :kept].tolist()
        took.append(kept)
    return history, took


def main():
    model = Decoder()
    prompt = [5, 17, 5, 40, 5, 17, 99, 5, 17, 5, 40]
    seq = model.pool.new()
    for at in range(0, len(prompt) - 1, 16):
        model.step(seq, prompt[at:min(at + 16, len(prompt) - 1)])
    other = model.pool.fork(seq)
    history, took = generate(model, seq, prompt, 48)
    print("greedy, tokens a step:", took)
    print("  ", history[len(prompt):])
    history, took = generate(model, other, prompt, 48, temperature=0.8, seed=3)
    print("temperature 0.8 from the same prompt's pages, tokens a step:", took)
    print("  ", history[len(prompt):])
    model.pool.free(seq)
    model.pool.free(other)
    assert model.pool.free_pages == model.pool.pages


if __name__ == "__main__":
    main()
