"""The prompt operators together, through the example decoder: sequences of a
batch are as alone; a verify step reads what chunks have cached; a captured step
replays."""

import os
import sys

import pytest
import torch

from gpu_helpers import DEV, say
from quantized_weight_skinny_amd import decode_api as qd
from quantized_weight_skinny_amd import prompt_api as qp

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import prompt_chunks as pc  # noqa: E402

pytestmark = pytest.mark.gpu


def _prompt(n, seed=0):
    return torch.randint(0, 1000, (n,), generator=torch.Generator().manual_seed(seed)).tolist()


def test_batched_sequences_are_as_alone():
    """Products of more than 64 rows whose k is not split, and attention of short runs, give a row the same bits
    whatever stands beside it."""
    say("batched chunks")
    prompts = [[t % 300 for t in _prompt(n, n)] for n in (150, 136, 200)]
    alone = []
    for p in prompts:
        model = pc.Decoder(vocab=300)
        seq = model.pool.new()
        alone.append((model.chunk([seq], [p[:70]]), model.chunk([seq], [p[70:]])))
    model = pc.Decoder(vocab=300)
    seqs = [model.pool.new() for _ in prompts]
    first = model.chunk(seqs, [p[:70] for p in prompts])
    second = model.chunk(seqs, [p[70:] for p in prompts])
    assert torch.equal(first, torch.cat([x for x, _ in alone]))
    assert torch.equal(second, torch.cat([x for _, x in alone]))


def test_a_verify_step_reads_what_chunks_have_cached():
    """Attention of a verify block over tokens that chunks appended, and a chunk of the same rows: both see the same
    cached tokens; they differ by the block's own keys and values in 4 bits."""
    model = pc.Decoder()
    seq = model.pool.new()
    model.chunk([seq], [_prompt(100)])
    gen = torch.Generator(device=DEV).manual_seed(3)
    q, k, v = (torch.randn((5, n, model.dim), device=DEV, generator=gen).bfloat16()
               for n in (model.heads, model.kv_heads, model.kv_heads))
    slots = torch.tensor(model.pool.extend(seq, 5), dtype=torch.int64, device=DEV)
    qd.kv4_append(model.cache, k, v, slots)
    as4k, as4v = qd.kv4_read(model.cache, slots, dtype=torch.bfloat16)
    table = torch.tensor([model.pool.table(seq)], dtype=torch.int32, device=DEV)
    verify, lse = qd.kv4_attention(q, model.cache, table, torch.tensor([105], dtype=torch.int32, device=DEV))
    # the chunk's own tokens given as the cache holds them (bf16 holds an E2M1 x E4M3 x tensor scale to 2^-8)
    chunk, lse2 = qp.kv4_chunk_attention(q, as4k, as4v, model.cache, table,
                                         torch.tensor([100], dtype=torch.int32, device=DEV))
    assert (verify.float() - chunk.float()).abs().max() <= 2.0 ** -6 * as4v.float().abs().max()
    assert (lse - lse2).abs().max() <= 2.0 ** -8 * (q.float().abs().sum(-1).max() * as4k.float().abs().max()) * model.dim ** -0.5


def test_a_captured_step_replays():
    """Products, attention, append and log-probabilities of a chunk in one graph; eager work between the replays."""
    say("captured chunk")
    heads, kvh, dim, page, hidden, vocab, rows = 8, 2, 64, 16, 512, 3001, 90
    gen = torch.Generator(device=DEV).manual_seed(0)
    w = [qp.BlockWeight.quantize(torch.randn(s, device=DEV, generator=gen) * 0.04)
         for s in (((heads + 2 * kvh) * dim, hidden), (hidden, heads * dim), (vocab, hidden))]
    cache = qd.KV4Cache(40, page, kvh, dim)
    table = torch.randperm(40, device=DEV, generator=gen).to(torch.int32).view(2, 20)
    x = torch.empty((rows, hidden), dtype=torch.bfloat16, device=DEV)
    tokens = torch.empty((rows,), dtype=torch.int32, device=DEV)
    kv_len, q_start = (torch.zeros(n, dtype=torch.int32, device=DEV) for n in (2, 3))
    slots = torch.zeros((rows,), dtype=torch.int64, device=DEV)
    work = [qp.fp8_block_workspace(rows, y.n, y.k) for y in w]
    aws = qp.kv4_chunk_workspace(cache, rows, heads, 2, rows, 320)
    lws = qp.token_logprobs_workspace(rows, vocab, 3)

    def step(ws=(None,) * 3, a_ws=None, l_ws=None):
        qkv = qp.fp8_block_linear(x, w[0], workspace=ws[0])
        q = qkv[:, :heads * dim].view(rows, heads, dim)
        k = qkv[:, heads * dim:(heads + kvh) * dim].view(rows, kvh, dim)
        v = qkv[:, (heads + kvh) * dim:].view(rows, kvh, dim)
        a, lse = qp.kv4_chunk_attention(q, k, v, cache, table, kv_len, q_start=q_start, max_q_len=rows, workspace=a_ws)
        qd.kv4_append(cache, k, v, slots)
        h = qp.fp8_block_linear(a.view(rows, -1), w[1], workspace=ws[1])
        return a, lse, *qp.token_logprobs(qp.fp8_block_linear(h, w[2], workspace=ws[2]), tokens, top=3, workspace=l_ws)

    def set_inputs(seed, lengths, first):
        g = torch.Generator(device=DEV).manual_seed(seed)
        x.copy_(torch.randn(x.shape, device=DEV, generator=g))
        tokens.copy_(torch.randint(0, vocab, (rows,), device=DEV, generator=g))
        kv_len.copy_(torch.tensor(lengths, dtype=torch.int32))
        q_start.copy_(torch.tensor([0, first, rows], dtype=torch.int32))
        at = [lengths[0] + i for i in range(first)] + [lengths[1] + i for i in range(rows - first)]
        b = [0] * first + [1] * (rows - first)
        slots.copy_(torch.tensor([int(table[c, t // page]) * page + t % page for c, t in zip(b, at)]))

    set_inputs(0, (0, 0), 40)
    step(work, aws, lws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(work, aws, lws)
    for seed, lengths, first in ((1, (0, 0), 40), (2, (40, 50), 1), (3, (41, 139), 90), (4, (200, 10), 0)):
        set_inputs(seed, lengths, first)
        graph.replay()
        torch.cuda.synchronize()
        got = [y.clone() for y in outs]
        for a, b in zip(got, step()):
            assert torch.equal(a, b)


def test_example_runs():
    say("example")
    pc.main()
