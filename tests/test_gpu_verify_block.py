"""The operators together, through the example decoder: speculative decoding
gives the tokens of one-at-a-time decoding, whatever is drafted; forks and
compaction leave every sequence as it was."""

import os
import sys

import pytest
import torch

from gpu_helpers import DEV, say
from quantized_weight_skinny_amd import decode_api as qd

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import verify_block as vb  # noqa: E402

pytestmark = pytest.mark.gpu
PROMPT = [5, 17, 5, 40, 5, 17, 99, 5, 17, 5, 40]


def _start(model):
    seq = model.pool.new()
    model.step(seq, PROMPT[:-1])
    return seq


def test_greedy_speculation_gives_the_plain_tokens():
    say("greedy speculation")
    model = vb.Decoder()
    base = _start(model)
    plain, took = vb.generate(model, model.pool.fork(base), PROMPT, 40, propose=lambda h, n: [])
    assert took == [1] * 40
    # drafts that are right, then wrong from some place on
    def propose(history, n):
        at = len(history)
        guess = plain[at:at + n]
        if at % 3 == 0 and len(guess) > 2:
            guess[2] = (guess[2] + 1) % model.vocab
        return guess
    fast, took = vb.generate(model, model.pool.fork(base), PROMPT, 40, propose=propose)
    assert fast[:len(PROMPT) + 40] == plain[:len(PROMPT) + 40]
    assert max(took) == 8 and 3 in took
    looked, _ = vb.generate(model, model.pool.fork(base), PROMPT, 40)
    assert looked[:len(PROMPT) + 40] == plain[:len(PROMPT) + 40]


def test_forks_and_compaction_keep_the_tokens():
    say("forks and compaction")
    model = vb.Decoder(seed=1)
    base = _start(model)
    want, _ = vb.generate(model, model.pool.fork(base), PROMPT, 30, temperature=0.9, seed=5)
    # other sequences come and go, pages move
    others = [model.pool.fork(base) for _ in range(3)]
    for i, o in enumerate(others):
        vb.generate(model, o, PROMPT, 25, temperature=1.5, seed=10 + i)
    model.pool.free(others[1])
    used = model.pool.compact()
    src, dst = (torch.tensor(p, dtype=torch.int32, device=DEV) for p in zip(*model.pool.take_copies()))
    before = model.cache.data.clone()
    qd.kv4_copy_pages(model.cache, src, dst)
    assert torch.equal(model.cache.data[:, dst.long()], before[:, src.long()])
    assert used == model.pool.pages - model.pool.free_pages
    got, _ = vb.generate(model, model.pool.fork(base), PROMPT, 30, temperature=0.9, seed=5)
    assert got == want


def test_example_runs():
    say("example")
    vb.main()
