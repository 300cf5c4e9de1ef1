"""Sums of token log-probabilities over rows of one slice, on the GPU, against
the definition in 64 bits.

Tolerance. A lane adds at most 128 elements in 32 bits, each addition off by 2^-24
of the sum so far, before they go to 64 bits; the weights are good to 2^-22 and 2^-23 of
their exponents. So log s is off by 2^-22 + 2^-23 E|x - m| / (t ln 2) + 128 * 2^-24, E over p, and the
entropy by that twice and that much of E|x - m| / t."""

import math

import pytest
import torch

from gpu_helpers import DEV, say
from quantized_weight_skinny_amd import prompt_api as qp

pytestmark = pytest.mark.gpu


def _check(x, tokens, some, got, top):
    logp, entropy, _, best, best_logp = got
    for r in some:
        y = x[r].double()
        m = y.max()
        p = torch.exp(y - m)
        z = p.sum()
        spread = float((p * (m - y)).sum() / z)
        lp = y - m - torch.log(z)
        h = float(torch.log(z) + spread)
        off = 2.0 ** -22 + 2.0 ** -23 * spread / math.log(2) + 128 * 2.0 ** -24
        want = float(lp[int(tokens[r])])
        assert abs(float(logp[r]) - want) <= off + 2.0 ** -23 * abs(want), (r, float(logp[r]), want)
        assert abs(float(entropy[r]) - h) <= (2 + spread) * off + 2.0 ** -23 * h, (r, float(entropy[r]), h)
        for j in range(top):
            want = float(lp[int(best[r, j])])
            assert abs(float(best_logp[r, j]) - want) <= off + 2.0 ** -23 * abs(want), (r, j)


@pytest.mark.parametrize("top", [0, 3])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_small_terms_of_a_long_row_count(dtype, top):
    """The largest vocabulary; a lane's first elements are so much larger that each later one is below
    half a step of their sum. 2048 rows of one memory, so that a row is one workgroup's."""
    vocab, rows = 1 << 24, 2048
    say("token_logprobs", rows, vocab, dtype, top)
    row = torch.full((vocab,), -17.375, dtype=dtype, device=DEV)   # e^-17.375 is 0.95 * 2^-25
    row[:4096] = 0
    x = row.expand(rows, vocab)
    tokens = torch.arange(rows, dtype=torch.int32, device=DEV) * 8191
    got = qp.token_logprobs(x, tokens, top=top)
    _check(x, tokens, (0, 1, 1000, rows - 1), got, top)
    assert torch.equal(got[2], tokens)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
def test_rows_of_one_slice(dtype):
    rows, vocab = 2100, 151936
    gen = torch.Generator(device=DEV).manual_seed(3)
    x = torch.empty((rows, vocab), dtype=dtype, device=DEV)
    for at in range(0, rows, 300):
        x[at:at + 300] = (torch.randn((300, vocab), device=DEV, generator=gen) * 2.5).to(dtype)
    tokens = torch.randint(0, vocab, (rows,), device=DEV, generator=gen).to(torch.int32)
    say("token_logprobs", rows, vocab, dtype, 5)
    some = list(range(0, rows, 131))
    _check(x, tokens, some, qp.token_logprobs(x, tokens, top=5), 5)
    # falling and rising rows: references that move late, or in every step
    slope = torch.linspace(-30, 30, vocab, device=DEV)
    x[0::2], x[1::2] = slope.to(dtype), slope.flip(0).to(dtype)
    _check(x, tokens, some, qp.token_logprobs(x, tokens, top=5), 5)
