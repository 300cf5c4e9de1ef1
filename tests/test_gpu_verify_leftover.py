"""GPU parity of what a rejected draft leaves over: rows that cancel exactly,
and rows that cancel but for a few tokens, where the passes that sum max(p - q,
0) and the one that finds the token in it must hold the same numbers."""

import numpy as np
import pytest
import torch

from gpu_helpers import say, to_host
from test_gpu_verify import block, check, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("vocab", [2, 8, 1000, 9001])
@pytest.mark.parametrize("temperature", [None, 0.37])
def test_equal_rows_and_a_refused_draft_leave_the_target(dtype, vocab, temperature):
    """The target's row equals the draft's bit for bit and the draft is refused,
    as a token outside the vocabulary or as one that both rows mask: nothing is
    left over, so the token comes from p, whatever u_sample is."""
    batch = 24
    x = block(vocab, batch, 2, vocab, dtype, "logits")
    x["target"][:, :2] = x["draft"]
    x["draft_tokens"][:, 0] = [(-1, vocab, 2 ** 31 - 1, b % vocab)[b % 4] for b in range(batch)]
    for b in range(3, batch, 4):
        x["target"][b, 0, b % vocab] = x["draft"][b, 0, b % vocab] = -float("inf")
    x["u_accept"][:] = 0.0
    x["u_sample"] = ((np.arange(batch) + 0.5) / batch).astype(np.float32)
    if temperature:
        x["temperature"] = np.full(batch, temperature, np.float32)
    got = run(x)
    assert (to_host(got[1]) == 0).all()
    check(x, got)


def test_nearly_equal_rows_of_many_chunks_give_a_token_that_is_left_over():
    """Rows that differ by exchanged logits of far tokens: the totals of p and q
    agree to the last bits or all, and what is left over besides is at most
    their rounding. Above 64 chunks of 4096 the totals are longer than a
    wavefront. u_sample = 0 asks for the first token with anything left; the last
    token of every chunk is masked, so that none of those can be given."""
    batch, vocab = 64, 300001
    rng = np.random.default_rng(5)
    p = (rng.standard_normal((batch, 1, vocab)) * 2).astype(np.float32)
    p[:, :, 4095::4096] = -np.inf
    p[:, :, -1] = -np.inf
    q = p.copy()
    for b in range(batch):
        for i, j in zip(41000 + rng.permutation(3000)[:6], 290000 + rng.permutation(4000)[:6]):
            q[b, 0, [i, j]] = q[b, 0, [j, i]]
    target = torch.from_numpy(np.concatenate([p, p], 1))
    x = {"target": target, "draft": torch.from_numpy(q), "draft_tokens": np.full((batch, 1), -1, np.int32),
         "u_accept": np.zeros((batch, 1), np.float32), "u_sample": np.zeros(batch, np.float32), "num_draft": None,
         "temperature": None}
    tokens = to_host(run(x)[0])[:, 0]
    say("tokens", tokens.tolist())
    assert ((tokens >= 0) & (tokens < vocab)).all()
    assert np.isfinite(p[np.arange(batch), 0, tokens]).all()
