"""GPU parity of what a rejected draft leaves over where rows cancel."""

import numpy as np
import pytest

from gpu_helpers import to_host
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
