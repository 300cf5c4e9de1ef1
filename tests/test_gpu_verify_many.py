"""GPU parity of verification where rows have more than 64 chunks of 4096
tokens, and where the accept tests have a launch of their own (more than 512
sequences x chunks). Tolerances are those of test_gpu_verify.py."""

import numpy as np
import pytest
import torch

from gpu_helpers import to_host
from test_gpu_verify import block, check, run

pytestmark = pytest.mark.gpu


def late(x, vocab):
    """Most of p's mass in tokens beyond 64 chunks, among them the drafts, and u_sample spread over it."""
    for name in ("target", "draft"):
        if x[name] is not None:
            x[name][..., 262144 + 4000:] += 4.0
    n = x["u_sample"].size
    x["u_sample"] = ((np.arange(n) + 0.5) / n).astype(np.float32)
    return x


@pytest.mark.parametrize("dtype", ["fp16", "fp32"])
@pytest.mark.parametrize("draft", [None, "logits"])
def test_many_chunks(dtype, draft):
    vocab = 270001
    x = late(block(31, 6, 2, vocab, dtype, draft), vocab)
    x["u_accept"][::2] = 0.9999                    # some are refused at once
    x["draft_tokens"][5, 1] = -1
    got = run(x)
    check(x, got)
    assert (to_host(got[0])[:, 0] >= 262144).any() and (to_host(got[0])[:, 0] < 262144).any()


@pytest.mark.parametrize("draft", [None, "logits"])
def test_many_chunks_of_probabilities(draft):
    vocab = 270001
    x = late(block(32, 5, 2, vocab, "fp32", draft), vocab)
    for name in ("target", "draft"):
        if x[name] is not None:
            x[name] = torch.softmax(x[name].double(), 2).float()
    x["u_accept"][::2] = 0.9999
    check(x, run(x, True), True)


def test_many_chunks_greedy_and_masked():
    """The largest logit in the first and in the last chunk at once (the first wins), and rows with nothing else."""
    vocab = 300001
    x = block(33, 3, 1, vocab, "bf16", None)
    x["temperature"] = np.array([0.0, 0.5, 1.0], np.float32)
    x["target"][0, :, [7, vocab - 1]] = 60.0
    x["draft_tokens"][0] = 7
    x["target"][1:, :, :299000] = -float("inf")
    x["target"][2, 0] = -float("inf")
    x["target"][2, 0, vocab - 1] = 1.0
    x["draft_tokens"][2] = vocab - 1
    x["u_accept"][2] = 0.5
    got = run(x)
    check(x, got)
    assert to_host(got[0])[0].tolist() == [7, 7] and to_host(got[0])[2, 0] == vocab - 1


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("draft", [None, "logits"])
def test_accept_tests_of_many_sequences(dtype, draft):
    """200 sequences x 3 chunks: greedy and sampled ones, of every number of drafts, drafts out of range and refused
    drafts of equal rows among them."""
    batch, drafts, vocab = 200, 5, 9001
    x = block(34, batch, drafts, vocab, dtype, draft)
    x["temperature"] = np.resize(np.array([1, 0, 0.6, 1.7, -1], np.float32), batch)
    x["num_draft"] = np.resize(np.array([5, 0, 3, 1, 9, 2, 4], np.int32), batch)
    for b in range(1, batch, 5):                   # greedy sequences accept some drafts
        x["draft_tokens"][b, :b % 6] = x["target"][b, :b % 6].float().argmax(1).numpy()
    x["draft_tokens"][2::10, 1] = [(-1, vocab, 2 ** 31 - 1, -2 ** 31)[i % 4] for i in range(20)]
    if draft:
        x["target"][3::20, 0] = x["draft"][3::20, 0]
        x["draft_tokens"][3::20, 0] = -1
    got = run(x)
    check(x, got)
    assert len(set(to_host(got[1]).tolist())) == drafts + 1
