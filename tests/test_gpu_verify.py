"""GPU parity of verify_drafts against the float64 oracle. Tokens and counts
are equal; the seeds are such that no decision of the oracle lies within 1e-9
(accept tests: 1e-5, their sums of exponentials are 32-bit precise) of its
border. Log-probabilities: the sum of exponentials is good to 2^-21 (fp32
exponentials of exponents up to 2^5, sums of 16), the result rounded once."""

import numpy as np
import pytest
import torch

import oracle.kv4 as ok
from gpu_helpers import DEV, say, to_host
from quantized_weight_skinny_amd import decode_api as qd

pytestmark = pytest.mark.gpu

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def block(seed, batch, drafts, vocab, dtype, draft="logits", spread=2.0, sharp=8.0):
    """Inputs on the CPU: the target near the draft, drafts drawn from the draft."""
    rng = np.random.default_rng(seed)
    q = rng.standard_normal((batch, drafts, vocab)) * spread
    if vocab > 4:
        at = rng.integers(0, vocab, (batch, drafts, 3))
        np.put_along_axis(q, at, np.take_along_axis(q, at, 2) + sharp * rng.random((batch, drafts, 3)), 2)
    p = np.concatenate([q + 0.6 * rng.standard_normal(q.shape), rng.standard_normal((batch, 1, vocab)) * 3], 1)
    noise = rng.gumbel(size=q.shape)
    tokens = (q.argmax(2) if draft is None else (q + noise).argmax(2)).astype(np.int32)
    as_type = lambda x: torch.from_numpy(x.astype(np.float32)).to(TYPES[dtype])  # noqa: E731
    return {"target": as_type(p), "draft": None if draft is None else as_type(q), "draft_tokens": tokens,
            "u_accept": rng.random((batch, drafts)).astype(np.float32),
            "u_sample": rng.random(batch).astype(np.float32), "num_draft": None, "temperature": None}


def run(x, probabilities=False, **kw):
    dev = {k: (v.to(DEV) if isinstance(v, torch.Tensor) else None if v is None else torch.from_numpy(v).to(DEV))
           for k, v in x.items()}
    say("verify", tuple(x["target"].shape), x["target"].dtype, "draft" if x["draft"] is not None else "none", kw.keys())
    return qd.verify_drafts(dev["target"], dev["draft_tokens"], dev["u_accept"], dev["u_sample"], draft=dev["draft"],
                            num_draft=dev["num_draft"], temperature=dev["temperature"], probabilities=probabilities,
                            **kw)


def check(x, got, probabilities=False):
    as64 = lambda t: None if t is None else t.double().numpy()  # noqa: E731
    tokens, accepted, logprobs, margin = ok.verify(
        as64(x["target"]), as64(x["draft"]), x["draft_tokens"], x["num_draft"], x["temperature"], x["u_accept"],
        x["u_sample"], probabilities)
    assert (margin > 1e-9).all(), "choose another seed"
    t, a, lp = (to_host(g) for g in got)
    assert np.array_equal(a, accepted)
    assert np.array_equal(t, tokens)
    assert np.all(np.abs(lp - logprobs) <= 2.0 ** -21 + 2.0 ** -24 * np.abs(logprobs))


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("draft", [None, "logits"])
@pytest.mark.parametrize("vocab", [1, 2, 17, 1000, 4096, 4097, 32003])
def test_verify_vocabularies(dtype, draft, vocab):
    x = block(vocab + 1, 6, 4, vocab, dtype, draft)
    check(x, run(x))


@pytest.mark.parametrize("draft", [None, "logits"])
@pytest.mark.parametrize("drafts", [0, 1, 15, 64])
def test_verify_block_lengths(draft, drafts):
    x = block(drafts, 5, drafts, 777, "fp16", draft)
    check(x, run(x))
    x["num_draft"] = np.array([0, drafts, drafts // 2, min(1, drafts), drafts + 9], np.int32)
    check(x, run(x))


def test_verify_output_head_size():
    x = block(3, 2, 7, 151936, "fp16", None)
    check(x, run(x))
    x = block(4, 2, 7, 151936, "fp32", "logits")
    check(x, run(x))


def test_verify_temperatures_and_greedy():
    for draft in (None, "logits"):
        x = block(5, 8, 5, 3001, "bf16", draft)
        x["temperature"] = np.array([0, 0.3, 1, 2.5, 0, -1, np.nan, 1e-30], np.float32)
        # at 1e-30 the largest logit is all there is: let it be one of a kind
        x["target"][7, :, 11] = 40.0
        if draft:
            x["draft"][7, :, 11] = 40.0
        for b in (0, 4, 5):      # greedy sequences accept some drafts
            x["draft_tokens"][b, :b] = x["target"][b, :b].float().argmax(1)
        check(x, run(x))


def test_verify_greedy_ties_take_the_lowest_index():
    x = block(6, 2, 2, 9000, "fp16", None)
    x["temperature"] = np.zeros(2, np.float32)
    x["target"][:, :, [8999, 5000, 4095]] = 30.0
    x["draft_tokens"][0] = [4095, 5000]
    got = run(x)
    check(x, got)
    assert to_host(got[0]).tolist() == [[4095, 4095, -1], [4095, -1, -1]]


def test_verify_probabilities():
    for draft in (None, "probs"):
        for vocab in (1, 50, 4097, 32003):
            x = block(vocab, 6, 3, vocab, "fp32", draft and "logits")
            p = torch.softmax(x["target"].double(), 2)
            p = torch.where(p >= 1e-3 * p.amax(2, True), p, 0)
            x["target"] = (p / p.sum(2, True)).float()
            if draft:
                q = torch.softmax(x["draft"].double(), 2)
                q = torch.where(q >= 1e-3 * q.amax(2, True), q, 0)
                x["draft"] = (q / q.sum(2, True)).float()
                if vocab > 50:
                    x["target"][0, 0, 5:9], x["draft"][1, 0, 5:9] = float("nan"), -0.5
            check(x, run(x, True), True)


def test_verify_draft_equal_to_the_target_is_always_accepted():
    x = block(8, 4, 6, 5000, "fp16", "logits")
    x["target"][:, :6] = x["draft"]
    x["u_accept"][:] = 0.999
    got = run(x)
    assert (to_host(got[1]) == 6).all()
    check(x, got)


def test_verify_what_is_left_over():
    """A draft that the target gives nothing to is always replaced, by what the
    draft row did not cover."""
    x = block(9, 3, 2, 300, "fp32", "logits")
    for b in range(3):
        x["target"][b, 0, x["draft_tokens"][b, 0]] = -float("inf")
    x["u_accept"][:] = 0.0
    check(x, run(x))
    # the target is certain of one other token
    x["target"][:] = -float("inf")
    x["target"][:, :, 123] = 2.0
    x["draft_tokens"][:, 0] = 7
    got = run(x)
    assert to_host(got[0]).tolist() == [[123, -1, -1]] * 3
    check(x, got)


def test_verify_one_candidate_left_without_a_draft_row():
    """Without a draft row a rejected draft is struck from p; if it was all of
    p, p is all there is."""
    x = block(10, 2, 1, 64, "fp32", None)
    x["target"][:] = -float("inf")
    x["target"][:, 0, 9] = 1.0
    x["draft_tokens"][:, 0] = [9, 8]
    x["target"][:, 1, 3] = 0.0
    x["u_accept"][:] = 0.5
    got = run(x)
    assert to_host(got[0]).tolist() == [[9, 3], [9, -1]]
    check(x, got)


def test_verify_infinities_and_nan():
    x = block(11, 4, 2, 500, "fp16", "logits")
    x["target"][0, 0, 100:] = -float("inf")
    x["target"][1, :, 77] = float("inf")
    x["target"][1, :, 78] = float("inf")
    x["target"][2, :, ::3] = float("nan")
    x["draft"][2, :, 1::3] = float("nan")
    x["target"][3] = float("nan")              # nothing can be picked
    got = run(x)
    assert to_host(got[0])[3].tolist() == [-1, -1, -1]
    xs = {k: (v[:3] if v is not None else None) for k, v in x.items()}
    check(xs, run(xs))
    assert torch.equal(got[0][:3], run(xs)[0])


def test_verify_draft_tokens_out_of_range():
    x = block(12, 3, 2, 100, "fp16", "logits")
    x["draft_tokens"][:, 0] = [-1, 100, 2 ** 31 - 1]
    x["u_accept"][:] = 0.0
    got = run(x)
    assert (to_host(got[1]) == 0).all()
    check(x, got)
    for draft in (None, "logits"):
        y = dict(x, temperature=np.zeros(3, np.float32))
        if draft is None:
            y["draft"] = None
        check(y, run(y))


def test_verify_extreme_random_numbers():
    """u = 0 takes the first token that counts, u just below 1 the last."""
    x = block(13, 2, 0, 5000, "fp32", None)
    x["target"][:] = -float("inf")
    x["target"][:, 0, 700:4200] = 0.0
    x["u_sample"][:] = [0.0, np.nextafter(np.float32(1), np.float32(0))]
    got = run(x)
    assert to_host(got[0]).ravel().tolist() == [700, 4199]
    assert np.all(np.abs(to_host(got[2]).ravel() + np.log(3500)) < 1e-5)


def test_verify_strided_rows():
    """Rows of a padded output head, starting anywhere, and one batch's rows shared by all."""
    for dtype in ("fp16", "fp32"):
        x = block(14, 3, 3, 2001, dtype, "logits")
        want = run(x)
        check(x, want)
        dev = {k: (v.to(DEV) if isinstance(v, torch.Tensor) else v) for k, v in x.items()}
        for lead, pad in ((0, 47), (3, 8), (5, 1)):
            def padded(t):
                buf = torch.full((t.shape[0] * t.shape[1] * (2001 + pad) + 16,), float("inf"), dtype=t.dtype, device=DEV)
                view = buf[lead:lead + t.shape[0] * t.shape[1] * (2001 + pad)].view(*t.shape[:2], 2001 + pad)[..., :2001]
                return view.copy_(t)
            y = dict(x, target=padded(dev["target"]), draft=padded(dev["draft"]))
            got = run(y)
            assert all(torch.equal(g, w) for g, w in zip(got, want)), (lead, pad)


def test_verify_distribution():
    """Over many blocks the first token is distributed as the target says,
    whatever the draft: speculative sampling's theorem. 40000 blocks; each
    frequency within five standard deviations."""
    vocab, n = 8, 40000
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    p = torch.tensor([0.0, 2.0, 1.0, -1.0, 0.5, 1.5, -2.0, 0.3], device=DEV)
    q = torch.tensor([1.0, 0.0, 1.0, 1.0, -0.5, 0.5, 0.0, 0.1], device=DEV)
    target, draft = p.expand(n, 2, vocab), q.expand(n, 1, vocab)
    drafts = torch.multinomial(torch.softmax(q, 0), n, True, generator=g).int().view(n, 1)
    u, v = torch.rand((n, 1), device=DEV, generator=g), torch.rand(n, device=DEV, generator=g)
    say("distribution")
    tokens, accepted, _ = qd.verify_drafts(target, drafts, u, v, draft=draft)
    pp = torch.softmax(p.double(), 0)
    freq = torch.bincount(tokens[:, 0].long(), minlength=vocab).double() / n
    assert ((freq - pp).abs() <= 5 * (pp * (1 - pp) / n).sqrt()).all()
    second = tokens[accepted == 1, 1].long()
    m = second.numel()
    freq = torch.bincount(second, minlength=vocab).double() / m
    assert ((freq - pp).abs() <= 5 * (pp * (1 - pp) / m).sqrt()).all()


def test_verify_empty_batch():
    say("empty")
    z = torch.zeros((0, 3, 10), device=DEV)
    t, a, lp = qd.verify_drafts(z, torch.zeros((0, 2), dtype=torch.int32, device=DEV), torch.zeros((0, 2), device=DEV),
                                torch.zeros(0, device=DEV))
    assert t.shape == (0, 3) and a.shape == (0,) and lp.shape == (0, 3)


def test_verify_graph_replay_and_outputs():
    x = block(15, 3, 4, 9001, "fp16", "logits")
    x["temperature"] = np.array([0.0, 0.7, 1.3], np.float32)
    dev = {k: (v.to(DEV) if isinstance(v, torch.Tensor) else None if v is None else torch.from_numpy(v).to(DEV))
           for k, v in x.items()}
    ws = qd.verify_workspace(3, 4, 9001)
    outs = {"tokens": torch.empty((3, 5), dtype=torch.int32, device=DEV),
            "accepted": torch.empty(3, dtype=torch.int32, device=DEV), "logprobs": torch.empty((3, 5), device=DEV)}

    def step():
        return qd.verify_drafts(dev["target"], dev["draft_tokens"], dev["u_accept"], dev["u_sample"],
                                draft=dev["draft"], temperature=dev["temperature"], workspace=ws, **outs)

    say("verify graph")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (16, 17, 18):
        y = block(seed, 3, 4, 9001, "fp16", "logits")
        y["temperature"] = np.array([1.0, 0.0, 0.5], np.float32)
        for k, v in y.items():
            if v is not None:
                if dev[k] is not None:
                    dev[k].copy_(v if isinstance(v, torch.Tensor) else torch.from_numpy(v))
        for o in outs.values():
            o.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        check(y, (outs["tokens"], outs["accepted"], outs["logprobs"]))
        got = {k: v.clone() for k, v in outs.items()}
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(got[k], outs[k]) for k in outs)
