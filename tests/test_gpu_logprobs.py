"""Log-probabilities of given tokens, entropies, ranks and first tokens, on the
GPU, against the definition in 64 bits.

Tolerances. A weight 2^((x - m) f) has an exponent of two roundings (2^-23 of its
size) and an exponential good to 2^-22; a lane adds 32-bit sums over at most 2^-9 of
the vocabulary's elements, one of 2^-24 each (the rest is 64 bits). So a row's sum is
off by 2^-22 + 2^-23 E|x - m| / (t ln 2) + n / 512 2^-24, E over p, and its logarithm by as much; the
rest of a log-probability is 64 bits and one rounding. The entropy has this twice, and
its dot product is off by that much of E|x - m| / t."""

import math

import pytest
import torch

from gpu_helpers import DEV, say
from quantized_weight_skinny_amd import QpnError
from quantized_weight_skinny_amd import prompt_api as qp

pytestmark = pytest.mark.gpu
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def _rows(rows, vocab, dtype, seed=0, std=2.5):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn((rows, vocab), device=DEV, generator=gen) * std
    tokens = torch.randint(0, vocab, (rows,), device=DEV, generator=gen).to(torch.int32)
    return x.to(TYPES[dtype]), tokens


def check(logits, tokens, top, got, temperature=None):
    logp, entropy, rank, best, best_logp = got
    rows, vocab = logits.shape
    for r in range(rows):
        x = logits[r].double()
        x = torch.where(torch.isnan(x), -math.inf, x)
        t = float(temperature[r]) if temperature is not None else 1.0
        t = t if t > 0 else 1.0
        m = x.max()
        if m == math.inf:
            p = (x == m).double()
            spread = 0.0
        elif m == -math.inf:
            p, spread = torch.zeros_like(x), 0.0
        else:
            p = torch.exp((x - m) / t)
            spread = float((p * torch.where(p > 0, (m - x) / t, 0.0)).sum() / p.sum())
        z = p.sum()
        p = p / z if z > 0 else p
        lp = torch.log(p)
        if m.isfinite():   # tiny probabilities keep their logarithm
            lp = torch.where(x > -math.inf, (x - m) / t - torch.log(z), -math.inf)
        off = 2.0 ** -22 + 2.0 ** -23 * spread / math.log(2) + vocab / 512 * 2.0 ** -24
        def near(a, b):
            return a == b or abs(a - b) <= off + 2.0 ** -23 * abs(b)
        order = torch.sort(x, descending=True, stable=True).indices
        assert torch.equal(best[r].long(), order[:top]), r
        for j in range(top):
            assert near(float(best_logp[r, j]), float(lp[order[j]])), (r, j)
        h = float(-(p[p > 0] * lp[p > 0]).sum())
        assert abs(float(entropy[r]) - h) <= (2 + spread) * off + 2.0 ** -23 * h, (r, float(entropy[r]), h)
        g = int(tokens[r])
        if 0 <= g < vocab:
            assert near(float(logp[r]), float(lp[g])), (r, float(logp[r]), float(lp[g]))
            assert int(rank[r]) == int((order == g).nonzero()[0, 0]), r
        else:
            assert float(logp[r]) == 0 and int(rank[r]) == -1


def run(logits, tokens, top, temperature=None, **kw):
    say("token_logprobs", tuple(logits.shape), logits.dtype, top)
    got = qp.token_logprobs(logits, tokens, top=top, temperature=temperature, **kw)
    check(logits, tokens, top, got, temperature)
    return got


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows,vocab,top", [
    (1, 1, 1), (2, 1, 0), (3, 7, 7), (5, 64, 64), (4, 65, 64), (7, 1000, 20), (2, 2047, 1), (3, 2049, 5), (3, 8191, 33),
    (2, 8193, 20), (9, 50021, 0), (9, 50021, 20), (1, 151936, 64), (33, 33333, 5), (3000, 100, 3)])
def test_against_the_definition(rows, vocab, top, dtype):
    run(*_rows(rows, vocab, dtype, seed=rows + vocab), top)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_many_rows_take_one_slice(dtype):
    """2048 rows and more: a row is one workgroup's."""
    x, tokens = _rows(2100, 20011, dtype)
    got = qp.token_logprobs(x, tokens, top=9)
    some = torch.arange(0, 2100, 61, device=DEV)
    check(x[some], tokens[some], 9, [y[some] for y in got])


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("order", ["rising", "falling", "equal", "few values", "late peak"])
def test_orders_that_lists_find_hard(order, dtype):
    vocab = 40000
    x = torch.linspace(-9, 9, vocab, device=DEV).expand(2, vocab)
    x = {"rising": x, "falling": x.flip(1), "equal": torch.zeros_like(x) - 3, "few values": (x * 7 % 3).round(),
         "late peak": torch.where(torch.arange(vocab, device=DEV) > vocab - 500, x + 5, -x)}[order]
    run(x.to(TYPES[dtype]).contiguous(), torch.tensor([17, vocab - 3], dtype=torch.int32, device=DEV), 40)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_odd_rows(dtype):
    """Infinities, NaN, the type's lowest and largest, signed zeros, and given tokens among them."""
    t = TYPES[dtype]
    vocab, inf, nan = 9000, math.inf, math.nan
    low, high = torch.finfo(t).min, torch.finfo(t).max
    x, _ = _rows(14, vocab, dtype, seed=4)
    x[0, :] = -inf
    x[1, :] = nan
    x[2, :] = low
    x[3, 5:] = -inf                      # fewer tokens than asked for
    x[4, ::3] = nan
    x[5, [7, 4000, 8999]] = inf          # share the probability
    x[6, :] = inf
    x[7, ::2], x[7, 1::2] = 0.0, -0.0    # equal
    x[8, 1:] = low                       # a mask of the lowest value
    x[9, [3, 4]] = high
    x[10, :] = -inf
    x[10, 8998] = 1.0
    x[11, 100] = nan
    x[12, 200] = -inf
    x[13, :] = nan
    x[13, 8191:8193] = torch.tensor([-inf, low], device=DEV).to(t)
    for at in (0, 3, 100, 200, 4000, 8191, 8192, 8998, 8999, -1, vocab, -2 ** 31, 2 ** 31 - 1):
        run(x, torch.full((14,), at, dtype=torch.int32, device=DEV), 12)
    run(x, torch.full((14,), 4, dtype=torch.int32, device=DEV), 64)
    run(x, torch.full((14,), 4, dtype=torch.int32, device=DEV), 0)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_temperatures(dtype):
    x, tokens = _rows(10, 5000, dtype, seed=6)
    t = torch.tensor([1.0, 0.3, 5.0, 0.0, -2.0, math.nan, 1e-6, 1e6, 0.05, 1.7], device=DEV)
    run(x, tokens, 10, temperature=t)


def test_extreme_temperatures_stay_finite():
    x, tokens = _rows(4, 300, "fp32", seed=8)
    t = torch.tensor([1e-45, 1e-38, 3e38, math.inf], device=DEV)
    logp, entropy, rank, best, best_logp = qp.token_logprobs(x, tokens, top=2, temperature=t)
    assert (best_logp[:2, 0] == 0).all() and (entropy[:2] == 0).all()
    assert (entropy[2:] - math.log(300)).abs().max() < 1e-5 and (best_logp[2:] + math.log(300)).abs().max() < 1e-5
    assert not torch.isnan(logp).any()


@pytest.mark.parametrize("dtype", list(TYPES))
def test_strides_alignment_and_what_lies_around(dtype):
    x, tokens = _rows(6, 10007, dtype, seed=9)
    got = run(x, tokens, 5)
    for shift in (1, 3):
        wide = torch.full((6, 10007 + 9), math.nan, dtype=TYPES[dtype], device=DEV)
        wide[:, shift:shift + 10007] = x
        wide[:, shift + 10007:] = math.inf
        outs = [torch.full((8, *y.shape[1:]), 77, dtype=y.dtype, device=DEV) for y in got]
        names = ("logprobs", "entropy", "rank", "top_tokens", "top_logprobs")
        again = qp.token_logprobs(wide[:, shift:shift + 10007], tokens, top=5,
                                  **{n: o[1:7] for n, o in zip(names, outs)})
        for a, b, o in zip(got, again, outs):
            assert torch.equal(a, b) and (o[0] == 77).all() and (o[7] == 77).all()


def test_rows_beyond_32_bits():
    rows, vocab = 15000, 151936  # 4.6 GB
    x = torch.zeros((rows, vocab), dtype=torch.float16, device=DEV)
    some = torch.tensor([0, 7066, 14133, 14134, rows - 1], device=DEV)
    y, _ = _rows(5, vocab, "fp16", seed=10)
    x[some] = y
    tokens = torch.arange(rows, dtype=torch.int32, device=DEV) * 10
    got = qp.token_logprobs(x, tokens, top=3)
    check(y, tokens[some], 3, [z[some] for z in got])
    assert (got[2][1:7066] == tokens[1:7066]).all()


def test_captured_and_on_another_stream():
    x, tokens = _rows(5, 30011, "bf16")
    ws = qp.token_logprobs_workspace(5, 30011, 8)
    outs = [torch.empty(s, dtype=d, device=DEV) for s, d in (((5,), torch.float32), ((5,), torch.float32),
            ((5,), torch.int32), ((5, 8), torch.int32), ((5, 8), torch.float32))]
    call = lambda: qp.token_logprobs(x, tokens, 8, None, *outs, workspace=ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed in range(4):
        y, t = _rows(5, 30011, "bf16", seed=seed + 20)
        x.copy_(y)
        tokens.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        check(x, tokens, 8, outs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = qp.token_logprobs(x, tokens, 8)
    again = qp.token_logprobs(x, tokens, 8)
    torch.cuda.synchronize()
    for a, b, c in zip(outs, other, again):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_refusals():
    x, tokens = _rows(3, 100, "fp16")
    with pytest.raises(ValueError, match="tokens"):
        qp.token_logprobs(x, tokens.long())
    with pytest.raises(ValueError, match="tokens"):
        qp.token_logprobs(x, tokens[:2])
    with pytest.raises(ValueError, match="logits"):
        qp.token_logprobs(x[None], tokens)
    with pytest.raises(ValueError, match="contiguous"):
        qp.token_logprobs(_rows(100, 3, "fp16")[0].T, tokens)
    with pytest.raises(ValueError, match="temperature"):
        qp.token_logprobs(x, tokens, temperature=torch.ones(3, device=DEV).half())
    with pytest.raises(QpnError):
        qp.token_logprobs(x, tokens, top=65)
    with pytest.raises(QpnError):
        qp.token_logprobs(x[:, :20], tokens, top=21)
    with pytest.raises(QpnError):
        qp.token_logprobs(x[:, :0], tokens)
    assert qp.token_logprobs(x[:0], tokens[:0], top=4)[3].shape == (0, 4)
