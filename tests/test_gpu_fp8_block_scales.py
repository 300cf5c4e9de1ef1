"""Block products whose scales of x and w have a product outside fp32's normal
range, on the GPU: results inside the range are right all the same.

Tolerances as in test_gpu_fp8_block: (k + 64) 2^-24 of the sum of magnitudes, for
16 bits also 2^-10 of the largest product of each block and the rounding. Results
below the normal range are off by at most half a step of the subnormals: 2^-150, bf16 2^-134."""

import pytest
import torch

from quantized_weight_skinny_amd import prompt_api as qp
from test_gpu_fp8_block import F8, HALF_STEP, _coded, _values, _weight

pytestmark = pytest.mark.gpu
K = 528   # four blocks and a short one
SIZES = [(5, 45), (20, 300), (40, 130), (64, 70), (100, 300), (900, 5200), (300, 33000)]  # each kernel and tile


def _inputs(m, n):
    """Blocks of factors 2^-1, 2^130, 2^-140, 2^-10 (of 2^90 and 2^-100) and 1 (short). Block 1 is zeros in even rows
    and one code of 2^-9 in odd ones, times weights of a few 2^-9; every third row has block 2 alone."""
    codes, _ = _coded(m, K)
    c8 = codes.view(torch.uint8)
    c8[:, 128:256] = 0
    c8[1::2, 128 + 77] = 0x81
    c8[::3, :256], c8[::3, 384:] = 0, 0
    xs = torch.tensor([0.5, 2.0 ** 100, 2.0 ** -100, 2.0 ** 90, 1.0], device="cuda").repeat(m, 1)
    xs *= 1 + torch.arange(m, device="cuda")[:, None] % 7 / 8
    xs[1::4] *= -1
    w = _weight(n, K)
    w8 = w.codes.view(torch.uint8)
    w8[:, 128:256] = w8[:, 128:256] & 0x87
    ws = torch.tensor([1.0, 2.0 ** 30, 2.0 ** -40, 2.0 ** -100, 1.0], device="cuda").repeat(-(-n // 128), 1)
    ws *= 1 + torch.arange(ws.shape[0], device="cuda")[:, None] % 5 / 8
    return codes, xs, qp.BlockWeight(w.codes, ws)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m,n", SIZES)
def test_factors_beyond_the_range(m, n, dtype):
    codes, xs, w = _inputs(m, n)
    y = qp.fp8_block_gemm(codes, xs, w, dtype=dtype)
    xv, wv = _values(codes, xs, 1), _values(w.codes, w.scales, 128)
    ref = xv @ wv.T
    tol = (K + 64) * 2.0 ** -24 * (xv.abs() @ wv.abs().T)
    if dtype is torch.bfloat16:
        for at in range(0, K, 128):
            tol += 2.0 ** -10 * xv[:, at:at + 128].abs().amax(1)[:, None] * wv[:, at:at + 128].abs().amax(1)[None]
        tol += HALF_STEP[dtype] * (ref.abs() + tol) + 2.0 ** -134
    tol += 2.0 ** -150
    assert y.isfinite().all()
    off = (y.double() - ref).abs()
    assert (off <= tol).all(), float((off / tol).max())
    assert (y[::3] != 0).any() and (ref[::3].abs() < 2.0 ** -100).all()   # (those rows show the smallest factors)
    assert (ref[1::6].abs().amax(1) > 2.0 ** 105).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m,n", SIZES)
def test_other_rows_keep_their_bits(m, n, dtype):
    """Rows of ordinary factors are the same beside rows whose factors leave the range."""
    codes, scales = _coded(m, K)
    w = _weight(n, K)
    y = qp.fp8_block_gemm(codes, scales, w, dtype=dtype)
    odd = scales.clone()
    odd[::5] *= 2.0 ** -125
    again = qp.fp8_block_gemm(codes, odd, w, dtype=dtype)
    keep = torch.arange(m, device="cuda") % 5 != 0
    assert torch.equal(y[keep], again[keep])


@pytest.mark.parametrize("m,n", SIZES)
def test_odd_scales(m, n):
    """Zeros, infinities and NaN among the scales, as fp32 multiplies them."""
    codes, scales = _coded(m, K)
    c8 = codes.view(torch.uint8)
    c8[c8 == 0x80] = 0
    w = _weight(n, K)
    clean = qp.fp8_block_gemm(codes, scales, w, dtype=torch.float32)
    odd = scales.clone()
    odd[0, 1], odd[1, 2], odd[2], odd[3, 4] = float("nan"), float("inf"), 0.0, -float("inf")
    y = qp.fp8_block_gemm(codes, odd, w, dtype=torch.float32)
    assert torch.isnan(y[0]).all() and not y[1].isfinite().any() and (y[2] == 0).all() and not y[3].isfinite().any()
    assert torch.equal(y[4:], clean[4:])


def test_codes_are_what_the_formats_say():
    assert float(torch.tensor([0x81], dtype=torch.uint8).view(F8).float()) == -2.0 ** -9
