"""Kernel variants of the block product that sizes of their own reach, signs of
codes, and blocks whose large products cancel, on the GPU. Tolerances as in
test_gpu_fp8_block."""

import pytest
import torch

from quantized_weight_skinny_amd import prompt_api as qp
from test_gpu_fp8_block import F8, _bounds, _check, _coded, _values, _weight

pytestmark = pytest.mark.gpu

SIZES = [
    # up to 16 rows that 16 wavefronts a workgroup share, whole and with a short last block
    (7, 100, 8336), (16, 64, 16384), (1, 4096, 8192),
    # 17 to 48 rows, eight wavefronts
    (20, 130, 4112), (32, 4096, 4224), (40, 100, 4240),
    # tiles of 256 alone: a last round almost full, whole rounds; two rounds and a rest in tiles of 128
    (513, 38300, 144), (1000, 16300, 144), (1025, 26800, 144),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_product(m, n, k, dtype):
    codes, scales = _coded(m, k)
    w = _weight(n, k)
    _check(qp.fp8_block_gemm(codes, scales, w, dtype=dtype), _values(codes, scales, 1), _values(w.codes, w.scales, 128))


@pytest.mark.parametrize("m,n,k", SIZES)
def test_linear(m, n, k):
    x = torch.randn((m, k), device="cuda", generator=torch.Generator("cuda").manual_seed(m)).bfloat16()
    w = _weight(n, k)
    codes, scales = qp.quantize_fp8_rows(x)
    assert torch.equal(qp.fp8_block_linear(x, w), qp.fp8_block_gemm(codes, scales, w))


@pytest.mark.parametrize("m,n", [(5, 45), (40, 130), (100, 300), (900, 5200), (300, 33000)])
def test_large_products_that_cancel(m, n):
    """Two products of 448 * 448 that cancel in every block, among small ones: a result of 32 bits keeps the small ones
    to fp32's rounding, one of 16 bits to 2^-10 of what has cancelled."""
    k = 528
    codes, _ = _coded(m, k)
    w = _weight(n, k, scales=torch.ones((-(-n // 128), -(-k // 128)), device="cuda"))
    c8, w8 = codes.view(torch.uint8), w.codes.view(torch.uint8)
    c8 &= 0x9F   # below 2^-2
    w8 &= 0x9F
    for at in (0, 130, 300, 511):
        c8[:, at:at + 2] = 0x7E
        w8[:, at], w8[:, at + 1] = 0x7E, 0xFE
    xs = torch.ones((m, 5), device="cuda")
    x, wv = _values(codes, xs, 1), _values(w.codes, w.scales, 128)
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        _check(qp.fp8_block_gemm(codes, xs, w, dtype=dtype), x, wv)
    ref, tol = _bounds(x, wv, torch.float32)
    assert float(ref.abs().max()) < 64 and float(tol.max()) < 60   # (against products of 200704)


def test_signs_of_codes():
    """Every element but NaN keeps its sign, those that round to zero too."""
    values = [0.0, 1e-42, 1e-44, 2.0 ** -130, 2.0 ** -20, 2.0 ** -11, 2.0 ** -10, 1.0, 447.0, float("inf"), float("nan")]
    x = torch.zeros((3, 128 * len(values)), device="cuda")
    for j, v in enumerate(values):
        x[0, 128 * j:128 * j + 128:3] = v
        x[1, 128 * j:128 * j + 128:2] = -v
        x[2, 128 * j:128 * j + 64], x[2, 128 * j + 64] = -v, 448.0
    for codes, _ in (qp.quantize_fp8_rows(x), qp.quantize_fp8_blocks(x)):
        there = x.isfinite()
        assert torch.equal(torch.signbit(codes.view(F8).float())[there], torch.signbit(x)[there])
        assert torch.equal(torch.isnan(codes.float()), ~there)
