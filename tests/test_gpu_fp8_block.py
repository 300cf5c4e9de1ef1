"""Products of 8-bit codes with a scale for each block of 128, on the GPU,
against the definition in 64 bits.

Tolerances. An fp32 result adds exact products in fp32: a sum of k terms is off
by at most (k + 64) 2^-24 of the sum of magnitudes, the two roundings of each
block's scaling among them. A result of 16 bits takes the matrix instruction of
the 8-bit formats, which keeps the products of a block to 2^-10 of the largest of
them (measured at most 2^-11.1 over random codes), so each block adds that, and
the result is rounded: by at most half a step of its type."""

import pytest
import torch

from quantized_weight_skinny_amd import QpnError
from quantized_weight_skinny_amd import prompt_api as qp

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn
HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(*shape, seed=0, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, device="cuda", generator=_gen(seed)) * std).to(dtype)


def _quantized(x, block_rows):
    """Codes and scales by the definition: the least power of two s >= 2^-126 with amax <= 448 s."""
    rows, k = x.shape
    wide = torch.nn.functional.pad(x.double(), (0, -k % 128, 0, -rows % block_rows))
    b = wide.view(wide.shape[0] // block_rows, block_rows, -1, 128)
    finite = torch.where(b.isfinite(), b, 0.0).abs().amax((1, 3))
    s = torch.ones_like(finite)
    for e in range(-126, 122):
        step = 2.0 ** e
        s = torch.where((finite > 448.0 * step / 2) & ((finite <= 448.0 * step) | (e == 121)), step, s)
    s = torch.where((finite > 0) & (finite <= 448.0 * 2.0 ** -126), 2.0 ** -126, s)
    q = b / s[:, None, :, None]
    a = q.abs().clamp(min=2.0 ** -6)
    step = (a.view(torch.int64) >> 52 << 52).view(torch.float64) / 8  # spacing of E4M3 at a
    v = torch.round(q / step) * step
    v = torch.where(b.isfinite(), v, float("nan"))
    return v.view(wide.shape)[:rows, :k], s


def _values(codes, scales, block_rows):
    rows, k = codes.shape
    s = scales.double().repeat_interleave(block_rows, 0)[:rows].repeat_interleave(128, 1)[:, :k]
    return codes.view(F8).float().double() * s


def _bounds(x, w, dtype):
    """The exact product of 64-bit values and how far a result of this type may be off."""
    y = x @ w.T
    k = x.shape[1]
    tol = (k + 64) * 2.0 ** -24 * (x.abs() @ w.abs().T)
    if dtype in HALF_STEP:
        for at in range(0, k, 128):
            # the largest product of a block is at most the product of its largest factors
            tol += 2.0 ** -10 * x[:, at:at + 128].abs().amax(1)[:, None] * w[:, at:at + 128].abs().amax(1)[None]
        tol += HALF_STEP[dtype] * (y.abs() + tol) + 2.0 ** -25
    return y, tol


def _weight(n, k, seed=1, scales=None):
    codes = _normal(n, k, seed=seed, std=90.0).clamp(-448, 448).to(F8)
    if scales is None:
        scales = torch.rand((-(-n // 128), -(-k // 128)), device="cuda", generator=_gen(seed + 50)) * 1e-3 + 1e-4
    return qp.BlockWeight(codes, scales)


def _coded(m, k, seed=2):
    codes = _normal(m, k, seed=seed, std=90.0).clamp(-448, 448).to(F8)
    return codes, torch.rand((m, -(-k // 128)), device="cuda", generator=_gen(seed + 50)) * 0.01 + 0.001


def _check(y, x, w, dtype=None):
    ref, tol = _bounds(x, w, y.dtype)
    off = (y.double() - ref).abs()
    assert (off <= tol).all(), (float((off / tol).max()), y.shape)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,k", [(1, 1), (1, 16), (3, 130), (33, 1296), (257, 127), (130, 129), (5, 1000)])
def test_quantizer_is_exact(dtype, rows, k):
    x = _normal(rows, k, seed=rows + k, std=3.0, dtype=dtype)
    x[rows // 2, :k // 2] = 0
    for block_rows, fn in ((1, qp.quantize_fp8_rows), (128, qp.quantize_fp8_blocks)):
        codes, scales = fn(x)
        v, s = _quantized(x, block_rows)
        assert torch.equal(scales.double(), s)
        assert torch.equal(codes.float().double(), v)


def test_quantizer_at_borders():
    top = torch.finfo(torch.float32).max
    blocks = [
        [448.0, 447.9, 1.0],                       # amax at the border: scale 1
        [448.00003, 1.0, -3.3],                    # just above: scale 2
        [224.0, -0.0, 0.0],                        # scale 1/2
        [0.0, -0.0, 0.0],                          # zeros: scale 1, signs kept
        [1e-42, -1e-44, 0.0],                      # subnormals: the least scale
        [2.0 ** -126 * 448, 2.0 ** -130, 1e-40],
        [top, -top, 1.0],
        [float("inf"), 7.0, -3.0],                 # does not count for the scale
        [float("-inf"), float("nan"), 0.5],
        [float("nan"), float("nan"), float("inf")],
        [17.0, 19.0, 448.0],                       # ties between 16, 18 and 20: to even
        [2.0 ** -10, 3 * 2.0 ** -10, 448.0],       # ties of the subnormals: 0 and 2 steps
    ]
    x = torch.zeros((2, 128 * len(blocks)), device="cuda")
    for j, b in enumerate(blocks):
        x[0, 128 * j:128 * j + 3] = torch.tensor(b, device="cuda")
        x[1, 128 * j + 125:128 * j + 128] = -torch.tensor(b, device="cuda")
    codes, scales = qp.quantize_fp8_rows(x)
    v, s = _quantized(x, 1)
    assert torch.equal(scales.double(), s)
    assert torch.equal(codes.float().double().nan_to_num(nan=1e9), v.nan_to_num(nan=1e9))
    assert torch.equal(torch.signbit(codes.float()), torch.signbit(x)) or torch.isnan(x).any()
    zero = (x == 0)
    assert torch.equal(torch.signbit(codes.float())[zero], torch.signbit(x)[zero])


def test_quantizer_strides():
    wide = _normal(40, 700, dtype=torch.bfloat16)
    x = wide[::2, 3:3 + 333]                      # rows apart, odd start
    codes = torch.full((20, 500), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((20, 9), -7.0, device="cuda")
    c, s = qp.quantize_fp8_rows(x, codes=codes[:, 5:338], scales=scales[:, 1:7:2])
    v, sr = _quantized(x, 1)
    assert torch.equal(c.view(F8).float().double(), v) and torch.equal(s.double(), sr)
    assert (codes[:, :5] == 0x55).all() and (codes[:, 338:] == 0x55).all()
    assert (scales[:, 0::2] == -7).all() and (scales[:, 7:] == -7).all()


SIZES = [(1, 1, 16), (1, 17, 128), (2, 130, 144), (16, 16, 2304), (17, 257, 1296), (33, 129, 112), (48, 40, 4096),
         (49, 300, 272), (64, 1, 128), (64, 513, 1040), (65, 128, 16), (128, 129, 128), (129, 127, 1296), (200, 64, 5120),
         (300, 25700, 144), (257, 1000, 2048), (300, 33000, 272), (513, 25000, 144), (1100, 4000, 400), (70, 200, 9232),
         (50, 10500, 4096), (130, 5500, 8192)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_product(m, n, k, dtype):
    codes, scales = _coded(m, k)
    w = _weight(n, k)
    y = qp.fp8_block_gemm(codes, scales, w, dtype=dtype)
    _check(y, _values(codes, scales, 1), _values(w.codes, w.scales, 128))


@pytest.mark.parametrize("x_dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,n,k", [(1, 200, 1296), (20, 33, 400), (100, 300, 528)])
def test_linear_is_the_quantizer_and_the_product(x_dtype, m, n, k):
    x, w = _normal(m, k, dtype=x_dtype), _weight(n, k)
    codes, scales = qp.quantize_fp8_rows(x)
    for dtype in (torch.float32, torch.bfloat16):
        assert torch.equal(qp.fp8_block_linear(x, w, dtype=dtype), qp.fp8_block_gemm(codes, scales, w, dtype=dtype))
    y = qp.fp8_block_linear(x, w, dtype=torch.float32)
    _check(y, _values(codes, scales, 1), _values(w.codes, w.scales, 128))
    assert qp.fp8_block_linear(x, w).dtype is x_dtype


@pytest.mark.parametrize("m,n", [(5, 300), (100, 300)])
def test_one_hot_rows_read_the_weight_back(m, n):
    """Row r picks element 37 r + 11 of the weight's rows: one product, every other 0."""
    k = 1296 * 4
    w = _weight(n, k, scales=torch.full((-(-n // 128), -(-k // 128)), 0.5, device="cuda"))
    at = (torch.arange(m, device="cuda") * 37 + 11) % k
    x = torch.zeros((m, k), device="cuda", dtype=torch.float16)
    x[torch.arange(m), at] = 1.0
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        y = qp.fp8_block_linear(x, w, dtype=dtype)
        assert torch.equal(y.double(), (w.codes.float().double() * 0.5)[:, at].T)


@pytest.mark.parametrize("m,n,k", [(3, 45, 272), (70, 141, 400), (300, 25700, 128)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strides_and_what_lies_around(m, n, k, dtype):
    codes, scales = _coded(m, k)
    w = _weight(n, k)
    y = qp.fp8_block_gemm(codes, scales, w, dtype=dtype)
    # rows further apart, scales transposed and apart, outputs inside a larger tensor at an odd place
    far = torch.full((m, k + 48), 0x7F, dtype=torch.uint8, device="cuda")
    far[:, 16:16 + k] = codes.view(torch.uint8)
    wide = torch.full((n, k + 32), 0x7F, dtype=torch.uint8, device="cuda")
    wide[:, :k] = w.codes.view(torch.uint8)
    st = torch.full((scales.shape[1], 2 * m), float("nan"), device="cuda")
    st[:, ::2] = scales.T
    wt = torch.full((w.scales.shape[1], w.scales.shape[0] + 3), float("nan"), device="cuda")
    wt[:, 1:-2] = w.scales.T
    apart = qp.BlockWeight(wide[:, :k], wt[:, 1:-2].T)
    around = torch.full((m, n + 9), 3.0, dtype=dtype, device="cuda")
    out = qp.fp8_block_gemm(far[:, 16:16 + k], st[:, ::2].T, apart, dtype=dtype, out=around[:, 3:3 + n])
    assert torch.equal(out, y)
    assert (around[:, :3] == 3).all() and (around[:, 3 + n:] == 3).all()


@pytest.mark.parametrize("m,n,k", [(4, 40, 256), (100, 200, 384)])
def test_nan_codes_stay_in_their_row_and_column(m, n, k):
    codes, scales = _coded(m, k)
    w = _weight(n, k)
    clean = qp.fp8_block_gemm(codes, scales, w)
    codes.view(torch.uint8)[2, 130] = 0x7F
    w.codes.view(torch.uint8)[33, 7] = 0xFF
    y = qp.fp8_block_gemm(codes, scales, w)
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[2], bad[:, 33] = True, True
    assert torch.isnan(y[bad]).all() and torch.equal(y[~bad], clean[~bad])


def test_empty_sizes():
    w = _weight(40, 128)
    assert qp.fp8_block_linear(torch.empty((0, 128), device="cuda"), w).shape == (0, 40)
    none = qp.BlockWeight(torch.empty((40, 0), dtype=F8, device="cuda"), torch.empty((1, 0), device="cuda"))
    for m in (3, 100):
        assert (qp.fp8_block_linear(torch.empty((m, 0), device="cuda"), none) == 0).all()
    empty = qp.BlockWeight(torch.empty((0, 128), dtype=F8, device="cuda"), torch.empty((0, 1), device="cuda"))
    assert qp.fp8_block_linear(torch.zeros((3, 128), device="cuda"), empty).shape == (3, 0)


def test_offsets_beyond_32_bits():
    """A weight of 2.5 GB and an output of 2.4 billion elements: their last rows and columns."""
    n, k = 151936, 16384
    codes = torch.zeros((n, k), dtype=torch.uint8, device="cuda")
    some = torch.tensor([0, 1, 131071, 131072, 131073, n - 17, n - 1], device="cuda")
    codes[some] = _normal(len(some), k, std=90.0).to(F8).view(torch.uint8)
    w = qp.BlockWeight(codes, torch.full((-(-n // 128), k // 128), 2.0 ** -6, device="cuda"))
    for m in (2, 80):
        c, s = _coded(m, k)
        y = qp.fp8_block_gemm(c, s, w, dtype=torch.float32)
        _check(y[:, some], _values(c, s, 1), codes[some].view(F8).float().double() * 2.0 ** -6)
        assert (y[:, 2:131071] == 0).all()
    del codes, w, y
    m, n, k = 16001, 151936, 128
    c, s = _coded(m, k)
    w = _weight(n, k)
    y = qp.fp8_block_gemm(c, s, w, dtype=torch.float16)
    rows, cols = torch.tensor([0, 14133, 14134, m - 1], device="cuda"), slice(n - 300, n)
    _check(y[rows][:, cols], _values(c, s, 1)[rows], _values(w.codes, w.scales, 128)[cols])


def test_captured_calls_and_workspaces_of_their_own():
    sizes = [(3, 200, 1296), (100, 200, 5120)]
    state = []
    for m, n, k in sizes:
        x, w = _normal(m, k, dtype=torch.bfloat16), _weight(n, k)
        state.append((x, w, qp.fp8_block_workspace(m, n, k), torch.empty((m, n), dtype=torch.bfloat16, device="cuda")))
    def call():
        for x, w, ws, out in state:
            qp.fp8_block_linear(x, w, out=out, workspace=ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed in range(4):
        for x, *_ in state:
            x.copy_(_normal(*x.shape, seed=seed + 9))
        graph.replay()
        torch.cuda.synchronize()
        for x, w, _, out in state:
            assert torch.equal(out, qp.fp8_block_linear(x, w))
    # the other stream's call has a workspace of its own
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y1 = qp.fp8_block_linear(state[1][0], state[1][1])
    y2 = qp.fp8_block_linear(state[1][0], state[1][1])
    torch.cuda.synchronize()
    assert torch.equal(y1, y2)


def test_rows_do_not_depend_on_their_neighbours():
    """A row alone gives what it gives among others where both take the same sums; and every repeat the same bits."""
    codes, scales = _coded(300, 2048)
    w = _weight(400, 2048)
    y = qp.fp8_block_gemm(codes, scales, w, dtype=torch.float32)
    assert torch.equal(y, qp.fp8_block_gemm(codes, scales, w, dtype=torch.float32))
    few = qp.fp8_block_gemm(codes[:30], scales[:30], w, dtype=torch.float32)
    assert torch.equal(few[7:8], qp.fp8_block_gemm(codes[7:8], scales[7:8], w, dtype=torch.float32))


def test_refusals():
    w = _weight(40, 256)
    x = _normal(3, 256, dtype=torch.float16)
    with pytest.raises(ValueError, match="shape"):
        qp.fp8_block_linear(x[:, :128], w)
    with pytest.raises(ValueError, match="contiguous"):
        qp.fp8_block_linear(_normal(256, 3).T, w)
    with pytest.raises(ValueError, match="one of"):
        qp.fp8_block_linear(x.double(), w)
    with pytest.raises(ValueError, match="dtype"):
        qp.fp8_block_linear(x, w, dtype=torch.float64)
    with pytest.raises(ValueError, match="out"):
        qp.fp8_block_linear(x, w, out=torch.empty((3, 41), dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError, match="CUDA"):
        qp.fp8_block_linear(x.cpu(), w)
    with pytest.raises(ValueError, match="scales"):
        qp.fp8_block_gemm(*_coded(3, 256)[:1], torch.ones((3, 3), device="cuda"), w)
    with pytest.raises(ValueError, match="16"):
        qp.BlockWeight(torch.zeros((40, 260), dtype=torch.uint8, device="cuda")[:, 2:258], torch.ones((1, 2), device="cuda"))
    with pytest.raises(ValueError, match="16"):
        qp.BlockWeight(torch.zeros((40, 250), dtype=torch.uint8, device="cuda"), torch.ones((1, 2), device="cuda"))
    with pytest.raises(ValueError, match="workspace"):
        qp.fp8_block_linear(x, w, workspace=torch.empty((64, 4096), dtype=torch.uint8, device="cuda").T)
    with pytest.raises(QpnError):
        qp.fp8_block_linear(_normal(3, 256)[:, :256], qp.BlockWeight(
            torch.zeros((2, 1 << 23), dtype=torch.uint8, device="cuda")[:, :256], torch.ones((1, 2), device="cuda")))
