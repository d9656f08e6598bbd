"""The 4-bit container and its product on the GPU against the 64-bit definitions (microscale_ref.py).

Quantisation and dequantisation are compared bit for bit: the formats define every rounding of the exact
quotient.  Products: with power-of-two scales of a small range every partial sum is a float, so the
result is exact whatever the order; with general scales a sum of K / block floats, each exact for one
block, is off by at most (K / block) * 2^-23 * sum |a b| (one truncation a step), plus 2^-24 relative for each of the
three factors of the scaling and half a step of the output's type.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import microscale_ref as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu
FMTS = ["mxfp4", "nvfp4"]
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dit_weight_compression_b200 import build
    build.build()
    import dit_weight_compression_b200 as ep
    return ep


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def sample(rows, cols, dtype, seed, spread=4.0):
    """Normal values with rows of different size, exact ties, a row of zeros, and signs of zero."""
    g = gen(seed)
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x *= torch.exp(spread * (torch.rand(rows, 1, generator=g, device="cuda") - 0.5))
    if rows > 2:
        x[1] = 0.0
        ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, -0.0], device="cuda")
        x[2] = ties.repeat(-(-cols // 10))[:cols] * torch.sign(x[2])
    return x.to(dtype)


def check_quantized(ep, q, x, g=None):
    ref = x.detach().double().cpu().numpy()
    el, byte, g = R.quantize(ref, q.format, g)
    rows, cols = ref.shape
    got = R.unpack(q.data.cpu().numpy())
    assert float(q.tensor_scale) == g
    assert np.array_equal(q.scale_rows().cpu().numpy(), byte)
    assert np.array_equal(got[:, :el.shape[1]], el[:, :got.shape[1]])
    assert not got[:, cols:].any()
    # the paddings of the scale tiles are zeros: as many non-zero bytes as the scales have
    assert int((q.scales != 0).sum()) == int((byte != 0).sum())
    return el, byte, g


SHAPES = [(1, 1), (1, 8192), (3, 17), (5, 64), (127, 33), (128, 128), (129, 257), (300, 1000), (64, 4096), (260, 72)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("shape", SHAPES)
def test_quantize(ep, fmt, dtype, shape):
    x = sample(*shape, dtype, 1000 * shape[0] + shape[1])
    check_quantized(ep, ep.fp4_quantize(x, fmt), x)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_quantize_every_16_bit_value_near_borders(ep, fmt, dtype):
    """Blocks whose scale takes every E4M3 significand, with values on and around every border."""
    tops = torch.arange(1, 257, device="cuda").float()                       # block maxima
    borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    rows = []
    for s in (-1, 0, 1):
        v = borders[None, :] * torch.arange(8, 16, device="cuda")[:, None]    # significand x border
        v = v.repeat(32, 1) * torch.exp2(torch.randint(-4, 3, (256, 1), generator=gen(5), device="cuda").float())
        v = v * (1 + s * torch.finfo(dtype).eps / 2)
        rows.append(torch.cat((tops[:, None], v.to(dtype).float(), -v.to(dtype).float()), 1)[:, :16])
    x = torch.cat(rows).to(dtype).repeat(1, 2)
    check_quantized(ep, ep.fp4_quantize(x, fmt), x)
    if fmt == "nvfp4":
        check_quantized(ep, ep.fp4_quantize(x, fmt, tensor_scale=0.125), x, 0.125)


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_extremes(ep, fmt):
    """Tiny, subnormal and huge values, and a matrix whose blocks span the whole range of a float."""
    x = torch.zeros(8, 96, device="cuda")
    x[0] = torch.linspace(-3e38, 3e38, 96, device="cuda")
    x[1] = 1e-45 * torch.arange(96, device="cuda")
    x[2] = 2.0 ** -126 * torch.arange(96, device="cuda")
    x[3] = torch.exp2(torch.arange(96, device="cuda").float() - 40)
    x[4] = 2.0 ** -120
    x[5, :3] = torch.tensor([1e-30, -1e-37, 1e-38], device="cuda")
    x[6] = torch.finfo(torch.float32).max
    check_quantized(ep, ep.fp4_quantize(x, fmt), x)
    check_quantized(ep, ep.fp4_quantize(x[1:3].contiguous(), fmt), x[1:3])
    z = torch.zeros(3, 40, device="cuda", dtype=torch.float16)
    check_quantized(ep, ep.fp4_quantize(z, fmt), z)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows", [4, 2000])
def test_quantize_not_finite(ep, fmt, dtype, rows):
    """A block with a NaN or an infinity gets a NaN scale and restores as NaNs; the others are as if it
    were not there.  (2000 rows: the maximum comes from its own pass.)"""
    x = sample(rows, 160, dtype, 9)
    x[0, 3], x[0, 70], x[3, 159] = float("nan"), float("inf"), float("-inf")
    q = ep.fp4_quantize(x, fmt)
    el, byte, g = check_quantized(ep, q, x)
    got = ep.fp4_dequantize(q, dtype=torch.float32).double().cpu().numpy()
    want = R.values(el, byte, g, 160, fmt)
    assert np.array_equal(got, want, equal_nan=True)
    blk = R.BLOCK[fmt]
    assert np.isnan(got[0, :blk]).all() and np.isnan(got).sum() == 3 * blk


@pytest.mark.parametrize("g", [2.0 ** -100, 2.0 ** -9, 1.0, 2.0 ** 20, 2.0 ** 117])
def test_quantize_given_tensor_scale(ep, g):
    x = sample(200, 100, torch.bfloat16, 3)
    check_quantized(ep, ep.fp4_quantize(x, "nvfp4", tensor_scale=g), x, g)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("off,stride", [(0, 272), (1, 272), (8, 264), (3, 261)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strides_and_alignment(ep, fmt, off, stride, dtype):
    """Column windows of wider matrices: in through the quantiser, out through the dequantiser, whose
    neighbours stay as they were."""
    big = sample(150, stride, dtype, 4)
    x = big[:, off:off + 250]
    q = ep.fp4_quantize(x, fmt)
    el, byte, g = check_quantized(ep, q, x)
    out = torch.full((150, stride), 7.0, dtype=dtype, device="cuda")
    ep.fp4_dequantize(q, out=out[:, off:off + 250])
    want = torch.full((150, stride), 7.0, dtype=torch.float64)
    want[:, off:off + 250] = torch.from_numpy(R.values(el, byte, g, 250, fmt))
    assert torch.equal(out.double().cpu(), want)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("off", [0, 5, 8])
def test_long_rows_apart(ep, dtype, off):
    """Rows of several runs of the maximum's own pass, with gaps between them; the largest value is the last."""
    big = sample(6, 20011, dtype, 8)
    x = big[:, off:off + 20000]
    x[5, 19999] = 3e4
    check_quantized(ep, ep.fp4_quantize(x, "nvfp4"), x)
    y = x.contiguous()
    assert torch.equal(ep.fp4_quantize(y, "nvfp4").data, ep.fp4_quantize(x, "nvfp4").data)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(1, 1), (3, 47), (129, 257), (200, 640)])
def test_dequantize_any_codes(ep, fmt, dtype, shape):
    """Every code and scale, rows made elsewhere, a tensor scale that is no power of two."""
    g = gen(shape[1])
    rows, cols = shape
    data = torch.randint(0, 256, (rows, 16 * -(-cols // 32)), generator=g, device="cuda", dtype=torch.uint8)
    lo, hi = (110, 140) if fmt == "mxfp4" else (0, 127)
    sc = torch.randint(lo, hi, (rows, -(-cols // R.BLOCK[fmt])), generator=g, device="cuda", dtype=torch.uint8)
    ts = torch.tensor([0.3 if fmt == "nvfp4" else 1.0], device="cuda")
    q = ep.FP4Tensor.from_rows(data, sc, ts, shape, fmt)
    assert torch.equal(q.scale_rows(), sc)
    got = ep.fp4_dequantize(q, dtype=dtype)
    v = R.values(R.unpack(data.cpu().numpy()), sc.cpu().numpy(), 1.0, cols, fmt)
    want = (torch.from_numpy(v).float() * ts.cpu()).to(dtype)
    assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("fmt", FMTS)
def test_empty(ep, fmt):
    for shape in ((0, 64), (5, 0), (0, 0)):
        q = ep.fp4_quantize(torch.zeros(shape, device="cuda"), fmt)
        assert ep.fp4_dequantize(q).shape == shape
        assert float(q.tensor_scale) == (1.0 if fmt == "mxfp4" else 2.0 ** -100)
    a = ep.fp4_quantize(torch.zeros(3, 0, device="cuda"), fmt)
    b = ep.fp4_quantize(torch.zeros(200, 0, device="cuda"), fmt)
    bias = torch.randn(200, device="cuda").bfloat16()
    assert torch.equal(ep.fp4_matmul(a, b, bias=bias), bias.expand(3, 200))
    assert not ep.fp4_matmul(a, b, dtype=torch.float32).any()
    e = ep.fp4_quantize(torch.zeros(0, 64, device="cuda"), fmt)
    w = ep.fp4_quantize(torch.ones(8, 64, device="cuda"), fmt)
    assert ep.fp4_matmul(e, w).shape == (0, 8) and ep.fp4_matmul(w, e).shape == (8, 0)


def test_offsets_past_32_bits(ep):
    """A matrix of 4.5 G elements: only its last rows hold anything."""
    rows, cols = 35000, 131072
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-3:] = sample(3, cols, torch.bfloat16, 5)
    q = ep.fp4_quantize(x, "mxfp4")
    el, byte, _ = R.quantize(x[-3:].double().cpu().numpy(), "mxfp4")
    assert np.array_equal(R.unpack(q.data[-3:].cpu().numpy()), el)
    y = ep.fp4_dequantize(q, out=x)
    assert torch.equal(y[-3:].double().cpu(), torch.from_numpy(R.values(el, byte, 1.0, cols, "mxfp4")))
    assert not y[-1000:-3].any()


# ---- products ----------------------------------------------------------------------------------
def random_fp4(ep, rows, cols, fmt, seed, plain):
    """Random codes; scales 0.5, 1 or 2 (`plain`: any partial sum of 4096 products is a float), or any
    from a wide range with a tensor scale."""
    g = gen(seed)
    data = torch.randint(0, 256, (rows, 16 * -(-cols // 32)), generator=g, device="cuda", dtype=torch.uint8)
    blocks = -(-cols // R.BLOCK[fmt])
    if plain:
        ks = torch.randint(-1, 2, (rows, blocks), generator=g, device="cuda")
        sc = (127 + ks if fmt == "mxfp4" else (7 + ks) * 8).to(torch.uint8)
        ts = torch.ones(1, device="cuda")
    else:
        lo, hi = (117, 137) if fmt == "mxfp4" else (1, 127)
        sc = torch.randint(lo, hi, (rows, blocks), generator=g, device="cuda", dtype=torch.uint8)
        ts = torch.tensor([0.37 if fmt == "nvfp4" else 1.0], device="cuda")
    q = ep.FP4Tensor.from_rows(data, sc, ts, (rows, cols), fmt)
    v = R.values(R.unpack(data.cpu().numpy()), sc.cpu().numpy(), float(ts), cols, fmt)
    return q, torch.from_numpy(v).cuda()


MATMULS = [(1, 1, 1), (1, 128, 256), (1, 300, 64), (2, 129, 65), (7, 40, 4096), (16, 257, 500), (17, 1000, 1024), (33, 128, 2048),
           (64, 513, 100), (65, 130, 333), (100, 100, 100), (128, 2, 3000), (129, 64, 64), (130, 300, 1111), (256, 256, 256),
           (300, 700, 1500), (520, 1030, 4096), (2100, 130, 320), (1, 5000, 4000), (3000, 4200, 96), (2500, 2600, 700), (1000, 512, 4096),
           (140, 20000, 128), (257, 255, 4095)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("m,n,k", MATMULS)
def test_matmul_exact(ep, fmt, m, n, k):
    a, av = random_fp4(ep, m, k, fmt, 1, True)
    b, bv = random_fp4(ep, n, k, fmt, 2, True)
    got = ep.fp4_matmul(a, b, dtype=torch.float32)
    ep.op_status()
    assert torch.equal(got.double(), av @ bv.T)


HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def check_product(got, av, bv, bias, blk):
    want, size = av @ bv.T, av.abs() @ bv.abs().T
    if bias is not None:
        want = want + bias.double()
        size = size + bias.double().abs()
    k = av.shape[1]
    tol = (-(-k // blk) + 2) * 2.0 ** -23 * size
    tol = tol + HALF[got.dtype] * (want.abs() + tol) + (2.0 ** -25 if got.dtype == torch.float16 else 0)
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), (err / tol).max().item()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("m,n,k", [(1, 700, 8192), (20, 333, 1000), (128, 640, 5000), (200, 520, 2100), (2048, 2304, 1024)])
def test_matmul_general_scales_and_bias(ep, fmt, dtype, m, n, k):
    a, av = random_fp4(ep, m, k, fmt, 3, False)
    b, bv = random_fp4(ep, n, k, fmt, 4, False)
    if dtype == torch.float16:  # keep the results inside the type's range
        a = ep.FP4Tensor.from_rows(a.data, a.scale_rows(), a.tensor_scale * 2.0 ** -12, a.shape, fmt)
        av = av * 2.0 ** -12
    bias = torch.randn(n, generator=gen(6), device="cuda").to(dtype)
    check_product(ep.fp4_matmul(a, b, bias=bias, dtype=dtype), av, bv, bias, R.BLOCK[fmt])
    check_product(ep.fp4_matmul(a, b, dtype=dtype), av, bv, None, R.BLOCK[fmt])
    ep.op_status()


@pytest.mark.parametrize("ga,gb", [(100, 90), (-100, -45), (-60, -100), (110, -110), (-90, 117), (127, 127)])
@pytest.mark.parametrize("m", [2, 140, 2400])
def test_matmul_tensor_scales_far_apart(ep, m, ga, gb):
    """2^ga and 2^gb whose product is no float: the sums here are multiples of 2^-4 below 2^14, so the
    result is the exact one rounded once, and sums that are zero stay zero."""
    a, av = random_fp4(ep, m, 64, "nvfp4", 20, True)
    b, bv = random_fp4(ep, 2300, 64, "nvfp4", 21, True)
    a.data[0] = 0
    av[0] = 0
    for sign in (1.0, -1.0):
        a.tensor_scale.fill_(sign * 2.0 ** ga)
        b.tensor_scale.fill_(2.0 ** gb)
        want = ((av @ bv.T) * (sign * 2.0 ** ga) * 2.0 ** gb).float()
        assert torch.equal(ep.fp4_matmul(a, b, dtype=torch.float32), want)
        bias = torch.zeros(2300, device="cuda")
        assert torch.equal(ep.fp4_matmul(a, b, bias=bias, dtype=torch.float32), want)


@pytest.mark.parametrize("m", [3, 150, 2400])
def test_matmul_strided_and_misaligned_out(ep, m):
    """Windows of a wider output: the neighbours stay as they were."""
    a, av = random_fp4(ep, m, 512, "nvfp4", 7, True)
    b, bv = random_fp4(ep, 2100, 512, "nvfp4", 8, True)
    want = av @ bv.T
    for off, stride in ((0, 2112), (3, 2111)):
        for dtype in (torch.float32, torch.bfloat16):
            out = torch.full((m, stride), 9.0, dtype=dtype, device="cuda")
            ep.fp4_matmul(a, b, out=out[:, off:off + 2100])
            assert torch.equal(out[:, off:off + 2100], want.to(dtype) if dtype == torch.bfloat16 else want.float())
            assert bool((out[:, :off] == 9).all()) and bool((out[:, off + 2100:] == 9).all())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("m", [4, 140, 2500])
def test_matmul_nan_stays_in_its_row_and_column(ep, fmt, m):
    n, k = 2300, 200
    x, w = sample(m, k, torch.float32, 10, 0.5), sample(n, k, torch.float32, 11, 0.5)
    x[m - 1, k - 1], w[5, 0] = float("inf"), float("nan")
    y = ep.fp4_matmul(ep.fp4_quantize(x, fmt), ep.fp4_quantize(w, fmt), dtype=torch.float32)
    bad = torch.zeros(m, n, dtype=torch.bool, device="cuda")
    bad[m - 1], bad[:, 5] = True, True
    assert torch.equal(y.isnan(), bad)


@pytest.mark.parametrize("m", [1, 40, 300, 3000])
def test_matmul_same_bits_again(ep, m):
    a, _ = random_fp4(ep, m, 4096, "nvfp4", 12, False)
    b, _ = random_fp4(ep, 2048, 4096, "nvfp4", 13, False)
    y = ep.fp4_matmul(a, b, dtype=torch.float32)
    for _ in range(5):
        assert torch.equal(ep.fp4_matmul(a, b, dtype=torch.float32), y)


# ---- as they are used ----------------------------------------------------------------------------
@pytest.mark.parametrize("fmt", FMTS)
def test_blob_to_linear_layer(ep, fmt):
    """A weight matrix from its blob into 4 bits, and a linear layer with it: the same bits as from the
    restored weights, and the values of the formats' definitions."""
    w = (torch.randn(520, 1000, generator=gen(20), device="cuda") * 0.02).bfloat16()
    blob = ep.compress(w, 4.0)
    w4 = ep.decompress_fp4(blob, fmt)
    ep.decode_status(blob)
    restored = ep.decompress(blob)
    el, byte, g = check_quantized(ep, w4, restored)
    q = ep.fp4_quantize(restored, fmt)
    assert torch.equal(q.data, w4.data) and torch.equal(q.scales, w4.scales) and torch.equal(q.tensor_scale, w4.tensor_scale)
    w32 = ep.decompress_fp4(blob, fmt, dtype=torch.float32)
    check_quantized(ep, w32, ep.decompress(blob, dtype=torch.float32))
    bias = torch.randn(520, generator=gen(21), device="cuda").bfloat16()
    wv = torch.from_numpy(R.values(el, byte, g, 1000, fmt)).cuda()
    for m in (1, 50, 400):
        x = sample(m, 1000, torch.bfloat16, 22 + m)
        xq = ep.fp4_quantize(x, fmt)
        xe, xb, xg = R.quantize(x.double().cpu().numpy(), fmt)
        xv = torch.from_numpy(R.values(xe, xb, xg, 1000, fmt)).cuda()
        check_product(ep.fp4_matmul(xq, w4, bias=bias), xv, wv, bias, R.BLOCK[fmt])


def test_streams_and_graphs(ep):
    """A captured linear layer replayed on new activations, two graphs and an eager call side by side, and
    calls on a stream given by hand."""
    w = ep.fp4_quantize(sample(1024, 512, torch.bfloat16, 30), "nvfp4")

    def layer(x):
        return ep.fp4_matmul(ep.fp4_quantize(x, "nvfp4"), w)

    xs = [sample(m, 512, torch.bfloat16, 31 + m) for m in (1, 700, 3)]
    want = [layer(x) for x in xs]
    torch.cuda.synchronize()
    graphs = []
    for x in xs[:2]:
        buf = torch.zeros_like(x)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = layer(buf)
        graphs.append((g, buf, y))
    side = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for (g, buf, y), x, s in zip(graphs, xs, side):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                y.zero_()
                buf.copy_(x)
                g.replay()
        assert torch.equal(layer(xs[2]), want[2])
        torch.cuda.synchronize()
        for (g, buf, y), e in zip(graphs, want):
            assert torch.equal(y, e)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for st in (s, s.cuda_stream):
        q = ep.fp4_quantize(xs[1], "nvfp4", stream=st)
        y = ep.fp4_matmul(q, w, stream=st)
        d = ep.fp4_dequantize(q, stream=st)
        s.synchronize()
        assert torch.equal(y, want[1]) and torch.equal(d, ep.fp4_dequantize(q))
    ep.op_status()


def test_products_side_by_side(ep):
    """Products of every kind on four streams at once, sharing weights: each as if it were alone."""
    w = ep.fp4_quantize(sample(3000, 2048, torch.bfloat16, 40), "nvfp4")
    xs = [ep.fp4_quantize(sample(m, 2048, torch.bfloat16, 41 + m), "nvfp4") for m in (1, 60, 300, 2100)]
    want = [ep.fp4_matmul(x, w) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for x, s in zip(xs, streams):
            got.append(ep.fp4_matmul(x, w, stream=s))
    torch.cuda.synchronize()
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % 4])
    ep.op_status()


def test_inputs_dropped_while_another_stream_reads_them(ep):
    """Calls on a stream given by hand hold on to their inputs: the allocator does not hand them out again
    before that stream is done with them."""
    s = torch.cuda.Stream()
    w = ep.fp4_quantize(sample(4096, 4096, torch.bfloat16, 50), "nvfp4")
    big = ep.fp4_quantize(sample(8192, 4096, torch.bfloat16, 51), "nvfp4")
    x = sample(2048, 4096, torch.bfloat16, 52)
    want = ep.fp4_matmul(ep.fp4_quantize(x, "nvfp4"), w)
    torch.cuda.synchronize()
    for _ in range(5):
        for _ in range(4):
            ep.fp4_matmul(big, w, stream=s)               # the stream is busy
        q = ep.fp4_quantize(x, "nvfp4")
        s.wait_stream(torch.cuda.current_stream())
        y = ep.fp4_matmul(q, w, stream=s)
        n = q._buffer.numel()
        del q
        for _ in range(8):
            torch.full((n,), 255, dtype=torch.uint8, device="cuda")
        s.synchronize()
        assert torch.equal(y, want)


def test_first_calls_in_a_capture(ep):
    """A process whose first product of every kind is captured: the look-ups that a first call makes are
    none that a capture forbids."""
    code = (
        "import torch, dit_weight_compression_b200 as ep\n"
        "g = torch.cuda.CUDAGraph()\n"
        "x = torch.randn(700, 512, device='cuda'); w = torch.randn(4096, 512, device='cuda')\n"
        "with torch.cuda.graph(g):\n"
        "    ys = [ep.fp4_matmul(ep.fp4_quantize(x[:m], f), ep.fp4_quantize(w, f)) for f in ('mxfp4', 'nvfp4') for m in (1, 20, 50, 100, 700)]\n"
        "g.replay(); torch.cuda.synchronize(); ep.op_status()\n"
        "for y, (f, m) in zip(ys, [(f, m) for f in ('mxfp4', 'nvfp4') for m in (1, 20, 50, 100, 700)]):\n"
        "    assert torch.equal(y, ep.fp4_matmul(ep.fp4_quantize(x[:m], f), ep.fp4_quantize(w, f)))\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_python_argument_errors(ep):
    x = torch.randn(4, 64, device="cuda")
    q, w = ep.fp4_quantize(x, "nvfp4"), ep.fp4_quantize(x, "mxfp4")
    with pytest.raises(ep.EPError):
        ep.fp4_matmul(q, w)
    with pytest.raises(ep.EPError):
        ep.fp4_matmul(q, ep.fp4_quantize(x[:, :32], "nvfp4"))
    with pytest.raises(ValueError):
        ep.fp4_matmul(q, q, bias=torch.zeros(3, device="cuda"))
    with pytest.raises(ValueError):
        ep.fp4_quantize(x, "nvfp4", out=w)
    with pytest.raises(ValueError):
        ep.fp4_quantize(x.T, "nvfp4")
    with pytest.raises(ep.EPError):
        ep.fp4_quantize(x[:1].expand(4, 64), "nvfp4")     # rows that overlap
    with pytest.raises(ep.EPError):
        ep.fp4_quantize(x, "mxfp4", tensor_scale=1.0)
    with pytest.raises(ep.EPError):
        ep.fp4_quantize(x.to(torch.int8), "nvfp4")
    with pytest.raises(ep.EPError):
        ep.fp4_dequantize(q, out=torch.empty(4, 64))
