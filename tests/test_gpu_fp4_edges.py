"""Edges of the 4-bit container and its product on the GPU, against the 64-bit definitions (microscale_ref.py):
tensor scales at the ends of a float, matrices without columns, every border between two codes, a wait that gives up."""
import ctypes

import numpy as np
import pytest
import torch

import microscale_ref as R
from test_gpu_fp4 import DTYPES, FMTS, check_quantized, random_fp4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dit_weight_compression_b200 import build
    build.build()
    import dit_weight_compression_b200 as ep
    return ep


@pytest.mark.parametrize("ga,gb", [(2.0 ** -149, 2.0 ** 127), (2.0 ** 127, -2.0 ** -148), (3e-40, 1e38), (-1e-44, 3e37), (2e38, 7e-45)])
@pytest.mark.parametrize("m", [2, 140, 2400])
def test_matmul_subnormal_tensor_scale(ep, m, ga, gb):
    """A tensor scale below a float's normal range beside a large one.  The sums are exact (multiples of 2^-4
    below 2^14), so that what is left are the roundings of two multiplications, 2^-24 each."""
    a, av = random_fp4(ep, m, 64, "nvfp4", 20, True)
    b, bv = random_fp4(ep, 2300, 64, "nvfp4", 21, True)
    a.tensor_scale.fill_(ga)
    b.tensor_scale.fill_(gb)
    want = (av @ bv.T) * float(a.tensor_scale) * float(b.tensor_scale)
    tol = (2.0 ** -23 + 2.0 ** -46) * want.abs()
    for bias in (None, torch.zeros(2300, device="cuda")):
        got = ep.fp4_matmul(a, b, bias=bias, dtype=torch.float32).double()
        assert bool(((got - want).abs() <= tol).all()), ((got - want).abs() / want.abs()).nan_to_num().max().item()


@pytest.mark.parametrize("m", [2, 140])
def test_matmul_tensor_scale_not_finite_or_zero(ep, m):
    """A tensor scale that is zero, infinite or NaN goes through the product as it would through floats."""
    a, av = random_fp4(ep, m, 64, "nvfp4", 22, True)
    b, bv = random_fp4(ep, 300, 64, "nvfp4", 23, True)
    for ga in (0.0, float("inf"), float("nan")):
        for gb in (1.0, 2.0 ** 100, 2.0 ** -149):
            a.tensor_scale.fill_(ga)
            b.tensor_scale.fill_(gb)
            want = ((av @ bv.T) * (ga * gb)).float()
            assert torch.equal(ep.fp4_matmul(a, b, dtype=torch.float32).nan_to_num(nan=7e30), want.nan_to_num(nan=7e30))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("shape", [(5, 0), (0, 64), (0, 0), (200, 0)])
def test_from_rows_empty(ep, fmt, shape):
    """Rows made elsewhere of a matrix without rows or columns, as the quantiser makes it."""
    rows, cols = shape
    data = torch.zeros(rows, 16 * -(-cols // 32), dtype=torch.uint8, device="cuda")
    sc = torch.zeros(rows, -(-cols // R.BLOCK[fmt]), dtype=torch.uint8, device="cuda")
    q = ep.FP4Tensor.from_rows(data, sc, torch.ones(1, device="cuda"), shape, fmt)
    like = ep.fp4_quantize(torch.zeros(shape, device="cuda"), fmt)
    assert q.shape == like.shape and q.nbytes == like.nbytes and q.scales.shape == like.scales.shape
    assert q.scale_rows().shape == sc.shape and float(q.tensor_scale) == 1.0
    assert ep.fp4_dequantize(q).shape == shape
    x = ep.fp4_quantize(torch.ones(3, cols, device="cuda"), fmt)
    y = ep.fp4_matmul(x, q, dtype=torch.float32)
    assert y.shape == (3, rows) and not y.any()


BORDERS = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]


def neighbours(v, dtype):
    """v, and the next numbers of its type on either side, as float64 (v > 0 is one itself)."""
    t = torch.from_numpy(v).to(dtype)
    assert torch.equal(t.double(), torch.from_numpy(v))
    bits = t.view(torch.int32 if dtype == torch.float32 else torch.int16)
    return [w.view(dtype).double().numpy() for w in (bits, bits - 1, bits + 1)]


def border_rows(fmt, dtype):
    """A row for each block scale q: 6 q first in every block, so that the scale is q, then every border of two
    codes times q, and its neighbours, with both signs."""
    sig, exp = (np.arange(8, 16) / 8.0, np.arange(-4, 6)) if fmt == "nvfp4" else (np.ones(1), np.arange(-6, 7))
    q = (sig[:, None] * np.exp2(exp)[None, :]).reshape(-1)
    on = q[:, None] * np.array(BORDERS)[None, :]
    v = np.concatenate(neighbours(on, dtype), 1)
    v = np.concatenate((v, -v), 1)
    per = R.BLOCK[fmt] - 1
    blocks = [np.concatenate((6 * q[:, None], v[:, i:i + per]), 1) for i in range(0, v.shape[1], per)]
    return q, np.concatenate(blocks, 1)


def check_borders_met(x, byte, fmt, dtype, g):
    """From the stored scales: every significand of a scale meets every border from both sides and on it."""
    q = R.scale_values(byte, fmt) * g
    blk = R.BLOCK[fmt]
    x = np.pad(x, ((0, 0), (0, -x.shape[1] % blk))).reshape(x.shape[0], -1, blk)
    seen = {(k, b): set() for k in range(3) for b in BORDERS}
    for b in BORDERS:
        for k, at in enumerate(neighbours(q * b, dtype)):
            for sign in (1, -1):
                hit = (x == sign * at[..., None]).any(-1)
                seen[(k, b)] |= {(float(s), sign) for s in np.frexp(q[hit])[0]}
    want = {(s / 16, sign) for s in (range(8, 16) if fmt == "nvfp4" else (8,)) for sign in (1, -1)}
    assert all(v == want for v in seen.values()), {k: len(v) for k, v in seen.items()}


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt,g", [("mxfp4", None), ("nvfp4", None), ("nvfp4", 1.0), ("nvfp4", 2.0)])
def test_quantize_on_and_beside_every_border(ep, fmt, dtype, g):
    q, x = border_rows(fmt, dtype)
    if fmt == "nvfp4" and g is None:  # the largest value is 6 * 60: the scale taken from the data is 2^-2
        assert R.tensor_scale(x) == 0.25
    t = torch.from_numpy(x).to(dtype).cuda()
    _, byte, used = check_quantized(ep, ep.fp4_quantize(t, fmt, **({} if g is None else {"tensor_scale": g})), t, g)
    assert np.array_equal(R.scale_values(byte, fmt) * used, np.repeat(q[:, None], byte.shape[1], 1))
    check_borders_met(x, byte, fmt, dtype, used)


def test_wait_that_gives_up_is_reported_once(ep):
    """A kernel whose barrier no copy ever reaches gives up after its short limit: the status is raised once,
    and the next product is right."""
    a, av = random_fp4(ep, 30, 256, "nvfp4", 1, True)
    b, bv = random_fp4(ep, 300, 256, "nvfp4", 2, True)
    L, st = ep.lib(), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    ep.op_status()
    assert L.ep_op_wait_probe(0, st) == -1
    ep.op_status()
    for _ in range(2):
        assert L.ep_op_wait_probe(2000, st) == 0, L.ep_last_error()
        with pytest.raises(ep.EPError) as e:
            ep.op_status()
        assert e.value.code == -6 and "gave up" in str(e.value)
        ep.op_status()
        assert torch.equal(ep.fp4_matmul(a, b, dtype=torch.float32).double(), av @ bv.T)
        ep.op_status()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("m,n,k,tile,rows,cols", [
    (100, 600, 4096, 3, (0, 100), (384, 512)),     # CTAs that share a tile: the last of them gives up
    (20, 600, 200, 4, (0, 20), (512, 600)),        # a CTA by itself
    (600, 1030, 512, 7, (256, 512), (512, 768))])  # pairs, a tile each
def test_tile_given_up_is_not_written(ep, fmt, m, n, k, tile, rows, cols):
    """A tile that one CTA gave up stays as it was, the others are right, and the status is raised once."""
    a, av = random_fp4(ep, m, k, fmt, 3, True)
    b, bv = random_fp4(ep, n, k, fmt, 4, True)
    want = (av @ bv.T).float()
    out = torch.full((m, n), 9.5, device="cuda")
    view = ep.EpTensor(out.data_ptr(), out.device.index, ep.F32, m, n, n)
    L, st = ep.lib(), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert L.ep_fp4_matmul_probe(a._ref, b._ref, ctypes.byref(view), -1, 1, st) == -1
    assert L.ep_fp4_matmul_probe(a._ref, b._ref, ctypes.byref(view), 0, 0, st) == -1
    ep.op_status()
    assert L.ep_fp4_matmul_probe(a._ref, b._ref, ctypes.byref(view), tile, 250000, st) == 0, L.ep_last_error()
    with pytest.raises(ep.EPError):
        ep.op_status()
    want_now = want.clone()
    want_now[rows[0]:rows[1], cols[0]:cols[1]] = 9.5
    assert torch.equal(out, want_now)
    assert torch.equal(ep.fp4_matmul(a, b, dtype=torch.float32), want)
    ep.op_status()
