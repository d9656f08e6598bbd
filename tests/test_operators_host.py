"""Refusals of the 4-bit and cache entry points, and the sizes they report: host checks that come before
any device is looked at, so they run without one.  No pointer given here is ever followed."""
import ctypes

import pytest
import torch

P = 4096  # an aligned address that is not used


@pytest.fixture(scope="module")
def ep():
    from dit_weight_compression_b200 import build
    build.build()
    import dit_weight_compression_b200 as ep
    return ep


def dense(ep, rows, cols, dtype=1, data=P, stride=None, device=0):
    return ep.EpTensor(data, device, dtype, rows, cols, cols if stride is None else stride)


def fp4(ep, rows, cols, fmt=7, data=P, scales=P, g=P, device=0):
    return ep.EpFP4Tensor(data, scales, g, device, fmt, rows, cols)



ARG, DTYPE, SHAPE = -1, -2, -3


@pytest.mark.parametrize("fmt,rows,cols,want", [
    (6, 1, 1, (16, 512)), (7, 1, 1, (16, 512)), (6, 129, 130, (129 * 80, 512 * 2 * 2)), (7, 128, 64, (128 * 32, 512)),
    (7, 128, 65, (128 * 48, 1024)), (6, 0, 5, (0, 0)), (7, 5, 0, (0, 0)), (6, 1 << 20, 1 << 14, ((1 << 33), 512 * (1 << 13) * 128))])
def test_sizes(ep, fmt, rows, cols, want):
    d, s = ctypes.c_size_t(), ctypes.c_size_t()
    assert ep.lib().ep_fp4_sizes(fmt, rows, cols, ctypes.byref(d), ctypes.byref(s)) == 0
    assert (d.value, s.value) == want


@pytest.mark.parametrize("fmt,rows,cols,want", [(5, 1, 1, DTYPE), (7, -1, 1, SHAPE), (7, 1, -1, SHAPE), (6, 1, (1 << 30) + 1, SHAPE)])
def test_sizes_refused(ep, fmt, rows, cols, want):
    d, s = ctypes.c_size_t(), ctypes.c_size_t()
    assert ep.lib().ep_fp4_sizes(fmt, rows, cols, ctypes.byref(d), ctypes.byref(s)) == want
    assert ep.lib().ep_fp4_sizes(7, 1, 1, None, ctypes.byref(s)) == ARG


def test_quantize_refused(ep):
    q = ep.lib().ep_fp4_quantize
    r = ctypes.byref

    def call(x, out, g=0.0):
        return q(r(x), r(out), g, None)

    x, out = dense(ep, 4, 64), fp4(ep, 4, 64)
    assert q(None, r(out), 0.0, None) == ARG and q(r(x), None, 0.0, None) == ARG
    assert call(dense(ep, 4, 64, dtype=3), out) == DTYPE and call(dense(ep, 4, 64, dtype=6), out) == DTYPE
    assert call(x, fp4(ep, 4, 64, fmt=1)) == DTYPE and call(x, fp4(ep, 4, 64, fmt=8)) == DTYPE
    assert call(x, fp4(ep, 4, 65)) == SHAPE and call(x, fp4(ep, 5, 64)) == SHAPE
    assert call(dense(ep, -4, 64), fp4(ep, -4, 64)) == SHAPE
    assert call(dense(ep, 4, 64, data=None), out) == ARG and call(dense(ep, 4, 64, data=P + 1), out) == ARG
    assert call(dense(ep, 4, 64, stride=63), out) == ARG
    for bad in (dict(data=None), dict(scales=None), dict(g=None), dict(data=P + 8), dict(scales=P + 4), dict(g=P + 2)):
        assert call(x, fp4(ep, 4, 64, **bad)) == ARG, bad
    for g in (-1.0, 3.0, 0.75, float("nan"), float("inf"), 2.0 ** -101, 2.0 ** 118):
        assert call(x, out, g) == ARG, g
    assert call(x, fp4(ep, 4, 64, fmt=6), 1.0) == ARG
    assert b"tensor_scale" in ep.lib().ep_last_error() or b"tensor scale" in ep.lib().ep_last_error()


def test_dequantize_refused(ep):
    dq, r = ep.lib().ep_fp4_dequantize, ctypes.byref
    x, out = fp4(ep, 4, 64), dense(ep, 4, 64)
    assert dq(None, r(out), None) == ARG and dq(r(x), None, None) == ARG
    assert dq(r(x), r(dense(ep, 4, 64, dtype=5)), None) == DTYPE
    assert dq(r(x), r(dense(ep, 4, 63)), None) == SHAPE
    assert dq(r(x), r(dense(ep, 4, 64, stride=60)), None) == ARG
    assert dq(r(fp4(ep, 4, 64, fmt=4)), r(out), None) == DTYPE


def test_matmul_refused(ep):
    mm, r = ep.lib().ep_fp4_matmul, ctypes.byref

    def call(a, b, out, bias=None):
        return mm(r(a), r(b), bias, r(out), None)

    a, b, out = fp4(ep, 4, 64), fp4(ep, 9, 64), dense(ep, 4, 9)
    assert mm(None, r(b), None, r(out), None) == ARG and mm(r(a), r(b), None, None, None) == ARG
    assert call(a, fp4(ep, 9, 64, fmt=6), out) == DTYPE
    assert call(a, fp4(ep, 9, 96), out) == SHAPE
    assert call(a, b, dense(ep, 4, 8)) == SHAPE and call(a, b, dense(ep, 9, 4)) == SHAPE
    assert call(a, b, dense(ep, 4, 9, dtype=3)) == DTYPE
    assert call(a, b, dense(ep, 4, 9, data=None)) == ARG and call(a, b, dense(ep, 4, 9, data=P + 1)) == ARG
    assert call(a, b, dense(ep, 4, 9, stride=8)) == ARG
    assert call(a, b, out, P + 1) == ARG


def test_decompress_fp4_refused(ep):
    blob = ep.compress(torch.randn(16, 64), 4.0)
    f, r = ep.lib().ep_decompress_fp4, ctypes.byref
    out, work = fp4(ep, 16, 64), dense(ep, 16, 64)
    assert f(None, r(out), 0.0, r(work), None) == ARG and f(blob.handle, r(out), 0.0, None, None) == ARG
    assert f(blob.handle, r(fp4(ep, 16, 32)), 0.0, r(dense(ep, 16, 32)), None) == SHAPE
    assert f(blob.handle, r(out), 0.0, r(dense(ep, 16, 64, dtype=3)), None) == DTYPE
    assert f(blob.handle, r(out), 0.3, r(work), None) == ARG


def cache(ep, fmt=3, n_pages=4, page=16, heads=2, dim=64, data=P, scales=P, device=0):
    return ep.EpCache(data, scales, device, fmt, n_pages, page, heads, dim)


def heads(ep, dtype=1, tokens=5, n=2, dim=64, data=P, ts=128, hs=64, device=0):
    return ep.EpHeads(data, device, dtype, tokens, n, dim, ts, hs)


BAD_PAIRS = [
    (dict(fmt=1), {}, DTYPE), (dict(fmt=4), {}, DTYPE), ({}, dict(dtype=3), DTYPE), ({}, dict(dtype=5), DTYPE),
    (dict(n_pages=-1), {}, SHAPE), (dict(page=0), {}, SHAPE), (dict(heads=0), dict(n=0), SHAPE), (dict(dim=0), dict(dim=0), SHAPE),
    (dict(dim=1025), dict(dim=1025), SHAPE), ({}, dict(tokens=-1), SHAPE), ({}, dict(n=3), SHAPE), ({}, dict(dim=32), SHAPE),
    (dict(n_pages=1 << 40), {}, SHAPE), ({}, dict(ts=-1), ARG), ({}, dict(hs=-64), ARG), (dict(data=None), {}, ARG),
    (dict(scales=None), {}, ARG), (dict(data=P + 8), {}, ARG), (dict(scales=P + 2), {}, ARG), ({}, dict(data=None), ARG),
    ({}, dict(data=P + 1), ARG)]


@pytest.mark.parametrize("c,h,want", BAD_PAIRS)
def test_cache_refused(ep, c, h, want):
    r = ctypes.byref
    L = ep.lib()
    assert L.ep_cache_write(r(cache(ep, **c)), r(heads(ep, **h)), 1, P, None) == want
    assert L.ep_cache_read(r(cache(ep, **c)), r(heads(ep, **h)), 1, P, 4, 4, 2, P, None) == want


def test_cache_arguments_refused(ep):
    r, L = ctypes.byref, ep.lib()
    c, h = cache(ep), heads(ep)
    assert L.ep_cache_write(None, r(h), 1, P, None) == ARG and L.ep_cache_write(r(c), None, 1, P, None) == ARG
    assert L.ep_cache_write(r(c), r(h), 0, P, None) == ARG and L.ep_cache_write(r(c), r(h), 3, P, None) == ARG
    assert L.ep_cache_write(r(c), r(h), 1, None, None) == ARG and L.ep_cache_write(r(c), r(h), 1, P + 4, None) == ARG
    assert L.ep_cache_read(r(c), r(h), 1, P, 3, 4, 2, P, None) == ARG      # stride below pages per sequence
    assert L.ep_cache_read(r(c), r(h), 1, P, 4, -1, 2, P, None) == ARG
    assert L.ep_cache_read(r(c), r(h), 1, P, 4, 4, -1, P, None) == ARG
    assert L.ep_cache_read(r(c), r(h), 1, None, 4, 4, 2, P, None) == ARG
    assert L.ep_cache_read(r(c), r(h), 1, P, 4, 4, 2, None, None) == ARG
    two = (ep.EpCache * 2)(c, cache(ep, page=32))
    assert L.ep_cache_write(two, (ep.EpHeads * 2)(h, h), 2, P, None) == SHAPE
    two = (ep.EpCache * 2)(c, cache(ep, fmt=5))
    assert L.ep_cache_write(two, (ep.EpHeads * 2)(h, h), 2, P, None) == SHAPE
    two = (ep.EpCache * 2)(c, c)
    assert L.ep_cache_write(two, (ep.EpHeads * 2)(h, heads(ep, tokens=4)), 2, P, None) == SHAPE
    assert L.ep_cache_write(two, (ep.EpHeads * 2)(h, heads(ep, dtype=4)), 2, P, None) == DTYPE


def test_python_refusals(ep):
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        ep.fp4_quantize(x, "nvfp4")          # not on a CUDA device
    with pytest.raises(ValueError):
        ep.FP4Tensor((4, 64), "fp4", "cpu")
    with pytest.raises(ValueError):
        ep.KVCache(1, 16, 2, 64, "int4", "cpu")
    with pytest.raises(ValueError):
        ep.FP4Tensor((1, (1 << 30) + 1), "mxfp4", "cpu")


def test_codec_refuses_the_new_containers(ep):
    """The 4-bit formats are no element type of a plain tensor: the codec's own calls refuse them."""
    t = ep.EpTensor(P, -1, 6, 4, 64, 64)
    h = ctypes.c_void_p()
    assert ep.lib().ep_compress(ctypes.byref(t), 4.0, ctypes.byref(h)) == DTYPE


# For calls that every check of pointers and sizes lets pass: the device that they name is not there, so
# they end before a launch with a GPU as well as without one.
NOWHERE = 4000


def refused(ep, rc, words):
    """Whether a call that ended with an error did so for `words`."""
    assert rc != 0
    return words in ep.lib().ep_last_error().decode()


def test_cache_write_into_one_pool_refused(ep):
    """Keys and values of one call may not share bytes (64 slots, 2 heads of 64: 8192 bytes of rows and 512
    of scales a cache)."""
    L, h = ep.lib(), heads(ep, device=NOWHERE)
    k = cache(ep, data=P, scales=P + 8192, device=NOWHERE)
    for data, scales, want in ((0, 32768, True), (16384, 8192, True), (8176, 32768, True), (8688, 32768, True),
                               (16384, 8188, True), (16384, 8700, True), (8704, 32768, False), (32768, 8704, False)):
        v = cache(ep, data=P + data, scales=P + scales, device=NOWHERE)
        for two in ((k, v), (v, k)):
            rc = L.ep_cache_write((ep.EpCache * 2)(*two), (ep.EpHeads * 2)(h, h), 2, P, None)
            assert refused(ep, rc, "share memory") == want, (data, scales)
            assert not want or rc == ARG


def test_cache_read_rows_apart(ep):
    """Output rows that overlap are refused; either order of tokens and heads is not."""
    L, r, c = ep.lib(), ctypes.byref, cache(ep, device=NOWHERE)
    big = 1 << 62

    def overlap(c=c, **kw):
        rc = L.ep_cache_read(r(c), r(heads(ep, device=NOWHERE, **kw)), 1, P, 4, 4, 2, P, None)
        return refused(ep, rc, "overlap")
    for ts, hs, want in ((128, 0, True), (0, 64, True), (127, 64, True), (128, 63, True), (64, 64, True), (64, 319, True),
                         (big, big, True), (64, big, False), (big, 64, False), (128, 64, False), (64, 320, False),
                         (65, 400, False)):
        assert overlap(ts=ts, hs=hs) == want, (ts, hs)
    assert not overlap(tokens=1, ts=0) and not overlap(tokens=0, ts=0) and overlap(tokens=1, ts=0, hs=63)
    one = cache(ep, heads=1, device=NOWHERE)
    assert not overlap(one, n=1, ts=64, hs=0) and overlap(one, n=1, ts=63, hs=0)
    h = heads(ep, device=NOWHERE)
    for other, want in ((h, True), (heads(ep, data=P + 4096, device=NOWHERE), False)):
        rc = L.ep_cache_read((ep.EpCache * 2)(c, c), (ep.EpHeads * 2)(h, other), 2, P, 4, 4, 2, P, None)
        assert refused(ep, rc, "outputs are one") == want
