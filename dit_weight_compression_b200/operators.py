"""Microscaled 4-bit floating point and the quantised key/value cache: Python binding.

Like the codec's binding, this only marshals arguments for ``libentropack.so``; formats, layouts
and roundings are defined in ``include/entropack.h``.  All tensors are CUDA tensors of one device,
and every call is asynchronous on the current stream of that device (or on ``stream``).  A ``stream`` is
a torch stream, which holds on to the call's tensors until it is done with them, or a cudaStream_t (a number,
or in an ExternalStream): then it is the caller who keeps the call's tensors until the work is done.  For
example::

    w4 = ep.fp4_quantize(w, "nvfp4")              # or ep.decompress_fp4(blob, "nvfp4")
    y = ep.fp4_matmul(ep.fp4_quantize(x, "nvfp4"), w4, bias=bias)      # x @ w.T + bias

    cache = ep.KVCache(n_pages, page_size, heads, head_dim, "fp8")
    ep.cache_write(cache, k, v, slots)            # k, v: tokens x heads x head_dim
    k, v = ep.cache_read(cache, page_table, cu_seqlens, total=n)

They serve inference: no gradients flow through them.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import (FP8_E4M3, INT8, MXFP4, NVFP4, _TORCH_TO_EP, _check, _stream_handle, CompressedTensor, EpCache,
               EpFP4Tensor, EpHeads, EpTensor, lib, tensor_view)

FORMATS = {"mxfp4": MXFP4, "nvfp4": NVFP4}
CACHE_FORMATS = {"fp8": FP8_E4M3, "int8": INT8, **FORMATS}
BLOCK = {"mxfp4": 32, "nvfp4": 16}
SCALE_FLOATS = 1024  # EP_FP4_SCALE_FLOATS


def _format(name: str, known: dict) -> int:
    if name not in known:
        raise ValueError(f"format must be one of {', '.join(known)}")
    return known[name]


# The current stream's handle without a Stream object around it (3 us of a small call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda d: torch.cuda.current_stream(d).cuda_stream)


class _Here:
    """Stands for a context that changes nothing."""

    def __enter__(self):
        pass

    def __exit__(self, *a):
        pass


_HERE = _Here()
_current_device = torch.cuda.current_device


def _on(device: torch.device, stream, *used):
    """(context in which `device` is current and temporaries belong to the call's stream, its handle).
    `used`: the tensors of the call, whose memory a torch stream given by hand then holds on to.  One
    that is not torch's own holds on to nothing: the allocator would use its handle when a tensor is freed,
    which may be long after the caller has destroyed it."""
    index = device.index
    if stream is None:
        return (_HERE if index == _current_device() else torch.cuda.device(device)), _raw_stream(index)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device) if int(stream) else torch.cuda.default_stream(device)
    if not isinstance(stream, torch.cuda.ExternalStream):
        for t in used:
            if t is not None and t.is_cuda:
                t.record_stream(stream)
    return torch.cuda.stream(stream), stream.cuda_stream


def _view(t: torch.Tensor) -> EpTensor:
    """tensor_view without its repeated look-ups: these calls are a few microseconds long."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or t.dtype not in _TORCH_TO_EP or (stride[1] != 1 and shape[1] > 1):
        return tensor_view(t)  # raises
    rows, cols = shape
    return EpTensor(t.data_ptr(), t.get_device(), _TORCH_TO_EP[t.dtype], rows, cols,
                    stride[0] if rows > 1 else cols)  # rows that overlap are refused by the library


def _cuda(t: torch.Tensor, what: str, device: torch.device | None = None) -> torch.Tensor:
    if not t.is_cuda or (device is not None and t.device != device):
        raise ValueError(f"{what} must be on {device or 'a CUDA device'}")
    return t


@functools.lru_cache(maxsize=4096)
def _geometry(rows: int, cols: int, format: str):
    """(C format, bytes of a row, scale tiles, where the tensor scale and the elements start, all bytes)."""
    fmt = _format(format, FORMATS)
    if not (0 <= rows < 2 ** 31 - 256 and 0 <= cols <= 2 ** 30):
        raise ValueError("FP4Tensor: size out of range")
    row_bytes = 16 * (-(-cols // 32))
    tiles = (-(-rows // 128), -(-(-(-cols // BLOCK[format])) // 4))
    n = 512 * tiles[0] * tiles[1]
    return fmt, row_bytes, tiles, (n, n + 4 * SCALE_FLOATS), n + 4 * SCALE_FLOATS + rows * row_bytes


class FP4Tensor:
    """A rows x cols matrix in microscaled 4-bit floating point: ``data`` (uint8, rows x row bytes),
    ``scales`` (uint8, the tiled layout) and ``tensor_scale`` (one float32), views of one buffer."""

    __slots__ = ("format", "shape", "device", "view", "_ref", "_buffer", "_row_bytes", "_scale_tiles", "_at")

    def __init__(self, shape, format: str, device=None):
        rows, cols = shape
        # the scales first (whole 512-byte tiles), then the tensor scale and its work space, the elements
        fmt, self._row_bytes, self._scale_tiles, self._at, size = _geometry(rows, cols, format)
        self.format, self.shape = format, (rows, cols)
        self._buffer = buffer = torch.empty(size, dtype=torch.uint8, device="cuda" if device is None else device)
        self.device = buffer.device
        p = buffer.data_ptr()
        self.view = EpFP4Tensor(p + self._at[1], p, p + self._at[0], self.device.index, fmt, rows, cols)
        self._ref = ctypes.byref(self.view)

    @property
    def data(self) -> torch.Tensor:
        return self._buffer[self._at[1]:].view(self.shape[0], self._row_bytes)

    @property
    def scales(self) -> torch.Tensor:
        return self._buffer[:self._at[0]]

    @property
    def tensor_scale(self) -> torch.Tensor:
        return self._buffer.narrow(0, self._at[0], 4).view(torch.float32)

    @property
    def nbytes(self) -> int:
        """Bytes of the elements and scales, paddings included."""
        return self._at[0] + 4 + self.shape[0] * self._row_bytes

    def scale_rows(self) -> torch.Tensor:
        """The scale bytes in rows: rows x ceil(cols / block), uint8."""
        i, j = self._scale_tiles
        t = self.scales.view(i, j, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(i * 128, j * 4)
        return t[:self.shape[0], :-(-self.shape[1] // BLOCK[self.format])].contiguous()

    @classmethod
    def from_rows(cls, data: torch.Tensor, scale_rows: torch.Tensor, tensor_scale: torch.Tensor, shape,
                  format: str) -> "FP4Tensor":
        """A copy of packed rows (uint8, rows x (16 * ceil(cols / 32)); the even column in the low half of a
        byte; elements past `cols` are cleared), scale bytes in rows (uint8, rows x ceil(cols / block))
        and one float32 tensor scale, such as another program made."""
        dev = _cuda(data, "data").device
        with torch.cuda.device(dev):
            t = cls(shape, format, dev)
            rows, cols = t.shape
            blocks = -(-cols // BLOCK[format])
            if data.dtype != torch.uint8 or tuple(data.shape) != (rows, t._row_bytes):
                raise ValueError(f"from_rows: data must be uint8 of shape {(rows, t._row_bytes)}")
            if scale_rows.dtype != torch.uint8 or tuple(scale_rows.shape) != (rows, blocks):
                raise ValueError(f"from_rows: scale_rows must be uint8 of shape {(rows, blocks)}")
            if tensor_scale.dtype != torch.float32 or tensor_scale.numel() != 1:
                raise ValueError("from_rows: tensor_scale must be one float32")
            t.data.copy_(data)
            if cols % 32:
                t.data[:, (cols + 1) // 2:] = 0
                if cols % 2:
                    t.data[:, cols // 2] &= 15
            i, j = t._scale_tiles
            if i and j:  # a matrix without rows or columns has no scales
                s = torch.zeros(i * 128, j * 4, dtype=torch.uint8, device=dev)
                s[:rows, :blocks] = scale_rows if format == "mxfp4" else scale_rows & 0x7F  # E4M3 scales have no sign
                # four scales of a row at a time: tiles of 32 x 4 words
                t.scales.view(torch.int32).view(i, j, 32, 4).copy_(s.view(torch.int32).view(i, 4, 32, j).permute(0, 3, 2, 1))
            t.tensor_scale.copy_(tensor_scale.reshape(1))
        return t


def _made(shape, format, device, out, what) -> FP4Tensor:
    if out is None:
        out = FP4Tensor(shape, format, device)
    elif out.format != format or out.shape != tuple(shape) or out.device != device:
        raise ValueError(f"{what}: out must be a {format} tensor of shape {tuple(shape)} on {device}")
    return out


def fp4_quantize(x: torch.Tensor, format: str = "nvfp4", *, tensor_scale: float | None = None,
                 out: FP4Tensor | None = None, stream=None) -> FP4Tensor:
    """Quantise a 2-D CUDA tensor (bf16, fp16 or fp32; columns contiguous) with ep_fp4_quantize.
    `tensor_scale` (nvfp4 only): a power of two, else it is taken from the data in a pass of its own."""
    _cuda(x, "x")
    view = _view(x)
    ctx, st = _on(x.device, stream, x, out and out._buffer)
    with ctx:
        out = _made(x.shape, format, x.device, out, "fp4_quantize")
        _check(lib().ep_fp4_quantize(ctypes.byref(view), out._ref, 0.0 if tensor_scale is None else float(tensor_scale), st),
               "ep_fp4_quantize")
    return out


def _dense(shape, dtype, device, out=None):
    """(`out`, or a new tensor, and its C view)."""
    if out is not None:
        return out, _view(out)
    if dtype not in _TORCH_TO_EP:
        raise TypeError(f"unsupported dtype {dtype}")
    rows, cols = shape
    out = torch.empty(rows, cols, dtype=dtype, device=device)
    return out, EpTensor(out.data_ptr(), device.index, _TORCH_TO_EP[dtype], rows, cols, cols)


def fp4_dequantize(x: FP4Tensor, *, dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    """The values of a 4-bit tensor as a bf16, fp16 or fp32 tensor (ep_fp4_dequantize)."""
    ctx, st = _on(x.device, stream, x._buffer, out)
    with ctx:
        out, view = _dense(x.shape, dtype, x.device, out)
        _check(lib().ep_fp4_dequantize(x._ref, ctypes.byref(view), st), "ep_fp4_dequantize")
    return out


def decompress_fp4(compressed: CompressedTensor, format: str = "nvfp4", *, tensor_scale: float | None = None,
                   dtype: torch.dtype = torch.bfloat16, out: FP4Tensor | None = None, device=None, stream=None) -> FP4Tensor:
    """Decompress a blob into the 4-bit container (ep_decompress_fp4): the blob restored in `dtype`,
    in a buffer of this call, and quantised as by fp4_quantize."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    if out is not None:
        dev = out.device
    elif dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    ctx, st = _on(dev, stream, out and out._buffer)
    with ctx:
        out = _made(compressed.shape, format, dev, out, "decompress_fp4")
        work, view = _dense(compressed.shape, dtype, dev)
        _check(lib().ep_decompress_fp4(compressed.handle, out._ref, 0.0 if tensor_scale is None else float(tensor_scale),
                                       ctypes.byref(view), st), "ep_decompress_fp4")
    return out


def fp4_matmul(a: FP4Tensor, b: FP4Tensor, *, bias: torch.Tensor | None = None, dtype: torch.dtype = torch.bfloat16,
               out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """a @ b.T + bias for two 4-bit tensors of one format (ep_fp4_matmul), as bf16, fp16 or fp32.
    `bias` has one element a row of b, of the output's type."""
    ctx, st = _on(a.device, stream, a._buffer, b._buffer, bias, out)
    with ctx:
        out, view = _dense((a.shape[0], b.shape[0]), dtype, a.device, out)
        p = None
        if bias is not None:
            _cuda(bias, "bias", a.device)
            if bias.dtype != out.dtype or tuple(bias.shape) != (b.shape[0],) or not bias.is_contiguous():
                raise ValueError("fp4_matmul: bias must be a contiguous vector of the output's type, one element a row of b")
            p = bias.data_ptr()
        _check(lib().ep_fp4_matmul(a._ref, b._ref, p, ctypes.byref(view), st), "ep_fp4_matmul")
    return out


class KVCache:
    """A paged cache of keys and values, quantised as it is written.  ``k`` and ``v`` hold the payload
    (n_pages x page_size x heads x row: float8_e4m3fn, int8, or packed uint8), ``k_scales`` and
    ``v_scales`` the scales (float32, one a row; uint8, one a block for the 4-bit formats).  It saves
    memory, not traffic: ``cache_read`` restores dense rows.  ``nvfp4`` rows have no tensor scale: blocks
    up to 0.0059 become zeros and values above 2688 are clamped; the other formats have no such bounds."""

    def __init__(self, n_pages: int, page_size: int, heads: int, head_dim: int, format: str = "fp8", device=None):
        _format(format, CACHE_FORMATS)
        dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        lead = (n_pages, page_size, heads)
        row, dt, scales, sdt = self._row(head_dim, format)

        def pool():
            return (torch.zeros(*lead, row, dtype=torch.uint8, device=dev).view(dt),
                    torch.zeros(*lead, scales, dtype=sdt, device=dev))
        self._set(*pool(), *pool(), format, head_dim)

    @staticmethod
    def _row(head_dim, format):
        if format in FORMATS:
            return 16 * (-(-head_dim // 32)), torch.uint8, -(-head_dim // BLOCK[format]), torch.uint8
        return head_dim, torch.float8_e4m3fn if format == "fp8" else torch.int8, 1, torch.float32

    @classmethod
    def from_tensors(cls, k, k_scales, v, v_scales, format: str, head_dim: int) -> "KVCache":
        """A cache over existing pools (shared, not copied) of the layout described above."""
        _format(format, CACHE_FORMATS)
        c = cls.__new__(cls)
        c._set(k, k_scales, v, v_scales, format, head_dim)
        return c

    def _set(self, k, k_scales, v, v_scales, format, head_dim):
        self._pools = (k, k_scales, v, v_scales)  # kept for as long as the pointers in _views
        self.format, self.head_dim, self.device = format, int(head_dim), k.device
        row, dt, scales, sdt = self._row(self.head_dim, format)
        if k.dim() != 4:
            raise ValueError("KVCache: pools are n_pages x page_size x heads x row")
        self.n_pages, self.page_size, self.heads = k.shape[:3]
        for t, last, want in ((k, row, dt), (v, row, dt), (k_scales, scales, sdt), (v_scales, scales, sdt)):
            if tuple(t.shape) != (self.n_pages, self.page_size, self.heads, last) or t.dtype != want or not t.is_contiguous():
                raise ValueError(f"KVCache: expected a contiguous {want} pool of shape "
                                 f"{(self.n_pages, self.page_size, self.heads, last)}")
            _cuda(t, "every pool", k.device)
        self._views = (EpCache * 2)(*[EpCache(p.data_ptr(), s.data_ptr(), k.device.index, CACHE_FORMATS[format], self.n_pages,
                                              self.page_size, self.heads, self.head_dim)
                                      for p, s in ((k, k_scales), (v, v_scales))])

    k = property(lambda self: self._pools[0])
    k_scales = property(lambda self: self._pools[1])
    v = property(lambda self: self._pools[2])
    v_scales = property(lambda self: self._pools[3])

    @property
    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in self._pools)


_TwoHeads = EpHeads * 2


def _heads(t: torch.Tensor, what: str) -> EpHeads:
    shape, stride = t.shape, t.stride()
    if len(shape) != 3:
        raise ValueError(f"{what} must be tokens x heads x head_dim")
    if t.dtype not in _TORCH_TO_EP:
        raise TypeError(f"unsupported dtype {t.dtype}")
    if stride[2] != 1 and shape[2] > 1:
        raise ValueError(f"{what}: the elements of a head must be contiguous")
    return EpHeads(t.data_ptr(), t.get_device(), _TORCH_TO_EP[t.dtype], *shape, stride[0], stride[1])


def cache_write(cache: KVCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, *, stream=None) -> None:
    """Quantise k and v (tokens x heads x head_dim; bf16, fp16 or fp32; any token and head strides) into
    the slots (int64, page * page_size + offset) of a cache.  Negative slots and slots past the last
    page are skipped; of tokens that name one slot the last is kept (ep_cache_write)."""
    for t, what in ((k, "k"), (v, "v"), (slots, "slots")):
        _cuda(t, what, cache.device)
    if slots.dtype != torch.int64 or slots.dim() != 1 or slots.shape[0] != k.shape[0] or not slots.is_contiguous():
        raise ValueError("cache_write: slots must be a contiguous int64 vector with one entry a token")
    views = _TwoHeads(_heads(k, "k"), _heads(v, "v"))
    ctx, st = _on(cache.device, stream, k, v, slots, *cache._pools)
    with ctx:
        _check(lib().ep_cache_write(cache._views, views, 2, slots.data_ptr(), st), "ep_cache_write")


def cache_read(cache: KVCache, page_table: torch.Tensor, cu_seqlens: torch.Tensor, *, total: int | None = None,
               dtype: torch.dtype = torch.bfloat16, out: tuple | None = None, stream=None) -> tuple:
    """Read sequences back as (k, v), tokens x heads x head_dim.  `page_table` (int32, sequences x pages)
    names the pages of each sequence, `cu_seqlens` (int32, sequences + 1) where each starts among the
    tokens; `total` is the number of tokens, or `out` the pair of tensors to fill.  Tokens past
    cu_seqlens[-1] are left as they are: in tensors that the call makes they are not set.  Positions without
    a valid page read as zeros."""
    for t, what in ((page_table, "page_table"), (cu_seqlens, "cu_seqlens")):
        _cuda(t, what, cache.device)
        if t.dtype != torch.int32:
            raise ValueError(f"cache_read: {what} must be int32")
    if page_table.dim() != 2 or (page_table.shape[1] > 1 and page_table.stride(1) != 1):
        raise ValueError("cache_read: page_table must be sequences x pages with contiguous rows")
    n = page_table.shape[0]
    if tuple(cu_seqlens.shape) != (n + 1,) or not cu_seqlens.is_contiguous():
        raise ValueError("cache_read: cu_seqlens must be a contiguous vector of one more entry than there are sequences")
    if out is None and total is None:
        raise ValueError("cache_read: give total or out")
    ctx, st = _on(cache.device, stream, page_table, cu_seqlens, *cache._pools, *(out or ()))
    with ctx:
        if out is None:
            rows, h, d, dev = int(total), cache.heads, cache.head_dim, cache.device
            out = (torch.empty(rows, h, d, dtype=dtype, device=dev), torch.empty(rows, h, d, dtype=dtype, device=dev))
        for t in out:
            _cuda(t, "out", cache.device)
        views = _TwoHeads(_heads(out[0], "out[0]"), _heads(out[1], "out[1]"))
        _check(lib().ep_cache_read(cache._views, views, 2, page_table.data_ptr(),
                                   page_table.stride(0) if n > 1 else page_table.shape[1],
                                   page_table.shape[1], n, cu_seqlens.data_ptr(), st), "ep_cache_read")
    return out


def op_status(stream=None) -> None:
    """Raise EPError if a 4-bit product on the current device gave up waiting since the last call."""
    _check(lib().ep_op_status(_stream_handle(stream)), "ep_op_status")
