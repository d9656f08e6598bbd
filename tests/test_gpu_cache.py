"""The quantised key/value cache on the GPU against the 64-bit definitions (microscale_ref.py), bit for bit:
payloads, scales and what is read back are all fixed by the formats (int8 values are one fp32 product and one
rounding to the output's type)."""
import numpy as np
import pytest
import torch

import microscale_ref as R

pytestmark = pytest.mark.gpu
FMTS = ["fp8", "int8", "mxfp4", "nvfp4"]
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


def tokens(n, heads, dim, dtype, seed):
    x = torch.randn(n, heads, dim, generator=gen(seed), device="cuda")
    x *= torch.exp(6 * (torch.rand(n, heads, 1, generator=gen(seed + 1), device="cuda") - 0.5))
    return x.to(dtype)


def reference(x, fmt):
    """(payload as the pool holds it, scales as the pool holds them, values in fp32) of rows x."""
    n, h, d = x.shape
    y = x.double().cpu().numpy().reshape(n * h, d)
    if fmt in R.BLOCK:
        el, byte, _ = R.quantize(y, fmt, 1.0)
        v = torch.from_numpy(R.values(el, byte, 1.0, d, fmt)).float()
        return el.reshape(n, h, -1), byte.reshape(n, h, -1), v.view(n, h, d)
    p, s = R.cache_row(y, fmt)
    v = torch.from_numpy(p).float() * torch.from_numpy(s).float()[:, None]
    return p.reshape(n, h, d), s.reshape(n, h, 1), v.view(n, h, d)


def payload(pool, fmt, dim):
    """The payload of a pool's slots as numbers, and its scales."""
    p = pool.flatten(0, 1)
    if fmt in R.BLOCK:
        a = p.cpu().numpy()
        return R.unpack(a.reshape(-1, a.shape[-1])).reshape(*a.shape[:2], -1)
    return p.double().cpu().numpy()


def same(a, b):
    return np.array_equal(a, b, equal_nan=True)


def check_slots(cache, slots, k, v):
    """The named slots hold k and v; every other slot is as a new cache's."""
    live = torch.tensor([i for i in range(len(slots)) if slots[i] >= 0])
    at = np.array([slots[i] for i in live])
    for pool, scales, x in ((cache.k, cache.k_scales, k), (cache.v, cache.v_scales, v)):
        p, s, _ = reference(x[live.to(x.device)], cache.format)
        got, sc = payload(pool, cache.format, cache.head_dim), scales.flatten(0, 1).cpu().numpy()
        w = min(p.shape[-1], got.shape[-1])
        assert same(got[at][..., :w], p[..., :w]) and not np.any(got[at][..., w:])
        assert same(sc[at].astype(np.float64), s.astype(np.float64))
        rest = np.ones(got.shape[0], bool)
        rest[at] = False
        assert not got[rest].any() and not sc[rest].any()


GEOMETRY = [(1, 1, 1, 16), (3, 2, 33, 8), (5, 3, 80, 16), (40, 8, 128, 64), (17, 1, 256, 1), (9, 5, 72, 128), (6, 2, 300, 16),
            (4, 1, 1024, 4), (300, 2, 64, 16), (7, 16, 40, 32), (5, 2, 7, 16)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,heads,dim,page", GEOMETRY)
def test_write_then_read(ep, fmt, dtype, n, heads, dim, page):
    pages = -(-n // page) + 3
    cache = ep.KVCache(pages, page, heads, dim, fmt)
    k, v = tokens(n, heads, dim, dtype, 1), tokens(n, heads, dim, dtype, 2)
    slots = torch.randperm(pages * page, generator=gen(3), device="cuda")[:n]
    ep.cache_write(cache, k, v, slots)
    check_slots(cache, slots.tolist(), k, v)
    # the whole pool as one sequence, then by slot
    table = torch.arange(pages, device="cuda", dtype=torch.int32).view(1, -1)
    cu = torch.tensor([0, pages * page], device="cuda", dtype=torch.int32)
    for out_dtype in DTYPES:
        got = ep.cache_read(cache, table, cu, total=pages * page, dtype=out_dtype)
        for g, x in zip(got, (k, v)):
            assert torch.equal(g[slots].cpu(), reference(x, fmt)[2].to(out_dtype))


@pytest.mark.parametrize("fmt", FMTS)
def test_strided_sources(ep, fmt):
    """Keys and values as windows of a fused projection, heads before tokens, and a shared head."""
    n, heads, dim = 21, 4, 64
    qkv = tokens(n, 3 * heads, dim, torch.bfloat16, 4)
    for k, v in ((qkv[:, heads:2 * heads], qkv[:, 2 * heads:]),
                 (qkv[:, :heads].transpose(0, 1).contiguous().transpose(0, 1), qkv[:, heads:2 * heads]),
                 (qkv[:, :1].expand(n, heads, dim), qkv[:1, :heads].expand(n, heads, dim)),
                 (qkv.view(-1)[1:1 + n * heads * dim].view(n, heads, dim), qkv[:, :heads])):
        cache = ep.KVCache(3, 16, heads, dim, fmt)
        slots = torch.arange(5, 5 + n, device="cuda")
        ep.cache_write(cache, k, v, slots)
        check_slots(cache, slots.tolist(), k, v)


@pytest.mark.parametrize("fmt", FMTS)
def test_special_rows(ep, fmt):
    """Rows of zeros, tiny and huge values, ties, NaN and infinities."""
    x = tokens(12, 1, 64, torch.float32, 5)
    x[0] = 0
    x[1] = 1e-40
    x[2] = torch.linspace(-3e38, 3e38, 64, device="cuda")
    x[3] = torch.arange(64, device="cuda") + 0.5
    x[3, 0, 0] = 127.0
    x[4] = 448.0
    x[5] = 2.0 ** -103
    x[6, 0, 3] = float("nan")
    x[7, 0, 40] = float("-inf")
    x[8] = torch.exp2(-torch.arange(64, device="cuda").float())
    cache = ep.KVCache(1, 16, 1, 64, fmt)
    slots = torch.arange(12, device="cuda")
    ep.cache_write(cache, x, x, slots)
    check_slots(cache, slots.tolist(), x, x)
    got = ep.cache_read(cache, torch.zeros(1, 1, device="cuda", dtype=torch.int32),
                        torch.tensor([0, 12], device="cuda", dtype=torch.int32), total=12, dtype=torch.float32)[0]
    assert same(got.cpu().numpy(), reference(x, fmt)[2].numpy())


def test_int8_borders(ep):
    """Quotients on and next to half-integers: values k + 1/2 steps of scales that are no power of two, and
    the floats on either side."""
    g = gen(6)
    top = 1 + torch.rand(512, 1, generator=g, device="cuda")
    s = (top / 127).double()
    h = torch.arange(63, device="cuda").double() + 0.5
    mid = (h * s).float()
    x = torch.cat((top, mid, torch.nextafter(mid, torch.zeros_like(mid)), torch.nextafter(mid, 2 * mid)), 1)[:, None]
    cache = ep.KVCache(4, 128, 1, x.shape[2], "int8")
    slots = torch.arange(512, device="cuda")
    ep.cache_write(cache, x, -x, slots)
    check_slots(cache, slots.tolist(), x, -x)


@pytest.mark.parametrize("n", [3, 600, 1024, 1025, 9000, 70000])
def test_skipped_and_repeated_slots(ep, n):
    """Padding (-1), slots past the last page, and slots named more than once: the last token wins, within a
    launch and across the launches of a long call."""
    heads, dim, pages, page = 2, 64, 40, 16
    k, v = tokens(n, heads, dim, torch.bfloat16, 7), tokens(n, heads, dim, torch.bfloat16, 8)
    slots = torch.randint(-3, pages * page + 3, (n,), generator=gen(9), device="cuda")
    if n == 3:
        slots[:] = torch.tensor([5, 5, -1], device="cuda")
    cache = ep.KVCache(pages, page, heads, dim, "fp8")
    ep.cache_write(cache, k, v, slots)
    last = {}
    for i, s in enumerate(slots.tolist()):
        if 0 <= s < pages * page:
            last[s] = i
    want = [-1] * n
    for s, i in last.items():
        want[i] = s
    check_slots(cache, want, k, v)


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
@pytest.mark.parametrize("n_seqs", [1, 6, 1500])
def test_read_ragged(ep, fmt, n_seqs):
    """Lengths from zero, pages that end inside a sequence, pages not handed out or past the pool (zeros), and
    tokens behind the last sequence (left as they were)."""
    heads, dim, page, pages = 2, 72, 8, 64
    cache = ep.KVCache(pages, page, heads, dim, fmt)
    n = pages * page
    k, v = tokens(n, heads, dim, torch.float16, 10), tokens(n, heads, dim, torch.float16, 11)
    ep.cache_write(cache, k, v, torch.arange(n, device="cuda"))
    g = gen(12)
    lens = torch.randint(0, 40, (n_seqs,), generator=g, device="cuda")
    lens[0] = 37
    if n_seqs > 2:
        lens[1], lens[-1] = 0, 1
    wide = 4  # a table narrower than the longest sequence needs
    table = torch.randint(-1, pages + 1, (n_seqs, wide + 1), generator=g, device="cuda", dtype=torch.int32)[:, :wide]
    cu = torch.nn.functional.pad(lens.cumsum(0), (1, 0)).to(torch.int32)
    total = int(cu[-1])
    out = [torch.full((total + 5, heads, dim), 3.0, dtype=torch.float32, device="cuda") for _ in range(2)]
    ep.cache_read(cache, table, cu, out=tuple(out))
    seq = torch.repeat_interleave(torch.arange(n_seqs, device="cuda"), lens)
    pos = torch.arange(total, device="cuda") - cu[seq]
    p = pos // page
    id_ = torch.where(p < wide, table[seq, p.clamp(max=wide - 1)].long(), -1)
    good = (id_ >= 0) & (id_ < pages)
    slot = torch.where(good, id_ * page + pos % page, 0).cpu()
    for o, x in zip(out, (k, v)):
        want = reference(x, fmt)[2][slot]
        want[~good.cpu()] = 0
        assert torch.equal(o[:total].cpu(), want)
        assert bool((o[total:] == 3).all())


def test_read_strided_out_and_cut(ep):
    """Outputs as windows of a wider tensor; sequences past the output's tokens are cut off."""
    cache = ep.KVCache(4, 16, 2, 64, "int8")
    k, v = tokens(64, 2, 64, torch.bfloat16, 13), tokens(64, 2, 64, torch.bfloat16, 14)
    ep.cache_write(cache, k, v, torch.arange(64, device="cuda"))
    table = torch.tensor([[0, 1, 2, 3]], device="cuda", dtype=torch.int32)
    cu = torch.tensor([0, 64], device="cuda", dtype=torch.int32)
    for off in (0, 3):
        both = torch.full((50, 4, 70), 5.0, dtype=torch.bfloat16, device="cuda")
        ep.cache_read(cache, table, cu, out=(both[:, :2, off:off + 64], both[:, 2:, off:off + 64]))
        for h, x in ((0, k), (2, v)):
            assert torch.equal(both[:, h:h + 2, off:off + 64].cpu(), reference(x, "int8")[2][:50].bfloat16())
        assert bool((both[:, :, :off] == 5).all()) and bool((both[:, :, off + 64:] == 5).all())


def test_nothing_to_do(ep):
    cache = ep.KVCache(2, 16, 2, 64, "fp8")
    e = torch.zeros(0, 2, 64, device="cuda")
    ep.cache_write(cache, e, e, torch.zeros(0, dtype=torch.int64, device="cuda"))
    table = torch.zeros(0, 3, dtype=torch.int32, device="cuda")
    out = torch.full((4, 2, 64), 2.0, device="cuda")
    ep.cache_read(cache, table, torch.zeros(1, dtype=torch.int32, device="cuda"), out=(out, out.clone()))
    assert bool((out == 2).all())
    k, _ = ep.cache_read(cache, table, torch.zeros(1, dtype=torch.int32, device="cuda"), total=0)
    assert k.shape == (0, 2, 64)
    zero_pages = ep.KVCache(0, 16, 2, 64, "fp8")
    x = tokens(3, 2, 64, torch.float32, 1)
    ep.cache_write(zero_pages, x, x, torch.arange(3, device="cuda"))


def test_offsets_past_32_bits(ep):
    """A pool of 5 GB of keys: the last page."""
    pages, page, heads, dim = 5000, 128, 32, 256
    cache = ep.KVCache(pages, page, heads, dim, "fp8")
    x = tokens(4, heads, dim, torch.bfloat16, 15)
    first = pages * page - 4
    ep.cache_write(cache, x, x, torch.arange(first, first + 4, device="cuda"))
    table = torch.tensor([[pages - 1]], device="cuda", dtype=torch.int32)
    k, v = ep.cache_read(cache, table, torch.tensor([0, page], device="cuda", dtype=torch.int32), total=page)
    want = reference(x, "fp8")[2].bfloat16()
    assert torch.equal(k[-4:].cpu(), want) and torch.equal(v[-4:].cpu(), want) and not k[:-4].any()


def test_decoding_loop_in_a_graph(ep):
    """Steps that append one token a sequence and read the histories, eager and as a replayed graph, with a
    4-bit linear layer before the cache."""
    seqs, heads, dim, page = 5, 2, 64, 8
    w = ep.fp4_quantize(torch.randn(2 * heads * dim, 128, generator=gen(16), device="cuda").bfloat16(), "nvfp4")
    table = torch.arange(seqs * 4, device="cuda", dtype=torch.int32).view(seqs, 4)
    steps = [torch.randn(seqs, 128, generator=gen(20 + i), device="cuda").bfloat16() for i in range(20)]

    def step(cache, x, slots, cu, out):
        kv = ep.fp4_matmul(ep.fp4_quantize(x, "nvfp4"), w).view(seqs, 2 * heads, dim)
        ep.cache_write(cache, kv[:, :heads], kv[:, heads:], slots)
        ep.cache_read(cache, table, cu, out=out)

    def at(i):
        pos = torch.full((seqs,), i, device="cuda")
        slots = (table[:, i // page].long() * page + i % page)
        return slots, (torch.arange(seqs + 1, device="cuda") * (i + 1)).to(torch.int32), pos

    results = []
    for captured in (False, True):
        cache = ep.KVCache(seqs * 4, page, heads, dim, "fp8")
        out = tuple(torch.zeros(seqs * 20, heads, dim, device="cuda", dtype=torch.bfloat16) for _ in range(2))
        x, slots, cu = steps[0].clone(), torch.zeros(seqs, dtype=torch.int64, device="cuda"), torch.zeros(seqs + 1, dtype=torch.int32, device="cuda")
        graph = None
        if captured:
            slots.fill_(-1)
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step(cache, x, slots, cu, out)
        seen = []
        for i in range(20):
            x.copy_(steps[i])
            s, c, _ = at(i)
            slots.copy_(s)
            cu.copy_(c)
            if captured:
                graph.replay()
            else:
                step(cache, x, slots, cu, out)
            seen.append([o[:seqs * (i + 1)].clone() for o in out])
        results.append(seen)
    for a, b in zip(*results):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_python_argument_errors(ep):
    cache = ep.KVCache(2, 16, 2, 64, "fp8")
    x = tokens(3, 2, 64, torch.bfloat16, 1)
    with pytest.raises(ValueError):
        ep.cache_write(cache, x, x, torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        ep.cache_write(cache, x, x, torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ep.EPError):
        ep.cache_write(cache, x[:, :1], x[:, :1], torch.zeros(3, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        ep.cache_write(cache, x.cpu(), x, torch.zeros(3, dtype=torch.int64, device="cuda"))
    t = torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        ep.cache_read(cache, t, torch.zeros(3, dtype=torch.int32, device="cuda"), total=1)
    with pytest.raises(ValueError):
        ep.cache_read(cache, t, torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ep.EPError):  # rows of the table that overlap
        ep.cache_read(cache, t.expand(3, 2), torch.zeros(4, dtype=torch.int32, device="cuda"), total=1)
    with pytest.raises(ValueError):
        ep.KVCache.from_tensors(cache.k, cache.v_scales, cache.v, cache.v_scales[:1], "fp8", 64)
    with pytest.raises(ep.EPError):  # outputs of two types, and of two lengths
        ep.cache_read(cache, t, torch.zeros(2, dtype=torch.int32, device="cuda"), out=(x, x.float()))
    with pytest.raises(ep.EPError):
        ep.cache_read(cache, t, torch.zeros(2, dtype=torch.int32, device="cuda"), out=(x, x[:2]))
