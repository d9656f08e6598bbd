"""The quantised cache where slots repeat, and the range of its 4-bit rows, against the 64-bit definitions
(microscale_ref.py)."""
import numpy as np
import pytest
import torch

from test_gpu_cache import DTYPES, FMTS, check_slots, gen, payload, reference, same, tokens

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dit_weight_compression_b200 import build
    build.build()
    import dit_weight_compression_b200 as ep
    return ep


def kept(slots, n_slots):
    """The slot of each token that is the last to name it, -1 for the others."""
    last = {s: i for i, s in enumerate(slots) if 0 <= s < n_slots}
    want = [-1] * len(slots)
    for s, i in last.items():
        want[i] = s
    return want


def dummy_slots(n, pages, page, share, seed):
    """n tokens in slots of their own, but a share of them, spread over the call, in slot 0."""
    slots = torch.randperm(pages * page - 1, generator=gen(seed), device="cuda")[:n] + 1
    slots[torch.rand(n, generator=gen(seed + 1), device="cuda") < share] = 0
    return slots


@pytest.mark.parametrize("share", [0.25, 0.9, 1.0])
@pytest.mark.parametrize("n", [1500, 20000])
def test_many_tokens_of_one_slot(ep, n, share):
    """Padding that names one valid slot: its last token is kept, whole, and the others are as always."""
    heads, dim, page = 2, 64, 16
    pages = n // page + 2
    cache = ep.KVCache(pages, page, heads, dim, "fp8")
    k, v = tokens(n, heads, dim, torch.bfloat16, 31), tokens(n, heads, dim, torch.bfloat16, 32)
    slots = dummy_slots(n, pages, page, share, 33)
    ep.cache_write(cache, k, v, slots)
    check_slots(cache, kept(slots.tolist(), pages * page), k, v)


def test_many_tokens_of_one_slot_take_no_longer(ep):
    """A long call with half its tokens in one slot takes about as long as one with a slot for each (twice, and
    the launches' own 10 us, are allowed)."""
    n, heads, dim, page = 65536, 2, 64, 64
    pages = n // page + 1
    cache = ep.KVCache(pages, page, heads, dim, "fp8")
    k = tokens(n, heads, dim, torch.bfloat16, 34)

    def best(slots):
        times = []
        for _ in range(10):
            e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
            torch.cuda.synchronize()
            e[0].record()
            ep.cache_write(cache, k, k, slots)
            e[1].record()
            torch.cuda.synchronize()
            times.append(e[0].elapsed_time(e[1]) * 1000)
        return min(times)

    apart, one = best(dummy_slots(n, pages, page, 0.0, 35)), best(dummy_slots(n, pages, page, 0.5, 35))
    print(f"{apart:.1f} us apart, {one:.1f} us with half the tokens in one slot")
    assert one <= 2 * apart + 10, (apart, one)


SHAPES = [(2, 64, 0), (3, 160, 0), (2, 72, 0), (2, 40, 1), (1, 300, 0), (2, 33, 0)]  # heads, head size, offset


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("heads,dim,off", SHAPES)
def test_repeated_slots_of_long_calls(ep, fmt, dtype, heads, dim, off):
    """More tokens than a write compares by itself, of which most are written over: every format, type, head size
    and alignment."""
    n, pages, page = 1700, 30, 16
    raw = tokens(1, 1, 2 * (n * heads * dim + 8), dtype, 41).view(-1)
    k, v = (raw[s + off:s + off + n * heads * dim].view(n, heads, dim) for s in (0, n * heads * dim + 8))
    slots = torch.randint(-2, pages * page + 2, (n,), generator=gen(42), device="cuda")
    cache = ep.KVCache(pages, page, heads, dim, fmt)
    ep.cache_write(cache, k, v, slots)
    check_slots(cache, kept(slots.tolist(), pages * page), k, v)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dims", [(192, 128), (64, 300)])
def test_repeated_slots_of_two_head_sizes(ep, fmt, dims):
    """Keys and values of different head sizes in one call of the C interface."""
    n, pages, page, heads = 1300, 20, 16, 2
    caches = [ep.KVCache(pages, page, heads, d, fmt) for d in dims]
    x = [tokens(n, heads, d, torch.bfloat16, 50 + i) for i, d in enumerate(dims)]
    slots = torch.randint(-2, pages * page + 2, (n,), generator=gen(52), device="cuda")
    views = (ep.EpCache * 2)(caches[0]._views[0], caches[1]._views[1])
    heads_ = (ep.EpHeads * 2)(*[ep.EpHeads(t.data_ptr(), 0, ep.BF16, n, heads, d, heads * d, d) for t, d in zip(x, dims)])
    rc = ep.lib().ep_cache_write(views, heads_, 2, slots.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert rc == 0, ep.lib().ep_last_error()
    want = kept(slots.tolist(), pages * page)
    live = [i for i in range(n) if want[i] >= 0]
    at = np.array([want[i] for i in live])
    for cache, pool, scales, t in ((caches[0], caches[0].k, caches[0].k_scales, x[0]), (caches[1], caches[1].v, caches[1].v_scales, x[1])):
        p, s, _ = reference(t[torch.tensor(live, device="cuda")], fmt)
        got, sc = payload(pool, fmt, cache.head_dim)[at], scales.flatten(0, 1).cpu().numpy()[at]
        w = min(p.shape[-1], got.shape[-1])
        assert same(got[..., :w], p[..., :w]) and same(sc.astype(np.float64), s.astype(np.float64))


def test_range_of_nvfp4_rows(ep):
    """NVFP4 rows have E4M3 scales and no tensor scale: a block up to 6 * 2^-10 is lost, one above 2688 is
    clamped; the other formats keep both."""
    x = torch.zeros(4, 1, 16, device="cuda")
    x[0, 0, 0], x[1, 0, 0], x[2, 0, 0], x[3, 0, 0] = 6 * 2.0 ** -10, 6 * 2.0 ** -9, 2688.0, 8192.0
    table, cu = (torch.tensor(t, dtype=torch.int32, device="cuda") for t in ([[0]], [0, 4]))
    for fmt in FMTS:
        cache = ep.KVCache(1, 4, 1, 16, fmt)
        ep.cache_write(cache, x, x, torch.arange(4, device="cuda"))
        got = ep.cache_read(cache, table, cu, total=4, dtype=torch.float32)[0][:, 0, 0].tolist()
        if fmt == "nvfp4":
            assert got == [0.0, 6 * 2.0 ** -9, 2688.0, 2688.0]
        else:
            assert all(abs(g - w) <= w / 4 for g, w in zip(got, x[:, 0, 0].tolist()))
