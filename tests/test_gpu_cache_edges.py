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
