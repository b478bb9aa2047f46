"""The append where a block keeps a scale of the caller's own, against the
oracle: values, NaN and the signs of zeros."""
import numpy as np
import pytest
import torch

from oracle import q8_oracle as Q
from q8_cases import held, random_cache

pytestmark = pytest.mark.gpu


def _kc():
    from sparse_attention_long_anchor_b200 import kascade as kc
    return kc


def _check(cache, kind, k, v, slots):
    """Appends and compares: scales, values, places of NaN, and (e4m3 has a
    negative zero) sign bits."""
    want = [x.copy() for x in held(cache, kind)]
    with np.errstate(invalid="ignore"):
        for which, x in enumerate((k, v)):
            Q.append(want[which], want[2], x.float().cpu().numpy(), list(slots), which, cache.scale_block, kind)
    _kc().q8_append(cache, k, v, torch.tensor(slots, dtype=torch.int32, device="cuda"))
    got = held(cache, kind)
    assert np.array_equal(got[2], want[2])
    for a, b in zip(got[:2], want[:2]):
        nan = np.isnan(b)
        assert np.array_equal(np.isnan(a), nan)
        assert np.array_equal(a[~nan], b[~nan])
        if kind == "e4m3":
            assert np.array_equal(np.signbit(a[~nan]), np.signbit(b[~nan]))


# (kv heads, tokens, block): runs of up to eight rows and longer ones of the form for few tokens, and the form for
# many (32 heads, more than 256 tokens), where a block is a tile of its own or one of several
FORMS = [(2, 6, 64), (2, 40, 64), (32, 300, 64), (32, 300, 8), (32, 300, 256)]


def _kept(kind, hkv, t, block, scale, dtype, spread, seed):
    """t rows behind the first half block of a cache whose scales are all
    `scale`: the first run continues that block and keeps it."""
    kc = _kc()
    d, page = 64, 256
    cache = random_cache(kc, 4, hkv, page, d, block, kind, seed)
    cache.scales.fill_(scale)
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(t, 2, hkv, d, generator=g) * spread
    x[0, 0, :, 5] = float("inf")
    x[1, :, 0, 6] = float("-inf")
    x[2, 1, 1, :3] = float("nan")
    x[3] = 0.0
    x[4, :, :, 1::2] = -0.0
    at = block // 2
    slots = [page * (1 + (at + i) // page) + (at + i) % page for i in range(t)]   # pages 1, 2, ..
    return cache, x.to(dtype).cuda(), slots


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("hkv,t,block", FORMS)
@pytest.mark.parametrize("scale", [0.3 * 2 ** 10, 0.7])
def test_infinities_under_a_scale_that_is_no_power_of_two(kind, hkv, t, block, scale):
    """Infinities saturate and NaN stays itself, as under a power of two."""
    for dtype in (torch.bfloat16, torch.float32):
        cache, x, slots = _kept(kind, hkv, t, block, scale, dtype, 3.0, t + block)
        _check(cache, kind, x[:, 0], x[:, 1], slots)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("hkv,t,block", FORMS)
@pytest.mark.parametrize("scale", [2.0 ** 122, 2.0 ** 123, 2.0 ** 126, 2.0 ** 127, 1.7 * 2.0 ** 127, float("inf")])
def test_scales_past_those_that_the_append_writes(kind, hkv, t, block, scale):
    """x / s for scales up to fp32's largest, whose reciprocals are below its
    normal range, and for an infinite one (zeros, and NaN for infinities)."""
    for dtype in (torch.bfloat16, torch.float32):
        cache, x, slots = _kept(kind, hkv, t, block, scale, dtype, 2.0 ** 124, t + block + 1)
        _check(cache, kind, x[:, 0], x[:, 1], slots)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("hkv,t,block", FORMS + [(2, 20, 1)])
def test_signs_of_values_that_round_to_zero(dtype, hkv, t, block):
    """Small values beside large ones, new ones and rows that a growing scale
    rounds again: a negative one becomes e4m3's negative zero."""
    kc = _kc()
    d, page = 64, 256
    cache = random_cache(kc, 4, hkv, page, d, block, "e4m3", t)
    g = torch.Generator().manual_seed(t + block)
    x = torch.randn(t, 2, hkv, d, generator=g)
    x[:, :, :, 1::4] *= 2.0 ** -14    # below half of the smallest value, 2^-10, at scales from 2^-8 up
    x[:, :, :, 2] = -0.0
    x *= 2.0 ** 13                    # old rows of size 1 fall below 2^-10 at the new scales
    at = block // 2
    slots = [page * (1 + (at + i) // page) + (at + i) % page for i in range(t)]
    x = x.to(dtype).cuda()
    _check(cache, "e4m3", x[:, 0], x[:, 1], slots)
    k = held(cache, "e4m3")[0]
    assert ((k == 0) & np.signbit(k)).any()


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("hkv,t,block", FORMS)
def test_a_scale_that_is_nan_counts_for_nothing(kind, hkv, t, block):
    """The new rows take the scale that they alone would; the bytes before them
    stay."""
    kc = _kc()
    d, page, at = 64, 256, block // 2
    caches = [random_cache(kc, 4, hkv, page, d, block, kind, t) for _ in range(2)]
    caches[0].scales.fill_(float("nan"))
    caches[1].scales.fill_(2.0 ** -100)
    for c in caches:   # (zeros: rounding them again at another scale keeps them)
        for p in (c.k_pages, c.v_pages):
            p.view(torch.uint8)[1, :, :at] = 0
    caches[0].k_pages.view(torch.uint8)[1, :, :at] = 3
    x = torch.randn(t, 2, hkv, d, generator=torch.Generator().manual_seed(t + block)).bfloat16().cuda()
    slots = torch.tensor([page * (1 + (at + i) // page) + (at + i) % page for i in range(t)], dtype=torch.int32, device="cuda")
    for c in caches:
        kc.q8_append(c, x[:, 0], x[:, 1], slots)
    got, want = [held(c, kind) for c in caches]
    written = ~np.isnan(got[2])
    assert written.any() and np.array_equal(got[2][written], want[2][written])
    assert (caches[0].k_pages.view(torch.uint8)[1, :, :at] == 3).all()
    assert (caches[0].v_pages.view(torch.uint8)[1, :, :at] == 0).all()
    got[0][1, :, :at] = 0
    assert np.array_equal(got[0], want[0], equal_nan=True) and np.array_equal(got[1], want[1], equal_nan=True)
