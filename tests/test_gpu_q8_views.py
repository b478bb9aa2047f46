"""Forms in which the append's rows may come."""
import pytest
import torch

from q8_cases import random_cache, raw

pytestmark = pytest.mark.gpu


def _kc():
    from sparse_attention_long_anchor_b200 import kascade as kc
    return kc


def _slots(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("t,hkv", [(1, 1), (1, 3), (5, 1)])
def test_strides_of_dimensions_of_one_do_not_matter(dtype, t, hkv):
    """A dimension of size 1 may have any stride: nothing is reached through it."""
    kc = _kc()
    d, page = 64, 16
    x = torch.randn(2, t, hkv, d, generator=torch.Generator().manual_seed(t)).to(dtype).cuda()
    odd = [a.as_strided((t, hkv, d), (a.stride(0) if t > 1 else 3, a.stride(1) if hkv > 1 else 1, 1)) for a in x]
    assert all(torch.equal(a, b) for a, b in zip(odd, x))
    caches = [random_cache(kc, 3, hkv, page, d, 4, "int8", 7) for _ in range(2)]
    for cache, (k, v) in zip(caches, (x, odd)):
        kc.q8_append(cache, k, v, _slots(list(range(18, 18 + t))))
    assert all((raw(getattr(caches[0], n)) == raw(getattr(caches[1], n))).all() for n in ("k_pages", "v_pages", "scales"))
    # a dimension that has more elements keeps its rule
    with pytest.raises(kc.KascadeError):
        y = torch.zeros(4, hkv, d + 1, dtype=dtype, device="cuda")[..., :d]
        kc.q8_append(caches[0], y, y, _slots([1, 2, 3, 4]))


def test_rows_of_another_rank_are_refused():
    """As every other wrong argument is: by the binding's own error."""
    kc = _kc()
    cache = random_cache(kc, 3, 2, 16, 64, 4, "e4m3", 7)
    before = raw(cache.k_pages).copy()
    x = torch.zeros(5, 2, 64, dtype=torch.bfloat16, device="cuda")
    slots = _slots([0, 1, 2, 3, 4])
    for k, v in ((x.view(5, 128), x.view(5, 128)), (x[None], x[None]), (x[0, 0], x[0, 0]), (x, x[None]), (x[None], x),
                 (x.sum(), x.sum())):
        with pytest.raises(kc.KascadeError):
            kc.q8_append(cache, k, v, slots)
    assert (raw(cache.k_pages) == before).all()
