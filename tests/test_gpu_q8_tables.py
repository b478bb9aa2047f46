"""Page tables whose entries no pool can have: the slots that come of them are
reported by the append that gets them, and write nothing."""
import numpy as np
import pytest
import torch

from oracle import q8_oracle as Q
from q8_cases import held, random_cache, raw

pytestmark = pytest.mark.gpu

I32 = torch.int32
BAD_SLOT = -2 ** 31


def _kc():
    from sparse_attention_long_anchor_b200 import kascade as kc
    return kc


def _i(v):
    return torch.tensor(v, dtype=I32, device="cuda")


# (tokens held and new, free pages, table): entries that are unset, negative, or would come back into the pool at 32 bits
CASES = [
    # the last row of a page that is not set: page -1 times 64 plus 63 is the padding mark
    dict(kv=[63, 5], new=[1, 1], free=[4], table=[[-1, -1], [2, -1]], bad=[0]),
    dict(kv=[127, 5], new=[1, 1], free=[4], table=[[1, -1], [2, -1]], bad=[0]),
    # 2^26 + 3 pages of 64 rows: page 3 at 32 bits; 2^25 is the first that no slot can name
    dict(kv=[10, 5], new=[2, 1], free=[4], table=[[2 ** 26 + 3, -1], [2, -1]], bad=[0, 1]),
    dict(kv=[10, 5], new=[2, 1], free=[4], table=[[2 ** 25, -1], [2, -1]], bad=[0, 1]),
    dict(kv=[10, 5], new=[2, 1], free=[4], table=[[-2 ** 31, -1], [2, -1]], bad=[0, 1]),
    # the same from the free list, behind a page that is held
    dict(kv=[64, 5], new=[2, 1], free=[2 ** 26 + 3], table=[[1, -1], [2, -1]], bad=[0, 1]),
    dict(kv=[0, 5], new=[64, 1], free=[-1], table=[[-1, -1], [2, -1]], bad=list(range(64))),
    # outside this pool, but not of every pool: the slot says so by itself
    dict(kv=[10, 5], new=[2, 1], free=[4], table=[[2 ** 25 - 1, -1], [2, -1]], bad=[]),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_entries_that_no_pool_has_become_slots_that_are_reported(case):
    kc, c = _kc(), CASES[case]
    page, hkv, d = 64, 2, 64
    table = _i(c["table"])
    t = sum(c["new"])
    lens, offsets, slots, info = kc.page_tables(page, _i(c["kv"]), _i(c["new"]), _i(c["free"]), table, t + 3)
    want = Q.page_tables(page, c["kv"], c["new"], c["free"], c["table"], t + 3)
    for i in c["bad"]:
        want[3][i] = BAD_SLOT
    assert [table.tolist(), lens.tolist(), offsets.tolist(), slots.tolist(), info.tolist()] == list(want)
    cache = random_cache(kc, 5, hkv, page, d, 16, "e4m3", 3)
    ws = kc.Workspace(kc.Shape.make(1, 2, 2, 64, 1, 16), (kc.OP_DENSE,))
    x = torch.randn(t + 3, 2, hkv, d, generator=torch.Generator().manual_seed(case)).bfloat16().cuda()
    ref = [a.copy() for a in held(cache, "e4m3")]
    for which in range(2):   # (slots outside the pool count for nothing)
        Q.append(ref[which], ref[2], x[:, which].float().cpu().numpy(), list(want[3]), which, 16, "e4m3")
    kc.q8_append(cache, x[:, 0], x[:, 1], slots, ws=ws)
    assert ws.error(clear=True) == kc.DEVERR_PAGE
    got = held(cache, "e4m3")
    assert all(np.array_equal(a, b) for a, b in zip(got, ref))
    # the pages that nothing was appended to are as they were
    fresh = random_cache(kc, 5, hkv, page, d, 16, "e4m3", 3)
    for a, b in ((cache.k_pages, fresh.k_pages), (cache.v_pages, fresh.v_pages)):
        assert np.array_equal(raw(a)[[0, 1, 3, 4]], raw(b)[[0, 1, 3, 4]])
