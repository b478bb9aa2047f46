"""Page tables, append and gather of the 8-bit paged cache against the oracle:
all of them exact, bit for bit."""
import numpy as np
import pytest
import torch

from oracle import q8_oracle as Q
from q8_cases import KINDS, held, random_cache, raw, tables_for

pytestmark = pytest.mark.gpu

I32 = torch.int32


def _kc():
    from sparse_attention_long_anchor_b200 import kascade as kc
    return kc


def _i(v):
    return torch.tensor(v, dtype=I32, device="cuda")


# ---------------------------------------------------------------- page tables

def _check_tables(page, kv, new, free, table, cap):
    kc = _kc()
    t = _i(table)
    out = kc.page_tables(page, _i(kv), _i(new), _i(free), t, cap)
    got = [t.tolist(), *[x.tolist() for x in out]]
    want = Q.page_tables(page, kv, new, free, table, cap)
    assert got == [want[0], want[1], want[2], want[3], want[4]]
    return out


@pytest.mark.parametrize("batch,page,kv_max,new_max,width", [
    (1, 16, 0, 1, 1), (1, 64, 64, 64, 2), (5, 16, 100, 40, 12), (3, 256, 3000, 1, 14), (300, 32, 90, 70, 6),
    (257, 16, 17, 3, 3), (4096, 16, 30, 5, 4), (2, 4096, 9000, 9000, 5), (7, 64, 40, 20000, 320),
])
def test_page_tables_match_the_oracle(batch, page, kv_max, new_max, width):
    rng = np.random.default_rng(batch * 131 + page)
    kv = rng.integers(0, kv_max + 1, batch).tolist()
    new = rng.integers(0, new_max + 1, batch).tolist()
    kv[0], new[-1] = 0, new_max
    total = sum(-(-(a + b) // page) for a, b in zip(kv, new)) + 3
    order = rng.permutation(total).tolist()
    table, at = [], 0
    for a in kv:
        n = -(-a // page)
        table.append(order[at:at + n] + [-7] * (width - n))
        at += n
    free = order[at:]
    for cap in (sum(new), sum(new) + 13):
        out = _check_tables(page, kv, new, free, table, cap)
        assert out[3].tolist()[0] >= 0
    # the same again with exactly the pages that it needs
    need = sum(-(-(a + b) // page) - -(-a // page) for a, b in zip(kv, new))
    _check_tables(page, kv, new, free[:need], table, sum(new) + 1)


def test_page_tables_all_or_nothing():
    page, table = 16, [[0, 1, -1], [2, -1, -1], [3, 4, 5]]
    good = dict(kv=[20, 3, 48], new=[5, 14, 0], free=[9, 8], cap=30)
    out = _check_tables(page, good["kv"], good["new"], good["free"], table, good["cap"])
    assert out[3].tolist() == [1, 19]
    for bad in (dict(kv=[20, -1, 48]), dict(new=[5, -14, 0]), dict(new=[29, 14, 0]), dict(cap=18), dict(free=[]),
                dict(new=[5, 14, 1]), dict(new=[5, 2**31 - 1, 0]), dict(kv=[2**31 - 1, 3, 48]),
                dict(new=[2**30, 2**30, 2**30])):
        a = {**good, **bad}
        out = _check_tables(page, a["kv"], a["new"], a["free"], table, a["cap"])
        assert out[3].tolist() == [-1, 0] and out[2].tolist() == [-1] * a["cap"] and out[0].tolist() == a["kv"]


def test_page_tables_nothing_new_and_given_buffers():
    kc = _kc()
    t = _i([[4, -1], [-1, -1]])
    out = kc.page_tables(16, _i([7, 0]), _i([0, 0]), torch.empty(0, dtype=I32, device="cuda"), t, 0)
    assert [x.tolist() for x in out] == [[7, 0], [0, 0, 0], [], [0, 0]] and t.tolist() == [[4, -1], [-1, -1]]
    # given buffers, the slots at an address that is not 16-byte aligned, with guards around them
    buf = torch.full((40,), 777, dtype=I32, device="cuda")
    out = (buf[0:2], buf[3:6], buf[9:20], buf[30:32])
    got = kc.page_tables(16, _i([7, 0]), _i([3, 5]), _i([9]), t, 11, out=out)
    assert got is out
    want = Q.page_tables(16, [7, 0], [3, 5], [9], [[4, -1], [-1, -1]], 11)
    assert [x.tolist() for x in out] == [want[1], want[2], want[3], want[4]] and t.tolist() == want[0]
    rest = buf.tolist()
    assert all(rest[i] == 777 for i in [2, 6, 7, 8, *range(20, 30), *range(32, 40)])
    with pytest.raises(kc.KascadeError):
        lens = _i([7, 0])
        kc.page_tables(16, lens, _i([3, 5]), _i([9]), t, 11, out=(lens, *out[1:]))


# ---------------------------------------------------------------- append

def _same(cache, kind, want):
    k, v, s = held(cache, kind)
    assert np.array_equal(s, want[2])
    for got, ref in ((k, want[0]), (v, want[1])):
        assert np.array_equal(np.isnan(got), np.isnan(ref))
        assert np.array_equal(got[~np.isnan(ref)], ref[~np.isnan(ref)])


def _append_and_check(cache, kind, k, v, slots, ws=None):
    kc = _kc()
    want = [x.copy() for x in held(cache, kind)]
    for which, x in enumerate((k, v)):
        Q.append(want[which], want[2], x.float().cpu().numpy(), list(slots), which, cache.scale_block, kind)
    kc.q8_append(cache, k, v, _i(slots), ws=ws)
    _same(cache, kind, want)


def _slots(kv, new, rows, page):
    return [r[p // page] * page + p % page for a, n, r in zip(kv, new, rows) for p in range(a, a + n)]


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("hkv,d,page,block", [(2, 64, 32, 16), (1, 128, 16, 1), (3, 128, 64, 64), (1, 64, 256, 256),
                                              (2, 128, 16, 8)])
def test_append_matches_the_oracle(kind, dtype, hkv, d, page, block):
    """Ragged chunks behind running contexts, then single tokens; the new rows
    grow some blocks' scales and not others."""
    seed = hkv * 1000 + d + page + block
    g = torch.Generator().manual_seed(seed)
    kv, new = [0, page - 1, 5, 3 * page // 2, block // 2], [2 * page + 3, 1, 9, page, 0]
    lens = [a + b + 4 for a, b in zip(kv, new)]
    width = max(-(-n // page) for n in lens)
    num = sum(-(-n // page) for n in lens) + 2
    rows, _ = tables_for(lens, page, width, num, seed)
    cache = random_cache(_kc(), num, hkv, page, d, block, kind, seed)
    for step in range(4):
        t = sum(new)
        # views of a fused projection; magnitudes that differ from block to block
        qkv = torch.randn(t, 3, hkv, d, generator=g) * torch.exp2(torch.randint(-6, 7, (t, 3, hkv, 1), generator=g).float())
        qkv = qkv.to(dtype).cuda()
        _append_and_check(cache, kind, qkv[:, 1], qkv[:, 2], _slots(kv, new, rows, page))
        kv = [a + b for a, b in zip(kv, new)]
        new = [1] * len(kv)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_append_long_prompt_takes_the_tiled_form(kind):
    """Enough tokens that a CTA takes more than eight of them; runs that cross
    its borders; heads side by side in memory ([T, d] slabs per head)."""
    g = torch.Generator().manual_seed(11)
    for page, block, kv, new in ((64, 64, [0, 37], [2100, 2333]), (32, 8, [3, 0], [1999, 2501]), (256, 256, [250], [4400])):
        hkv, d = 4, 64
        lens = [a + b for a, b in zip(kv, new)]
        width = max(-(-n // page) for n in lens)
        rows, _ = tables_for(lens, page, width, sum(-(-n // page) for n in lens) + 1, 5)
        cache = random_cache(_kc(), sum(-(-n // page) for n in lens) + 1, hkv, page, d, block, kind, 9)
        x = (torch.randn(2, hkv, sum(new), d, generator=g) * 3).bfloat16().cuda()
        _append_and_check(cache, kind, x[0].transpose(0, 1), x[1].transpose(0, 1), _slots(kv, new, rows, page))


@pytest.mark.parametrize("kind,dtype,d,page,block", [
    ("e4m3", torch.float32, 64, 64, 1), ("int8", torch.float16, 64, 16, 4), ("int8", torch.bfloat16, 128, 256, 256),
    ("e4m3", torch.float16, 128, 64, 64), ("int8", torch.float32, 64, 128, 128), ("e4m3", torch.bfloat16, 64, 32, 2)])
def test_append_tiled_form_values_gaps_and_old_rows(kind, dtype, d, page, block):
    """Many heads bring few tokens to the form for prompts: skipped tokens
    inside and between runs, infinities and NaN, zero rows, blocks whose scale
    grows over their old rows, and a caller's scale that is no power of two."""
    kc = _kc()
    hkv = 32
    kv, new = [block // 2, 3, 2 * page - 1], [520, 40, 333]
    lens = [a + b + 2 for a, b in zip(kv, new)]
    width = max(-(-n // page) for n in lens)
    num = sum(-(-n // page) for n in lens) + 1
    rows, _ = tables_for(lens, page, width, num, d + block)
    cache = random_cache(kc, num, hkv, page, d, block, kind, block)
    cache.scales[:, ::3] *= 0.7
    g = torch.Generator().manual_seed(block)
    slots = []
    for i, sl in enumerate(_slots(kv, new, rows, page)):
        slots.append(sl)
        if i % 97 == 50:
            slots += [-1] * (i % 31 + 1)
        if i in (519, 559):
            slots += [-1] * 90
    t = len(slots)
    x = torch.randn(t, 2, hkv, d, generator=g) * torch.exp2(torch.randint(-5, 6, (t, 2, hkv, 1), generator=g).float())
    x[60:70] = 0.0
    x[100, 0, ::2, 3] = float("inf")
    x[101:103, 1, 1, 4] = float("-inf")
    x[200, :, 5] = float("nan")
    x[300:300 + block, :, 7, :] = float("nan")
    x = x.to(dtype).cuda()
    ws = kc.Workspace(kc.Shape.make(1, 2, 2, 64, 1, 16), (kc.OP_DENSE,))
    _append_and_check(cache, kind, x[:, 0], x[:, 1], slots, ws)
    assert ws.error() == 0
    bad = list(slots)
    bad[10], bad[400] = num * page, -7
    _append_and_check(cache, kind, x[:, 1], x[:, 0], bad, ws)
    assert ws.error(clear=True) == kc.DEVERR_PAGE


@pytest.mark.parametrize("kind,dtype,d,page,block", [
    ("e4m3", torch.bfloat16, 128, 64, 64), ("int8", torch.bfloat16, 128, 128, 32), ("e4m3", torch.float32, 128, 128, 128),
    ("int8", torch.float32, 64, 64, 4), ("e4m3", torch.float16, 64, 256, 256), ("int8", torch.float16, 128, 16, 16),
    ("e4m3", torch.float32, 128, 256, 256), ("int8", torch.bfloat16, 64, 32, 8), ("e4m3", torch.float32, 64, 16, 1)])
def test_append_whole_blocks(kind, dtype, d, page, block):
    """Prompts of whole blocks, which the form for prompts takes without a
    search: from a block's first row and from its middle, with values that are
    not finite, with a row left out, one skipped, one outside the pool, and
    with a head count that leaves warps without work."""
    kc = _kc()
    tile = max(64, block)
    hkv = {64: 21, 128: 9, 256: 5}[tile]   # enough rows for that form, none a multiple of a CTA's
    kv, new = [0, block // 2 + 1, 3 * block, 0], [2 * tile, 2 * tile + 17, 2 * tile + 1, 2 * tile + block // 2]
    lens = [a + b for a, b in zip(kv, new)]
    width = max(-(-n // page) for n in lens)
    num = sum(-(-n // page) for n in lens) + 1
    rows, _ = tables_for(lens, page, width, num, 7 * d + block)
    cache = random_cache(kc, num, hkv, page, d, block, kind, block + 1)
    slots = _slots(kv, new, rows, page)
    t = len(slots)
    g = torch.Generator().manual_seed(block + d)
    x = torch.randn(t, 2, hkv, d, generator=g) * torch.exp2(torch.randint(-5, 6, (t, 2, hkv, 1), generator=g).float())
    x[3, 0, ::2, 3] = float("inf")
    x[tile + 5, 1, 1, 4] = float("-inf")
    x[2 * tile + 70, :, 2] = float("nan")
    x[block:2 * block, :, 3, :] = float("nan")
    x[0:block, 1, 4, :] = 0.0
    x = x.to(dtype).cuda()
    ws = kc.Workspace(kc.Shape.make(1, 2, 2, 64, 1, 16), (kc.OP_DENSE,))
    _append_and_check(cache, kind, x[:, 0], x[:, 1], slots, ws)
    left = [i for i in range(t) if i not in (2, 4 * tile + 18)]   # blocks with a row that no token fills
    fewer, y = [slots[i] for i in left], x[torch.tensor(left, device="cuda")] * 2
    fewer[tile + 9] = -1
    _append_and_check(cache, kind, y[:, 1], y[:, 0], fewer, ws)
    assert ws.error() == 0
    fewer[tile + 9] = num * page
    _append_and_check(cache, kind, y[:, 0], y[:, 1], fewer, ws)
    assert ws.error(clear=True) == kc.DEVERR_PAGE


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_append_values_at_the_edges(kind):
    """Zero blocks, infinities, NaN, the largest and smallest magnitudes, values
    at rounding borders, and a block that keeps a scale of the caller's own."""
    kc = _kc()
    hkv, d, page, block = 2, 64, 16, 4
    cache = kc.Q8Cache.empty(6, hkv, d, page, block, KINDS[kind])
    x = torch.randn(24, hkv, d, generator=torch.Generator().manual_seed(1))
    x[0:4] = 0.0
    x[4:8, :, 5] = float("inf")
    x[5, 0, 6] = float("-inf")
    x[6, 1, :3] = float("nan")
    x[8:12] *= 1e36
    x[12:16] *= 1e-38
    x[16:20] = (torch.arange(4 * hkv * d).float().view(4, hkv, d) / 16)
    x[20:24] = float("nan")
    slots = [16 * (i // 8) * 2 + (i % 8) for i in range(24)]
    ws = kc.Workspace(kc.Shape.make(1, 2, 2, 64, 1, 16), (kc.OP_DENSE,))
    _append_and_check(cache, kind, x.cuda(), x.flip(0).contiguous().cuda(), slots, ws)
    # the caller's scale, not a power of two, larger than the new rows need
    cache.scales[1, :, 0] = 0.3
    y = torch.randn(2, hkv, d, generator=torch.Generator().manual_seed(2)).cuda()
    _append_and_check(cache, kind, y, 2 * y, [page + 1, page + 2], ws)
    # and smaller: the rows before are rounded again
    _append_and_check(cache, kind, 1000 * y[:1], 3000 * y[:1], [page + 3], ws)
    assert ws.error() == 0


def test_append_skips_padding_and_reports_slots_outside_the_pool():
    kc = _kc()
    hkv, d, page, block = 2, 128, 32, 32
    cache = random_cache(kc, 5, hkv, page, d, block, "e4m3", 3)
    x = torch.randn(9, hkv, d, generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    ws = kc.Workspace(kc.Shape.make(1, 2, 2, 64, 1, 16), (kc.OP_DENSE,))
    _append_and_check(cache, "e4m3", x, -x, [40, 41, -1, 42, -1, -1, 7, -1, -1], ws)
    assert ws.error() == 0
    _append_and_check(cache, "e4m3", x, -x, [-1] * 9, ws)
    assert ws.error() == 0
    for bad in (5 * 32, 2**31 - 1, -2):
        _append_and_check(cache, "e4m3", x, -x, [64, bad, 65, 96, 97, 98, bad, bad, 0], ws)
        assert ws.error(clear=True) == kc.DEVERR_PAGE
    # longer stretches of padding: 31 skipped tokens inside a block, and many between blocks, for a
    # short run and for one that a whole CTA takes
    for rows in (6, 24):
        slots = []
        for i in range(rows):
            slots += [96 + i] + [-1] * (31 if i in (1, rows - 2) else 0)
        slots += [-1] * 100 + [3, 4] + [-1] * 50 + [130]
        y = torch.randn(len(slots), hkv, d, generator=torch.Generator().manual_seed(rows)).bfloat16().cuda()
        _append_and_check(cache, "e4m3", y, 3 * y, slots, ws)
    assert ws.error() == 0
    before = raw(cache.k_pages).copy()
    kc.q8_append(cache, x[:0], x[:0], _i([]))
    assert np.array_equal(before, raw(cache.k_pages))


# ---------------------------------------------------------------- gather

@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("hkv,d,page,block,n,lens", [
    (2, 64, 16, 4, 100, [100, 1, 0, 57]), (1, 128, 64, 64, 1, [1]), (3, 128, 32, 1, 333, [333, 32, 33]),
    (1, 64, 4096, 256, 700, [650])])
def test_gather_matches_the_cache(kind, dtype, hkv, d, page, block, n, lens):
    kc = _kc()
    width = -(-n // page) + 1
    num = sum(-(-x // page) for x in lens) + 2
    rows, _ = tables_for(lens, page, width, num, n)
    cache = random_cache(kc, num, hkv, page, d, block, kind, n + d, scale="free")
    k = torch.full((len(lens), hkv, n, d), 9.0, dtype=dtype, device="cuda")
    v = k.clone()
    ws = kc.Workspace(kc.Shape.make(1, 2, 2, 64, 1, 16), (kc.OP_DENSE,))
    got = kc.q8_gather(cache, _i(rows), n, _i(lens), k=k, v=v, ws=ws)
    assert got[0] is k and got[1] is v and ws.error() == 0
    kval, vval, sc = held(cache, kind)
    for which, (out, val) in enumerate(((k, kval), (v, vval))):
        want = torch.full(out.shape, 9.0, dtype=dtype)
        for b, m in enumerate(lens):
            for h in range(hkv):
                x = np.zeros((m, d), dtype=np.float32)
                for j in range(m):
                    pg, r = rows[b][j // page], j % page
                    # one fp32 product, then one rounding
                    x[j] = val[pg, h, r].astype(np.float32) * np.float32(sc[pg, h, r // block, which])
                want[b, h, :m] = torch.from_numpy(x).to(dtype)
        assert torch.equal(out.cpu(), want)
    # one of the two alone; slabs of the call's own are zero behind the rows
    k1, v1 = kc.q8_gather(cache, _i(rows), n, _i(lens), v=torch.full_like(v, 9.0))
    assert k1 is None and torch.equal(v1, v)
    k2, v2 = kc.q8_gather(cache, _i(rows), n, _i(lens), dtype=dtype)
    live = torch.arange(n, device="cuda")[None] < _i(lens)[:, None]
    assert torch.equal(k2, torch.where(live[:, None, :, None], k, torch.zeros_like(k)))


def test_gather_lengths_out_of_range_and_bad_pages():
    kc = _kc()
    hkv, d, page, n = 2, 64, 16, 64
    cache = random_cache(kc, 8, hkv, page, d, 16, "int8", 1)
    good = _i([[3, 1, 0, 2], [4, 5, 6, 7]])
    ws = kc.Workspace(kc.Shape.make(1, 2, 2, 64, 1, 16), (kc.OP_DENSE,))
    full = kc.q8_gather(cache, good, n, None, ws=ws)
    clamped = kc.q8_gather(cache, good, n, _i([n + 1000, -5]), ws=ws)
    assert torch.equal(clamped[0][0], full[0][0]) and (clamped[0][1] == 0).all() and ws.error() == 0
    for bad in (8, -1, 2**31 - 1, -2**31):
        t = good.clone()
        t[1, 2] = bad
        out = kc.q8_gather(cache, t, n, None, ws=ws)
        assert ws.error(clear=True) == kc.DEVERR_PAGE
        assert torch.equal(out[0][0], full[0][0]) and torch.equal(out[1][1, :, :32], full[1][1, :, :32])
    # entries behind the rows are not looked at
    t = good.clone()
    t[1, 2:] = 99
    kc.q8_gather(cache, t, n, _i([n, 32]), ws=ws)
    assert ws.error() == 0
