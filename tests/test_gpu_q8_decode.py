"""Single-token attention over the 8-bit paged cache against the oracle, with
the bounds that its roundings give (q8_cases.attention_bound)."""
import numpy as np
import pytest
import torch

import oracle as O
from q8_cases import check_decode, held, random_cache, tables_for

pytestmark = pytest.mark.gpu

I32 = torch.int32
DT = {"bf16": (torch.bfloat16, 0), "fp16": (torch.float16, 2)}


def _kc():
    from sparse_attention_long_anchor_b200 import kascade as kc
    return kc


def _i(v):
    return torch.tensor(v, dtype=I32, device="cuda")


def _lists(lens, n_lists, n, frac, seed):
    """Ascending random lists per row, and the padded index buffer."""
    rng = np.random.default_rng(seed)
    kk = O.topk_count(n, *frac)
    idx = np.full((len(lens), n_lists, kk), -1, dtype=np.int32)
    lists = []
    for b, m in enumerate(lens):
        k = O.topk_count(m, *frac)
        lists.append([np.sort(rng.permutation(m)[:k]) for _ in range(n_lists)])
        for p in range(n_lists):
            idx[b, p, :k] = lists[b][p]
    return lists, torch.from_numpy(idx).cuda()


def _case(kind, qt, hq, hkv, d, page, block, n, lens, frac, mode=0, hm=None, scale="pow2", seed=0, spoil=False,
          flags=0, qscale=1.5):
    kc = _kc()
    dtype, code = DT[qt]
    lens = [n] * lens if isinstance(lens, int) else lens
    width = -(-n // page) + 1
    num = sum(-(-x // page) for x in lens) + 2
    rows, _ = tables_for(lens, page, width, num, seed + n)
    cache = random_cache(kc, num, hkv, page, d, block, kind, seed + d, scale=scale)
    hc = held(cache, kind)
    if spoil:
        # every row and scale that no request holds is NaN (int8: -128 and a NaN scale)
        used = np.zeros((num, page), dtype=bool)
        for b, m in enumerate(lens):
            for j in range(m):
                used[rows[b][j // page], j % page] = True
        u = torch.from_numpy(used).cuda()
        bad = 0x7f if kind == "e4m3" else 0x80
        for pages in (cache.k_pages, cache.v_pages):
            by = pages.view(torch.uint8)
            by.copy_(torch.where(u[:, None, :, None], by, torch.full_like(by, bad)))
        ub = u.view(num, page // block, block).any(-1)
        cache.scales.copy_(torch.where(ub[:, None, :, None], cache.scales, torch.full_like(cache.scales, float("nan"))))
    g = torch.Generator().manual_seed(seed + 5)
    q = (qscale * torch.randn(len(lens), hq, 1, d, generator=g)).to(dtype).cuda()
    s = kc.Shape.make(len(lens), hq, hkv, d, 1, n, frac or (1, 1), mode=mode, dtype=code, flags=flags)
    lists = idx = None
    if frac:
        lists, idx = _lists(lens, s.n_lists, n, frac, seed)
    lse = torch.empty(len(lens), hq, device="cuda")
    ws = kc.Workspace(s, (kc.OP_SPARSE_DECODE_Q8,))
    ws.buf[256:].fill_(0xff)   # nothing depends on what the workspace holds
    ragged = lens != [n] * len(lens)
    o = kc.sparse_decode_q8(s, q, cache, _i(rows), idx, None if hm is None else _i(hm),
                            kv_lens=_i(lens) if ragged else None, lse=lse, ws=ws)
    torch.cuda.synchronize()
    assert ws.error() == 0
    name = (kind, qt, hq, hkv, d, page, block, n, lens, frac, mode)
    check_decode(name, q.view(len(lens), hq, d).double().cpu().numpy(), hc, rows, lens, lists,
                 o.view(len(lens), hq, d).double().cpu().numpy(), lse.double().cpu().numpy(), dtype, hm, mode == 1)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 127, 200, 1000])
@pytest.mark.parametrize("kind,qt,hq,hkv,d", [("e4m3", "bf16", 8, 2, 128), ("int8", "fp16", 4, 4, 64),
                                              ("e4m3", "fp16", 8, 1, 64), ("int8", "bf16", 3, 1, 128)])
def test_dense_lengths(kind, qt, hq, hkv, d, n):
    _case(kind, qt, hq, hkv, d, 16, 8, n, 2, None, seed=n)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (5, 1), (12, 2), (7, 1), (8, 1), (6, 6)])
@pytest.mark.parametrize("kind,qt,d", [("e4m3", "bf16", 128), ("int8", "fp16", 64)])
def test_group_sizes(kind, qt, d, hq, hkv):
    _case(kind, qt, hq, hkv, d, 32, 32, 150, [150, 77], (30, 100), seed=hq)


@pytest.mark.parametrize("page,block", [(16, 1), (16, 16), (64, 2), (128, 64), (1024, 256), (4096, 16)])
@pytest.mark.parametrize("scale", ["pow2", "free"])
def test_pages_blocks_and_scales(page, block, scale):
    _case("e4m3", "bf16", 8, 2, 128, page, block, 700, [700, 16, 333], None, scale=scale, seed=page)
    _case("int8", "bf16", 8, 2, 64, page, block, 700, [700, 1, 512], (20, 100), scale=scale, seed=block, hm=[1, 0])


@pytest.mark.parametrize("mode,hm", [(0, None), (0, [1, 1]), (1, None), (1, [7, 0, 3, 3, 1, 6, 5, 2]), (2, None)])
def test_selection_modes(mode, hm):
    _case("e4m3", "bf16", 8, 2, 128, 64, 64, 900, [900, 450, 3], (10, 100), mode=mode, hm=hm, seed=mode)
    _case("int8", "fp16", 8, 2, 64, 32, 4, 257, 1, (1, 3), mode=mode, hm=hm, seed=mode)


def test_rows_without_keys_and_maps_out_of_range():
    """A context of no keys, and a head whose map entry names no list, give
    zeros and a log-sum-exp of minus infinity."""
    for n in (100, 5000):   # one split, and many
        _case("e4m3", "bf16", 8, 2, 128, 64, 64, n, [0, n, 0], None)
        _case("e4m3", "bf16", 8, 2, 128, 64, 64, n, [0, n, 1], (10, 100), hm=[1, 2])
        _case("int8", "fp16", 8, 2, 64, 64, 64, n, [n, 0], (10, 100), hm=[-1, 0])


@pytest.mark.parametrize("n,lens,frac", [(5000, [5000, 4097], None), (4999, [4999, 31], (10, 100)),
                                         (20011, [20011], None), (3001, [1, 2, 3, 3001, 1500, 64, 65, 0], (50, 100))])
def test_many_splits(n, lens, frac):
    _case("e4m3", "bf16", 8, 2, 128, 64, 16, n, lens, frac, seed=n)
    _case("int8", "fp16", 16, 2, 64, 128, 128, n, lens, frac, seed=n + 1, scale="free")


@pytest.mark.parametrize("B,hkv,n,frac", [(40, 2, 600, None), (70, 1, 900, (40, 100)), (33, 8, 300, None),
                                          (100, 3, 1400, None), (160, 2, 200, None), (148, 2, 260, None),
                                          (38, 2, 2400, None), (37, 2, 3000, None), (74, 1, 4200, None)])
def test_batches_past_a_warp_of_rows_and_past_the_resident_ctas(B, hkv, n, frac):
    """More rows than a warp counts at once; more problems than CTAs run at
    once, with one and several CTAs to a problem; as many as they are."""
    rng = np.random.default_rng(B)
    lens = rng.integers(0, n + 1, B).tolist()
    lens[3], lens[-1] = n, 0
    _case("e4m3", "bf16", 2 * hkv, hkv, 64, 16, 16, n, lens, frac, seed=B)
    _case("int8", "fp16", hkv, hkv, 128, 64, 4, n, [n] * B, frac, seed=B + 1)


def test_rows_do_not_depend_on_how_the_batch_is_split():
    """Each row of a ragged batch against the row alone, within both calls'
    bounds of the oracle (the split follows the batch's lengths)."""
    kc = _kc()
    lens, n, hkv, d = [9000, 130, 0, 4321, 1], 9000, 2, 128
    rows, _ = tables_for(lens, 64, 141, 400, 3)
    cache = random_cache(kc, 400, hkv, 64, d, 64, "e4m3", 3)
    q = torch.randn(5, 8, 1, d, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    o = kc.sparse_decode_q8(kc.Shape.make(5, 8, hkv, d, 1, n), q, cache, _i(rows), kv_lens=_i(lens))
    hc = held(cache, "e4m3")
    for b, m in enumerate(lens):
        if m:
            one = kc.Shape.make(1, 8, hkv, d, 1, m)
            lse = torch.empty(1, 8, device="cuda")
            alone = kc.sparse_decode_q8(one, q[b:b + 1].contiguous(), cache, _i([rows[b]]), lse=lse)
            for x in (alone, o[b:b + 1]):
                check_decode(b, q[b:b + 1].view(1, 8, d).double().cpu().numpy(), hc, [rows[b]], [m], None,
                             x.view(1, 8, d).double().cpu().numpy(), lse.double().cpu().numpy(), torch.bfloat16)
        else:
            assert (o[b] == 0).all()


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("frac", [None, (25, 100)])
def test_places_outside_the_contexts_do_not_matter(kind, frac):
    """NaN values and scales behind the last row of each request, and page-table
    entries behind its pages that name no page."""
    _case(kind, "bf16", 8, 2, 128, 64, 16, 300, [300, 1, 17, 0, 129], frac, spoil=True, seed=3)
    _case(kind, "fp16", 8, 2, 64, 32, 1, 2500, [2500, 1001], frac, spoil=True, seed=4)


@pytest.mark.parametrize("qscale", [1e-30, 1e-6, 30.0, 1e4])
def test_query_magnitudes(qscale):
    """Tiny queries (nearly even weights) and large ones (one key takes all)."""
    _case("e4m3", "bf16", 8, 2, 128, 64, 64, 400, 2, None, qscale=qscale)
    _case("int8", "bf16", 8, 2, 64, 64, 64, 400, 2, (10, 100), qscale=qscale)


def test_query_of_zeros_infinities_and_nan():
    kc = _kc()
    cache = random_cache(kc, 8, 2, 64, 128, 64, "e4m3", 1)
    t = _i([[3, 1, 0, 2, 4]])
    s = kc.Shape.make(1, 8, 2, 128, 1, 300)
    q = torch.randn(1, 8, 1, 128, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    q[0, 1] = 0
    q[0, 2, 0, 5] = float("nan")
    q[0, 3, 0, 7] = float("inf")
    ws = kc.Workspace(s, (kc.OP_SPARSE_DECODE_Q8,))
    o = kc.sparse_decode_q8(s, q, cache, t, ws=ws)
    clean = q.clone()
    clean[0, 2:4] = 0
    ref = kc.sparse_decode_q8(s, clean, cache, t, ws=ws)
    torch.cuda.synchronize()
    assert o[0, 2].isnan().all() and o[0, 3].isnan().all()
    keep = [0, 1, 4, 5, 6, 7]
    assert torch.equal(o[:, keep], ref[:, keep]) and torch.isfinite(ref).all()


@pytest.mark.parametrize("B,n", [(1, 100), (1, 6000), (1, 40000), (50, 1500)])
def test_flags_give_the_same_bits(B, n):
    """A CTA to a list, clusters, shares and waves: calls launched to overlap
    their predecessors, sharing one workspace and the outputs' memory."""
    kc = _kc()
    per = -(-n // 64)
    cache = random_cache(kc, 700, 2, 64, 128, 64, "e4m3", 6)
    t = _i([[(b * 13 + i) % 700 for i in range(per)] for b in range(B)])
    s = kc.Shape.make(B, 8, 2, 128, 1, n)
    qs = [torch.randn(B, 8, 1, 128, generator=torch.Generator().manual_seed(n + i)).bfloat16().cuda() for i in range(2)]
    lens = _i([max(1, n - 31 * b) for b in range(B)])
    ws = kc.Workspace(s, (kc.OP_SPARSE_DECODE_Q8,))
    for kv in (None, lens):
        ref = [kc.sparse_decode_q8(s, q, cache, t, kv_lens=kv, ws=ws).clone() for q in qs]
        for flags in (kc.FLAG_PDL, kc.FLAG_PDL | kc.FLAG_INPUTS_STABLE):
            outs = [kc.sparse_decode_q8(s.with_flags(flags), qs[i % 2], cache, t, kv_lens=kv, ws=ws) for i in range(20)]
            torch.cuda.synchronize()
            assert ws.error() == 0
            assert all(torch.equal(o, ref[i % 2]) for i, o in enumerate(outs))
        # each call's query is the output of the call before it
        chains = []
        for flags in (0, kc.FLAG_PDL, kc.FLAG_PDL | kc.FLAG_INPUTS_STABLE):
            x = [qs[0].clone(), torch.empty_like(qs[0])]
            for i in range(24):
                kc.sparse_decode_q8(s.with_flags(flags), x[i % 2], cache, t, kv_lens=kv, o=x[1 - i % 2], ws=ws)
            torch.cuda.synchronize()
            chains.append(x)
        assert all(torch.equal(a, b) for c in chains[1:] for a, b in zip(c, chains[0]))


def test_bad_list_and_table_entries_are_reported():
    kc = _kc()
    n, page = 1000, 64
    cache = random_cache(kc, 20, 2, page, 128, 64, "e4m3", 6)
    t = _i([list(range(16))])
    s = kc.Shape.make(1, 8, 2, 128, 1, n, (10, 100))
    q = torch.randn(1, 8, 1, 128, generator=torch.Generator().manual_seed(8)).bfloat16().cuda()
    lists, idx = _lists([n], 2, n, (10, 100), 5)
    ws = kc.Workspace(s, (kc.OP_SPARSE_DECODE_Q8,))
    for bad, near in ((n, n - 1), (2**31 - 1, n - 1), (-1, 0), (-2**31, 0)):
        i = idx.clone()
        i[0, 1, 7] = bad
        o = kc.sparse_decode_q8(s, q, cache, t, i, ws=ws)
        assert ws.error(clear=True) == kc.DEVERR_INDEX_LIST
        i[0, 1, 7] = near
        assert torch.equal(o, kc.sparse_decode_q8(s, q, cache, t, i, ws=ws)) and ws.error() == 0
    for bad in (20, -1, 2**31 - 1, -2**31):
        tb = t.clone()
        tb[0, 3] = bad
        o = kc.sparse_decode_q8(s, q, cache, tb, None, ws=ws)
        assert ws.error(clear=True) == kc.DEVERR_PAGE
        tb[0, 3] = 0
        assert torch.equal(o, kc.sparse_decode_q8(s, q, cache, tb, None, ws=ws)) and ws.error() == 0
    # lengths outside [0, N] are held to it
    o = kc.sparse_decode_q8(s, q, cache, t, None, kv_lens=_i([n + 5]), ws=ws)
    assert torch.equal(o, kc.sparse_decode_q8(s, q, cache, t, None, ws=ws)) and ws.error() == 0
    assert (kc.sparse_decode_q8(s, q, cache, t, None, kv_lens=_i([-3]), ws=ws) == 0).all()


def test_the_binding_checks_its_tensors():
    kc = _kc()
    cache = random_cache(kc, 20, 2, 64, 128, 64, "e4m3", 6)
    t = _i([list(range(16))])
    s = kc.Shape.make(1, 8, 2, 128, 1, 1000, (10, 100))
    q = torch.randn(1, 8, 1, 128).bfloat16().cuda()
    _, idx = _lists([1000], 2, 1000, (10, 100), 5)
    lse = torch.empty(1, 8, device="cuda")
    good = dict(q=q, page_table=t, idx=idx, head_map=_i([0, 1]), kv_lens=_i([7]), lse=lse)

    def call(**kw):
        a = {**good, **kw}
        return kc.sparse_decode_q8(s, a.pop("q"), cache, a.pop("page_table"), **a)
    call()
    for kw in (dict(q=q.half()), dict(q=torch.randn(1, 8, 1, 256).bfloat16().cuda()[..., ::2]),
               dict(q=q[:, :4]), dict(q=q.cpu()), dict(page_table=t.long()), dict(page_table=t[0]),
               dict(page_table=t.expand(2, -1)), dict(idx=idx[:, :1]), dict(idx=idx.long()), dict(idx=idx.transpose(1, 2)),
               dict(head_map=_i([0])), dict(head_map=torch.tensor([0, 1], device="cuda")), dict(kv_lens=_i([7, 7])),
               dict(lse=lse[:, ::2]), dict(lse=lse.half()), dict(o=q.float()), dict(o=q[:, :4])):
        with pytest.raises(kc.KascadeError):
            call(**kw)


def test_rows_past_four_gigabytes():
    """Pages whose byte offsets pass 32 bits."""
    kc = _kc()
    hkv, d, page, block = 8, 128, 64, 64
    num = 70000                        # 4.6 GB each for K and V
    kind = "e4m3"
    cache = kc.Q8Cache(*(torch.zeros(num, hkv, page, d, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
                         for _ in range(2)), torch.zeros(num, hkv, 1, 2, device="cuda"))
    rows = [[num - 1, 0, num - 2, 66000, 65535, 65536]]
    lens = [6 * page - 5]
    g = torch.Generator().manual_seed(1)
    x = torch.randn(2, lens[0], hkv, d, generator=g).bfloat16().cuda()
    slots = [rows[0][j // page] * page + j % page for j in range(lens[0])]
    kc.q8_append(cache, x[0], x[1], _i(slots))
    small = kc.Q8Cache(*(p.view(torch.uint8)[_i(rows[0]).long()].contiguous().view(torch.float8_e4m3fn)
                         for p in (cache.k_pages, cache.v_pages)), cache.scales[_i(rows[0]).long()].contiguous())
    srows = [list(range(6))]
    hc = held(small, kind)
    k, v = kc.q8_gather(cache, _i(rows), lens[0])
    ks, vs = kc.q8_gather(small, _i(srows), lens[0])
    assert torch.equal(k, ks) and torch.equal(v, vs)
    # within a rounding of what was put in: e4m3's half step, 2^-4, of each value or of the block's smallest steps
    err = (k[0].transpose(0, 1).float() - x[0].float()).abs()
    top = small.scales.max().item() * 2.0 ** -10
    assert (err <= x[0].float().abs() * (2.0 ** -4 + 2.0 ** -8) + top).all()
    s = kc.Shape.make(1, 32, hkv, d, 1, lens[0])
    q = torch.randn(1, 32, 1, d, generator=g).bfloat16().cuda()
    lse = torch.empty(1, 32, device="cuda")
    o = kc.sparse_decode_q8(s, q, cache, _i(rows), lse=lse)
    check_decode("far", q.view(1, 32, d).double().cpu().numpy(), hc, srows, lens, None,
                 o.view(1, 32, d).double().cpu().numpy(), lse.double().cpu().numpy(), torch.bfloat16)
