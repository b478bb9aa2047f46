"""The 8-bit cache's calls together, as a decode loop runs them: prompts and
steps through page tables and appends, an anchor layer's selection on gathered
rows, reuse layers on the cache; the same in captured graphs and on streams."""
import numpy as np
import pytest
import torch

import oracle as O
from oracle import q8_oracle as Q
from q8_cases import check_decode, held

pytestmark = pytest.mark.gpu

I32 = torch.int32


def _kc():
    from sparse_attention_long_anchor_b200 import kascade as kc
    return kc


def _i(v):
    return torch.tensor(v, dtype=I32, device="cuda")


@pytest.mark.parametrize("dtype", [torch.float8_e4m3fn, torch.int8])
def test_decode_loop(dtype):
    """Four requests: ragged prompts, then steps; every step appends, an anchor
    selects on the gathered rows, and a reuse layer attends over its lists."""
    kc = _kc()
    kind = "e4m3" if dtype is torch.float8_e4m3fn else "int8"
    B, hq, hkv, d, page, block, n = 4, 8, 2, 128, 64, 16, 512
    frac, num = (20, 100), 30
    cache = kc.Q8Cache.empty(num, hkv, d, page, block, dtype)
    g = torch.Generator().manual_seed(0)
    free = torch.randperm(num, generator=g).int().cuda()
    table = torch.full((B, n // page), -1, dtype=I32, device="cuda")
    lens = _i([0] * B)
    kv, used = [0] * B, 0
    s = kc.Shape.make(B, hq, hkv, d, 1, n, frac)
    ws = kc.Workspace(s, (kc.OP_SPARSE_DECODE_Q8, kc.OP_SELECT_VARLEN))
    hm = [1, 0]
    truth = [[[], []] for _ in range(B)]
    for new in ([300, 1, 64, 129], [1] * 4, [1] * 4, [70, 1, 0, 200], [1] * 4):
        cap = sum(new) + 5
        lens, offsets, slots, info = kc.page_tables(page, lens, _i(new), free[used:].contiguous(), table, cap)
        used += info.tolist()[0]
        x = torch.randn(cap, 2, hkv, d, generator=g).bfloat16().cuda()
        kc.q8_append(cache, x[:, 0], x[:, 1], slots, ws=ws)
        off = offsets.tolist()
        for b in range(B):
            for w in range(2):
                truth[b][w].append(x[off[b]:off[b + 1], w].float().cpu())
        kv = [a + b for a, b in zip(kv, new)]
        assert lens.tolist() == kv and off[-1] == sum(new)
        k, v = kc.q8_gather(cache, table, n, lens, ws=ws)
        # what comes back is what went in, within the cache's precision
        for b in range(B):
            for w, out in enumerate((k, v)):
                want = torch.cat(truth[b][w]).transpose(0, 1)
                got = out[b, :, :kv[b]].float().cpu()
                big = want.abs().amax()
                # a row may be rounded once for each scale of its block (at most 3 here: normal values
                # of a block differ by less than 2^3 in their largest); int8: half a step of amax / 63.5
                step = want.abs() * 2.0 ** -4 + big * 2.0 ** -9 if kind == "e4m3" else big / 63.5 / 2
                assert ((got - want).abs() <= 3 * step + want.abs() * 2.0 ** -8).all()
        q = (1.5 * torch.randn(B, hq, 1, d, generator=g)).bfloat16().cuda()
        idx = kc.select_varlen(s, q, k, lens, ws=ws)
        kk = O.topk_count(n, *frac)
        rows = idx.view(B, hkv, kk).cpu().numpy()
        lists = [[rows[b, h, :O.topk_count(kv[b], *frac)] for h in range(hkv)] for b in range(B)]
        lse = torch.empty(B, hq, device="cuda")
        o = kc.sparse_decode_q8(s, q, cache, table, idx, _i(hm), kv_lens=lens, lse=lse, ws=ws)
        torch.cuda.synchronize()
        assert ws.error() == 0
        check_decode("loop", q.view(B, hq, d).double().cpu().numpy(), held(cache, kind), table.tolist(), kv, lists,
                     o.view(B, hq, d).double().cpu().numpy(), lse.double().cpu().numpy(), torch.bfloat16, hm)


def test_equals_the_bf16_cache_where_that_holds_the_same_values():
    """A cache of values that bf16 holds exactly: the 8-bit attention against
    the bf16 call over the gathered rows, both within the bf16 call's tolerance
    of the oracle (2e-2 largest, 2e-3 mean), so within twice that of each other."""
    kc = _kc()
    from q8_cases import random_cache, tables_for
    n, hq, hkv, d, page = 3001, 32, 8, 128, 64
    rows, _ = tables_for([n, n], page, 48, 100, 2)
    cache = random_cache(kc, 100, hkv, page, d, 64, "e4m3", 5)
    t = _i(rows)
    k, v = kc.q8_gather(cache, t, n)
    s = kc.Shape.make(2, hq, hkv, d, 1, n, (10, 100))
    ws = kc.Workspace(s, (kc.OP_SELECT, kc.OP_SPARSE_DECODE, kc.OP_SPARSE_DECODE_Q8))
    q = torch.randn(2, hq, 1, d, generator=torch.Generator().manual_seed(9)).bfloat16().cuda()
    idx = kc.select(s, q, k, ws=ws)
    err = (kc.sparse_decode(s, q, k, v, idx, ws=ws).float() - kc.sparse_decode_q8(s, q, cache, t, idx, ws=ws).float()).abs()
    assert err.max() <= 4e-2 and err.mean() <= 4e-3
    err = (kc.dense_ref(s, q, k, v, causal=False).float() - kc.sparse_decode_q8(s, q, cache, t, ws=ws).float()).abs()
    assert err.max() <= 4e-2 and err.mean() <= 4e-3


def test_captured_steps_replay():
    """One captured graph of a whole step (tables, append, gather, attention),
    replayed with new inputs in its buffers, against the same calls made
    eagerly; two graphs share one workspace and run one after the other."""
    kc = _kc()
    B, hq, hkv, d, page, n, num = 3, 8, 2, 64, 16, 2048, 500

    def fresh():
        c = kc.Q8Cache.empty(num, hkv, d, page, page)
        return dict(cache=c, table=torch.full((B, n // page), -1, dtype=I32, device="cuda"), lens=_i([0] * B))
    s = kc.Shape.make(B, hq, hkv, d, 1, n)
    ws = kc.Workspace(s, (kc.OP_SPARSE_DECODE_Q8,))
    cap = 640
    buf = dict(new=_i([0] * B), free=torch.zeros(num, dtype=I32, device="cuda"),
               x=torch.zeros(cap, 2, hkv, d, dtype=torch.bfloat16, device="cuda"),
               q=torch.zeros(B, hq, 1, d, dtype=torch.bfloat16, device="cuda"))

    def step(st):
        lens, off, slots, info = kc.page_tables(page, st["lens"], buf["new"], buf["free"], st["table"], cap)
        kc.q8_append(st["cache"], buf["x"][:, 0], buf["x"][:, 1], slots, ws=ws)
        st["lens"].copy_(lens)
        k, v = kc.q8_gather(st["cache"], st["table"], n, st["lens"], ws=ws)
        o = kc.sparse_decode_q8(s, buf["q"], st["cache"], st["table"], kv_lens=st["lens"], ws=ws)
        return o, k, v, info
    warm = fresh()
    step(warm)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        st = fresh()
        st["graph"] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(st["graph"]):
            st["out"] = step(st)
        graphs.append(st)
    eager = fresh()
    g = torch.Generator().manual_seed(3)
    order = torch.randperm(num, generator=g).int()
    used = 0
    for new in ([200, 17, 300], [1, 1, 1], [0, 1, 33], [1, 1, 1]):
        buf["new"].copy_(torch.tensor(new, dtype=I32))
        buf["free"][:num - used].copy_(order[used:])
        buf["x"].copy_(torch.randn(cap, 2, hkv, d, generator=g))
        buf["q"].copy_(torch.randn(B, hq, 1, d, generator=g))
        want = step(eager)
        for st in graphs:
            st["graph"].replay()
        torch.cuda.synchronize()
        used += want[3].tolist()[0]
        for st in graphs:
            for a, b in zip(st["out"], want):
                assert torch.equal(a, b)
            assert torch.equal(st["table"], eager["table"]) and torch.equal(st["lens"], eager["lens"])
            assert torch.equal(st["cache"].scales, eager["cache"].scales)
    assert ws.error() == 0


def test_streams_and_two_calls_at_once():
    """Calls on streams of the caller's, each with buffers that the call makes,
    two at a time with workspaces of their own."""
    kc = _kc()
    from q8_cases import random_cache
    cache = random_cache(kc, 200, 2, 64, 128, 64, "int8", 6)
    t = _i([list(range(200))])
    s = kc.Shape.make(1, 8, 2, 128, 1, 12000)
    q = torch.randn(1, 8, 1, 128, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    ref = kc.sparse_decode_q8(s, q, cache, t)
    rk, rv = kc.q8_gather(cache, t, 12000, _i([11111]))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for _ in range(10):
        for st in streams:
            outs.append(kc.sparse_decode_q8(s, q, cache, t, stream=st))
            outs.append(kc.sparse_decode_q8(s, q, cache, t, stream=st.cuda_stream))
        outs.append(kc.sparse_decode_q8(s, q, cache, t))
        outs.append(kc.sparse_decode_q8(s, q, cache, t, stream=0))
    k, v = kc.q8_gather(cache, t, 12000, _i([11111]), stream=streams[0])
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)
    assert torch.equal(k, rk) and torch.equal(v, rv)
    # the order on one stream holds: append, then the attention that reads it
    c2 = kc.Q8Cache.empty(4, 2, 128, 64, 64, torch.int8)
    x = torch.randn(100, 2, 128, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    s2 = kc.Shape.make(1, 8, 2, 128, 1, 100)
    lens, table = _i([0]), _i([[-1, -1]])
    free, new = _i([2, 3]), _i([100])
    torch.cuda.synchronize()
    with torch.cuda.stream(streams[1]):
        lens, _, slots, _ = kc.page_tables(64, lens, new, free, table, 100)
        kc.q8_append(c2, x, x, slots)
        o = kc.sparse_decode_q8(s2, q, c2, table, kv_lens=lens)
    torch.cuda.synchronize()
    assert table.tolist() == [[2, 3]]
    hv = held(c2, "int8")
    want, _, _, _ = Q.attend(q[0, :4, 0].double().cpu().numpy(), Q.rows_of(hv[0], hv[2], 0, [2, 3], 0, 100),
                             Q.rows_of(hv[1], hv[2], 1, [2, 3], 0, 100))
    # (bf16's half step of values up to 4, and the weights' fp16 rounding)
    assert np.abs(o[0, :4, 0].double().cpu().numpy() - want).max() <= 4 * 2.0 ** -8


def test_calls_from_two_host_threads():
    """The library is entered from several threads at once (the binding's calls
    release the interpreter lock), on streams and workspaces of their own."""
    import threading
    kc = _kc()
    from q8_cases import random_cache
    cache = random_cache(kc, 200, 2, 64, 128, 64, "e4m3", 6)
    t = _i([list(range(200))])
    shapes = [kc.Shape.make(1, 8, 2, 128, 1, n) for n in (100, 3000, 12000)]
    q = torch.randn(1, 8, 1, 128, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    refs = [kc.sparse_decode_q8(s, q, cache, t) for s in shapes]
    torch.cuda.synchronize()
    got, bad = [], []

    def work():
        try:
            st = torch.cuda.Stream()
            for _ in range(20):
                for s, ref in zip(shapes, refs):
                    got.append((kc.sparse_decode_q8(s, q, cache, t, stream=st), ref))
            st.synchronize()
        except Exception as exc:   # noqa: BLE001  (reported below, from the test's own thread)
            bad.append(exc)
    threads = [threading.Thread(target=work) for _ in range(4)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    assert not bad, bad
    assert len(got) == 240 and all(torch.equal(o, ref) for o, ref in got)


def test_a_first_call_inside_a_capture():
    """A process whose first call of each kind is captured."""
    import subprocess
    import sys
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = """
import torch
from sparse_attention_long_anchor_b200 import kascade as kc
i = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
c = kc.Q8Cache.empty(40, 2, 128, 64)
kv, new, free, table = i([0]), i([2000]), i(list(range(40))), i([[-1] * 40])
x = torch.randn(2000, 2, 128, device="cuda").bfloat16()
s = kc.Shape.make(1, 8, 2, 128, 1, 2560)
q = torch.randn(1, 8, 1, 128, device="cuda").bfloat16()
ws = kc.Workspace(s, (kc.OP_SPARSE_DECODE_Q8,))
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    lens, _, slots, info = kc.page_tables(64, kv, new, free, table, 2000)
    kc.q8_append(c, x, x, slots)
    o = kc.sparse_decode_q8(s, q, c, table, kv_lens=lens, ws=ws)
    k, v = kc.q8_gather(c, table, 2560, lens)
g.replay()
torch.cuda.synchronize()
want = kc.sparse_decode_q8(s, q, c, table, kv_lens=i([2000]))
assert info.tolist() == [32, 2000] and torch.equal(o, want) and (o != 0).any() and ws.error() == 0
print("captured")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stdout + r.stderr
