"""The 8-bit cache on the CPU: its index arithmetic (compiled from the
library's header with the host compiler), what the C entry points refuse, what
the binding refuses, and the oracle against torch's conversions."""
import ctypes
import math
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from oracle import q8_oracle as Q

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "sparse_attention_long_anchor_b200", "csrc")


def _kc():
    from sparse_attention_long_anchor_b200 import kascade as kc
    return kc


# ---------------------------------------------------------------- index arithmetic

def _run(tmp_path, body):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    src = tmp_path / "t.cpp"
    src.write_text('#include <cstdio>\n#include <cstring>\n#include "q8_index.h"\nusing namespace kascade;\n'
                   "int main() {\n%s\n  return 0;\n}\n" % body)
    exe = tmp_path / "t"
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-fsanitize=undefined", "-I", CSRC, str(src), "-o",
                    str(exe)], check=True)
    return subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()


def test_pages_keys_and_slots_out_of_range_are_caught(tmp_path):
    pages = [0, 6, 7, -1, -2**31, 2**31 - 1]
    keys = [0, 9, 10, -1, -2**31, 2**31 - 1]
    slots = [0, 7 * 32 - 1, 7 * 32, -1, -2**31, 2**31 - 1]
    body = ["bool b;"]
    for p in pages:
        body.append('b = false; { const uint32_t r = q8_page((int32_t)(%dLL), 7, b); std::printf("%%u %%d\\n", r, (int)b); }' % p)
    for k in keys:
        body.append('b = false; { const int r = q8_key((int32_t)(%dLL), 10, b); std::printf("%%d %%d\\n", r, (int)b); }' % k)
    for s in slots:
        body.append('std::printf("%%d\\n", (int)q8_slot_ok((int32_t)(%dLL), 7, 5));' % s)
    out = list(map(int, _run(tmp_path, "\n".join(body))))
    assert out[:12] == [0, 0, 6, 0, 0, 1, 0, 1, 0, 1, 0, 1]
    assert out[12:24] == [0, 0, 9, 0, 9, 1, 0, 1, 0, 1, 9, 1]
    assert out[24:] == [1, 1, 0, 0, 0, 0]


def test_rows_stay_inside_the_pool(tmp_path):
    """The last row of the largest pools is the last row number, below 2^31."""
    pools = [(1, 1, 4), (7, 8, 6), (131071, 8, 11), (524287, 1, 12), (1 << 20, 8, 7)]
    body = ['std::printf("%%u\\n", q8_row(%du - 1, (1u << %d) - 1u, %d - 1, %d, %d));' % (n, ps, h, h, ps)
            for n, h, ps in pools]
    out = list(map(int, _run(tmp_path, "\n".join(body))))
    assert out == [n * h * (1 << ps) - 1 for n, h, ps in pools]
    assert max(out) < 2 ** 31


def test_owner_skips_empty_requests(tmp_path):
    sizes = [[3], [0, 0, 4, 0, 1, 0], [1] * 9, [5, 0], [0, 1], [2, 0, 0, 0, 7]]
    body, want = [], []
    for i, s in enumerate(sizes):
        pre = [0]
        for x in s:
            pre.append(pre[-1] + x)
        body.append("const int p%d[] = {%s};" % (i, ", ".join(map(str, pre))))
        for x in range(pre[-1]):
            body.append('std::printf("%%d\\n", q8_owner(p%d, %d, %d));' % (i, len(s), x))
            want.append(next(b for b in range(len(s)) if pre[b] <= x < pre[b + 1]))
    assert list(map(int, _run(tmp_path, "\n".join(body)))) == want


def test_list_lengths_by_reciprocal(tmp_path):
    """ceil(n num / den) at and around every kind of border, up to the largest
    lengths and budgets that a call takes."""
    top = 1 << 20
    rng = np.random.default_rng(0)
    cases = [(n, num, den) for den in (1, 2, 3, 7, 10, 100, 255, 256, 4099, 99991, top - 1, top)
             for num in {1, den, max(1, den // 3), max(1, den - 1)} for n in (0, 1, 2, den - 1, den, min(den + 1, top), 3277, 65535, top - 1, top)]
    for _ in range(3000):
        den = int(rng.integers(1, top + 1))
        num = int(rng.integers(1, den + 1))
        n = int(rng.integers(0, top + 1))
        k = int(rng.integers(0, top * num // den + 1))          # n num a multiple of den, or next to one
        cases += [(n, num, den), (min(top, k * den // num), num, den), (min(top, k * den // num + 1), num, den)]
    cases = [c for c in cases if c[1] <= c[2] <= top and c[0] <= top]
    body = ["static const int c[][3] = {%s};" % ", ".join("{%d,%d,%d}" % c for c in cases),
            'for (auto& x : c) std::printf("%d\\n", q8_count(x[0], x[1], x[2], q8_reciprocal(x[2])));']
    got = list(map(int, _run(tmp_path, "\n".join(body))))
    assert got == [-(-n * num // den) for n, num, den in cases]


def test_scale_exponents(tmp_path):
    vals = [0.0, 1.0, 448.0, 448.0 * (1 + 2 ** -20), 447.9, 127.0, 127.0 * (1 + 2 ** -20), 126.9, 3e38, 1e-44, 2.0 ** -95,
            2.0 ** -130, 1e30, 0.3]
    vals = [float(np.float32(v)) for v in vals]
    body = ["float f; unsigned u;"]
    for v in vals:
        for t in (0, 1):
            body.append('f = (float)%r; std::memcpy(&u, &f, 4); std::printf("%%d\\n", q8_scale_exp(u, %d));' % (v, t))
    out = iter(map(int, _run(tmp_path, "\n".join(body))))
    for v in vals:
        for kind in ("e4m3", "int8"):
            assert 2.0 ** next(out) == Q.scale_for(v, kind), (v, kind)


# ---------------------------------------------------------------- oracle

def test_oracle_values_and_rounding_match_torch():
    vals = Q.e4m3_values()
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(vals), np.isnan(t)) and np.array_equal(vals[~np.isnan(vals)], t[~np.isnan(t)])
    g = torch.Generator().manual_seed(3)
    x = torch.cat([torch.randn(4000, generator=g) * 10.0 ** torch.randint(-4, 3, (4000,), generator=g),
                   torch.tensor(vals[:127]).float(), (torch.tensor(vals[:126]) + torch.tensor(vals[1:127])).float() / 2])
    x = torch.cat([x, -x]).clamp(-448, 448)
    assert np.array_equal(Q.nearest(x.numpy(), "e4m3"), x.to(torch.float8_e4m3fn).double().numpy())
    assert Q.nearest(np.array([1e9, -1e9, math.inf]), "e4m3").tolist() == [448.0, -448.0, 448.0]
    assert math.isnan(Q.nearest(np.array([math.nan]), "e4m3")[0])
    y = x.double() / 3
    assert np.array_equal(Q.nearest(y.numpy(), "int8"), y.round().clamp(-127, 127).numpy())
    assert Q.nearest(np.array([0.5, 1.5, -2.5, 127.5, math.nan]), "int8").tolist() == [0.0, 2.0, -2.0, 127.0, 0.0]


# ---------------------------------------------------------------- refusals

def _cache(kc, **kw):
    f = dict(k_pages=256, v_pages=256, scales=256, num_pages=10, num_kv_heads=2, head_dim=64, page_size=64,
             scale_block=16, type=0)
    f.update(kw)
    return kc._Q8CacheArgs(**f)


BAD_CACHES = [
    (dict(num_pages=0), 1), (dict(num_kv_heads=0), 1), (dict(k_pages=None), 1), (dict(v_pages=None), 1),
    (dict(scales=None), 1), (dict(head_dim=96), 2), (dict(head_dim=0), 2), (dict(page_size=8, scale_block=8), 2),
    (dict(page_size=48), 2), (dict(page_size=8192), 2), (dict(scale_block=0), 2), (dict(scale_block=24), 2),
    (dict(scale_block=128), 2), (dict(page_size=1024, scale_block=512), 2), (dict(type=2), 2), (dict(type=-1), 2),
    (dict(k_pages=264), 2), (dict(v_pages=257), 2), (dict(scales=260), 2), (dict(num_pages=2**31 - 1), 2),
    (dict(num_pages=2**25, num_kv_heads=1), 2), (dict(num_kv_heads=65536), 2),
]


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_bad_caches_are_refused(bad, status):
    kc = _kc()
    L = kc.lib
    c = ctypes.byref(_cache(kc, **bad))
    hkv, d = bad.get("num_kv_heads", 2), bad.get("head_dim", 64)
    s = ctypes.byref(kc.Shape.make(1, max(hkv, 1), max(hkv, 1), d if d in (64, 128) else 64, 1, 100))
    assert L.kascade_q8_append(c, 256, 256, 64, 64, 64, 64, 0, 4, 256, None, 0, None) == status
    assert L.kascade_q8_gather(c, 1, 100, 256, 1 << 20, None, 0, 256, 256, None, 0, None) == status
    assert L.kascade_sparse_decode_q8(s, c, 256, 256, 1 << 20, None, None, None, 256, None, 256, 1 << 30, None) == status
    assert L.kascade_q8_append(None, 256, 256, 64, 64, 64, 64, 0, 4, 256, None, 0, None) == kc.ERR_INVALID_ARG


def test_append_refusals():
    kc = _kc()
    f = kc.lib.kascade_q8_append
    c = ctypes.byref(_cache(kc))
    assert f(c, 256, 256, 64, 64, 64, 64, 0, 0, None, None, 0, None) == kc.OK       # no tokens: nothing to do
    assert f(c, 256, 256, 64, 64, 64, 64, 0, -1, 256, None, 0, None) == kc.ERR_INVALID_ARG
    assert f(c, None, 256, 64, 64, 64, 64, 0, 4, 256, None, 0, None) == kc.ERR_INVALID_ARG
    assert f(c, 256, None, 64, 64, 64, 64, 0, 4, 256, None, 0, None) == kc.ERR_INVALID_ARG
    assert f(c, 256, 256, 64, 64, 64, 64, 0, 4, None, None, 0, None) == kc.ERR_INVALID_ARG
    assert f(c, 256, 256, 64, 64, 64, 64, 3, 4, 256, None, 0, None) == kc.ERR_UNSUPPORTED
    assert f(c, 258, 256, 64, 64, 64, 64, 0, 4, 256, None, 0, None) == kc.ERR_UNSUPPORTED
    assert f(c, 256, 256, 64, 64, 64, 64, 0, 4, 258, None, 0, None) == kc.ERR_UNSUPPORTED
    for bad in ((68, 64, 64, 64), (64, 66, 64, 64), (64, 64, 65, 64), (64, 64, 64, 4)):
        assert f(c, 256, 256, *bad, 0, 4, 256, None, 0, None) == kc.ERR_UNSUPPORTED
    assert f(c, 256, 256, 66, 64, 64, 64, 1, 4, 256, None, 0, None) == kc.ERR_UNSUPPORTED
    assert f(c, 256, 256, 64, 64, 64, 64, 0, 1 << 30, 256, None, 0, None) == kc.ERR_UNSUPPORTED   # rows are numbered in 31 bits


def test_gather_refusals():
    kc = _kc()
    f = kc.lib.kascade_q8_gather
    c = ctypes.byref(_cache(kc))
    ok = (1, 100, 256, 2, None, 0, 256, 256, None, 0, None)

    def but(**kw):
        names = ("batch", "n", "table", "width", "lens", "dtype", "k", "v", "ws", "nb", "st")
        return f(c, *[kw.get(n, v) for n, v in zip(names, ok)])
    assert but(batch=0) == but(n=0) == but(table=None) == but(k=None, v=None) == but(width=1) == kc.ERR_INVALID_ARG
    assert but(n=65, width=1) == kc.ERR_INVALID_ARG
    assert but(dtype=3) == but(table=258) == but(lens=258) == but(k=264) == but(v=264) == kc.ERR_UNSUPPORTED
    assert but(n=(1 << 20) + 1, width=1 << 20) == kc.ERR_UNSUPPORTED
    assert but(batch=1 << 20, n=1 << 20, width=1 << 20) == kc.ERR_UNSUPPORTED       # more CTAs than a grid holds


def test_decode_refusals():
    kc = _kc()
    f = kc.lib.kascade_sparse_decode_q8
    s = kc.Shape.make(1, 8, 2, 64, 1, 256)
    need = kc.workspace_bytes(s, kc.OP_SPARSE_DECODE_Q8)
    c = _cache(kc)

    def call(shape=s, cache=c, q=256, table=256, width=4, lens=None, idx=None, hm=None, o=256, lse=None, ws=256,
             nb=need):
        return f(ctypes.byref(shape), ctypes.byref(cache), q, table, width, lens, idx, hm, o, lse, ws, nb, None)
    assert call(q=None) == call(o=None) == call(table=None) == call(width=3) == kc.ERR_INVALID_ARG
    for kw in (dict(q=264), dict(o=264), dict(table=258), dict(lens=258), dict(idx=258), dict(hm=258), dict(lse=258)):
        assert call(**kw) == kc.ERR_UNSUPPORTED
    assert call(ws=None, nb=0) == call(nb=need - 1) == call(ws=258) == kc.ERR_WORKSPACE
    assert call(shape=kc.Shape.make(1, 8, 2, 64, 256, 256)) == kc.ERR_UNSUPPORTED            # prefill
    assert call(shape=kc.Shape.make(1, 8, 2, 64, 1, 256, dtype=kc.DTYPE_F32)) == kc.ERR_UNSUPPORTED
    assert call(shape=s.with_flags(kc.FLAG_CHECK_INDICES)) == kc.ERR_UNSUPPORTED
    assert call(shape=kc.Shape.make(1, 8, 4, 64, 1, 256)) == kc.ERR_INVALID_ARG             # another Hkv than the cache's
    assert call(shape=kc.Shape.make(1, 8, 2, 128, 1, 256)) == kc.ERR_INVALID_ARG
    assert call(shape=kc.Shape.make(1, 32, 2, 64, 1, 256)) == kc.ERR_UNSUPPORTED            # G > 8


def test_page_tables_refusals():
    kc = _kc()
    f = kc.lib.kascade_page_tables
    names = ("batch", "page", "width", "kv", "new", "free", "nfree", "table", "out", "off", "slots", "cap", "info", "st")
    ok = (4, 64, 8, 4096, 8192, 12288, 3, 16384, 20480, 24576, 28672, 10, 32768, None)

    def but(**kw):
        return f(*[kw.get(n, v) for n, v in zip(names, ok)])
    for kw in (dict(batch=0), dict(width=0), dict(nfree=-1), dict(cap=-1), dict(kv=None), dict(new=None), dict(free=None),
               dict(table=None), dict(out=None), dict(off=None), dict(slots=None), dict(info=None),
               dict(out=4096), dict(out=8192), dict(table=8192), dict(kv=16384 + 4 * 31), dict(out=4108), dict(off=4096), dict(info=8192), dict(slots=4096 - 36)):
        assert but(**kw) == kc.ERR_INVALID_ARG, kw
    for kw in (dict(batch=4097), dict(page=48), dict(page=8), dict(page=8192), dict(kv=4098), dict(table=16386)):
        assert but(**kw) == kc.ERR_UNSUPPORTED, kw


def test_workspace_of_the_q8_decode():
    kc = _kc()
    op = kc.OP_SPARSE_DECODE_Q8
    small = kc.Shape.make(1, 8, 2, 64, 1, 16)
    assert kc.workspace_bytes(small, op) == 256                 # one CTA per list: no partial results
    s = kc.Shape.make(8, 32, 8, 128, 1, 65536)
    assert 256 < kc.workspace_bytes(s, op) < 64 << 20 and kc.workspace_bytes(s, op) % 256 == 0
    assert kc.workspace_bytes(kc.Shape.make(1, 8, 2, 64, 64, 64), op) == 0
    big = kc.Shape.make(64, 32, 8, 128, 1, 1 << 20)
    assert kc.workspace_bytes(big, op) < 2 << 30


def test_binding_refuses_wrong_tensors():
    kc = _kc()
    f8, i8 = torch.float8_e4m3fn, torch.int8

    def pages(dtype=f8, shape=(4, 2, 32, 64)):
        return torch.zeros(shape, dtype=torch.uint8).view(dtype)
    sc = torch.zeros(4, 2, 2, 2)
    c = kc.Q8Cache(pages(), pages(), sc)
    assert (c.num_pages, c.num_kv_heads, c.page_size, c.head_dim, c.scale_block) == (4, 2, 32, 64, 16)
    for bad in ((pages(torch.uint8), pages(torch.uint8), sc), (pages(), pages(i8), sc), (pages(), pages(), sc.double()),
                (pages(), pages(shape=(5, 2, 32, 64)), sc), (pages(), pages(), torch.zeros(4, 2, 2)),
                (pages(), pages(), torch.zeros(4, 2, 3, 2)), (pages(), pages(), torch.zeros(4, 2, 2, 4)[..., ::2]),
                (pages().transpose(1, 2), pages().transpose(1, 2), sc)):
        with pytest.raises(kc.KascadeError):
            kc.Q8Cache(*bad)
    with pytest.raises(kc.KascadeError):
        kc.Q8Cache.empty(4, 2, 64, 32, 24, device="cpu")
    i32 = torch.int32
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    slots = torch.zeros(3, dtype=i32)
    for bad in ((x[:, :1], x, slots), (x, x.half(), slots), (x.double(), x.double(), slots),
                (x.transpose(1, 2).contiguous().transpose(1, 2), x, slots)):
        with pytest.raises(kc.KascadeError):
            kc.q8_append(c, *bad)
    # tensors of the host: every call says so before it reaches the library
    with pytest.raises(kc.KascadeError):
        kc.q8_append(c, x, x, slots)
    with pytest.raises(kc.KascadeError):
        kc.q8_gather(c, torch.zeros(1, 4, dtype=i32), 100)
    with pytest.raises(kc.KascadeError):
        kc.page_tables(32, slots, slots, slots, torch.zeros(3, 4, dtype=i32), 8)
    with pytest.raises(kc.KascadeError):
        kc.sparse_decode_q8(kc.Shape.make(1, 8, 2, 64, 1, 100), torch.zeros(1, 8, 1, 64, dtype=torch.bfloat16), c,
                            torch.zeros(1, 4, dtype=i32))
