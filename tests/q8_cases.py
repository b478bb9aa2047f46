"""Helpers of the 8-bit cache tests: caches with known contents and the
bounds that the kernels' roundings give."""
from __future__ import annotations

import numpy as np
import torch

from oracle import q8_oracle as Q

KINDS = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}   # eps / 2


def raw(t: torch.Tensor) -> np.ndarray:
    """A tensor's bytes."""
    return t.detach().contiguous().view(torch.uint8).cpu().numpy()


def held(cache, kind):
    """(K values, V values, scales) of a Q8Cache as numpy."""
    return (Q.decode_bytes(raw(cache.k_pages), kind), Q.decode_bytes(raw(cache.v_pages), kind),
            cache.scales.cpu().numpy().astype(np.float64))


def random_cache(kc, num_pages, hkv, page, d, block, kind, seed, scale="pow2", device="cuda"):
    """A cache of normal values: scales as the append writes them, or any
    ("free": not powers of two, V's over a factor of 2^12)."""
    g = torch.Generator().manual_seed(seed)
    cache = kc.Q8Cache.empty(num_pages, hkv, d, page, block, KINDS[kind], device=device)
    top = 448.0 if kind == "e4m3" else 127.0
    blocks = page // block
    for which, pages in enumerate((cache.k_pages, cache.v_pages)):
        x = torch.randn(num_pages, hkv, blocks, block, d, generator=g)
        amax = x.abs().amax((3, 4))
        if scale == "pow2":
            s = torch.exp2(torch.ceil(torch.log2(amax / top)))
        else:
            s = amax / top
        y = (x / s[..., None, None]).clamp(-top, top)
        y = y.to(torch.float8_e4m3fn) if kind == "e4m3" else y.round().to(torch.int8)
        if scale == "free" and which == 1:
            s = s * torch.exp2(12 * torch.rand(s.shape, generator=g) - 6)
        pages.copy_(y.view(num_pages, hkv, page, d).to(device))
        cache.scales[..., which] = s.to(device)
    return cache


def tables_for(lens, page, width, num_pages, seed):
    """Shuffled distinct pages for each request (host lists); unused entries
    are out of the pool, so that reading one is an error."""
    g = torch.Generator().manual_seed(seed)
    order = torch.randperm(num_pages, generator=g).tolist()
    rows, at = [], 0
    for n in lens:
        per = -(-n // page)
        rows.append(order[at:at + per] + [num_pages + 17] * (width - per))
        at += per
    return rows, order[at:]


def attention_bound(dtype, d, n, o, mass_v, mass_qk, v_top, two_e):
    """Largest error of one output row.

    * the output is rounded once: half a step of `dtype` relative (and half of
      fp16's smallest step, 2^-25);
    * p vs is rounded to fp16, 2^-11 relative, or by half of its smallest step
      2^-24 in units of 2^(E - 14), 2^E <= the largest |vs|, each times |v8|;
    * scores carry d products and sums in fp32 and a few factors: (d + 8)
      2^-24 of sum |q k| / sqrt(d), which moves p and the sum by that relative;
      exp2 and the sums add (n / 16 + 64) 2^-24 at most (a warp adds at most
      n / 16 slices one after the other)."""
    u = HALF_STEP[dtype]
    ds = (d + 8) * 2.0 ** -24 * mass_qk
    rel = 2.0 ** -11 + 2 * ds * (1 + ds) + 2 * (n / 16 + 64) * 2.0 ** -24
    inner = rel * mass_v + n * 2.0 ** -25 * two_e * 2.0 ** -14 * v_top
    return u * (np.abs(o) + inner) + inner + (2.0 ** -25 if dtype is torch.float16 else 1e-38)


def lse_bound(d, n, lse, mass_qk):
    """The same score and sum errors on the logarithm, and its own rounding
    (the sum of two fp32 terms of that size, each off by a few half steps)."""
    return (d + 8) * 2.0 ** -24 * mass_qk + (n / 16 + 64) * 2.0 ** -24 + 4 * 2.0 ** -24 * (np.abs(lse) + mass_qk + 1)


def check_decode(case, q, held_cache, tables, lens, lists, o, lse, dtype, head_map=None, per_head=False):
    """o [B, Hq, d], lse [B, Hq] against the oracle over the cache's values.
    lists: None (dense) or [B][L] lists of keys."""
    kval, vval, scales = held_cache
    bsz, hq, d = q.shape
    hkv = kval.shape[1]
    group = hq // hkv
    v_top = np.nanmax(np.abs(vval))
    for b in range(bsz):
        n = lens[b]
        for h in range(hkv):
            if n:
                k = Q.rows_of(kval, scales, 0, tables[b], h, n)
                v = Q.rows_of(vval, scales, 1, tables[b], h, n)
            else:
                k = v = np.zeros((0, d))
            for qh in range(h * group, (h + 1) * group):
                kk, vv = k, v
                if lists is not None:
                    entry = qh if per_head else h
                    if len(lists[b]) == 1:
                        entry = 0
                    elif head_map is not None:
                        entry = head_map[entry]
                    pick = np.asarray(lists[b][entry], dtype=np.int64) if 0 <= entry < len(lists[b]) else np.zeros(0, np.int64)
                    kk, vv = k[pick], v[pick]
                want, wl, mv, mqk = Q.attend(q[b, qh:qh + 1], kk, vv)
                if len(kk) == 0:
                    assert (o[b, qh] == 0).all() and lse[b, qh] == -np.inf, (case, b, qh)
                    continue
                top_scale = np.abs(scales[..., 1]).max() if np.isfinite(scales).all() else 1.0
                err = np.abs(o[b, qh] - want[0])
                tol = attention_bound(dtype, d, len(kk), want[0], mv[0], mqk, v_top, top_scale)
                assert (err <= tol).all(), (case, b, qh, float((err / tol).max()))
                assert abs(lse[b, qh] - wl[0]) <= lse_bound(d, len(kk), wl[0], mqk), (case, b, qh, lse[b, qh], wl[0])
