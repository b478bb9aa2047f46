"""Attention over keys whose scores are minus infinity: they have no weight."""
import math

import numpy as np
import pytest
import torch

from oracle import q8_oracle as Q
from q8_cases import attention_bound, held, lse_bound, random_cache, tables_for

pytestmark = pytest.mark.gpu


def _kc():
    from sparse_attention_long_anchor_b200 import kascade as kc
    return kc


def _i(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# a CTA to a list, clusters, shares found on the device, waves; keys of minus infinity in front, behind, all but one
@pytest.mark.parametrize("batch,n", [(1, 90), (1, 3000), (8, 5000), (40, 900)])
@pytest.mark.parametrize("kind,d", [("e4m3", 128), ("int8", 64)])
@pytest.mark.parametrize("where", ["front", "behind", "most", "all"])
def test_keys_of_minus_infinity_have_no_weight(batch, n, kind, d, where):
    kc = _kc()
    hq, hkv, page, block = 4, 2, 64, 1
    lens = [n - 7 * (b % 5) for b in range(batch)]
    width = -(-n // page)
    rows, _ = tables_for(lens, page, width, batch * width + 1, n)
    cache = random_cache(kc, batch * width + 1, hkv, page, d, block, kind, d)
    # positive queries; the lost keys are negative in every dim, with an infinite scale
    q = torch.rand(batch, hq, 1, d, generator=torch.Generator().manual_seed(n)).bfloat16().cuda() + 0.125
    one = 0xb8 if kind == "e4m3" else 0xff          # -1
    lost = []
    table = torch.tensor(rows)
    for b, m in enumerate(lens):
        at = {"front": range(m * 7 // 10), "behind": range(m // 3, m), "most": [j for j in range(m) if j != m // 2],
              "all": range(m)}[where]
        lost.append(np.array(list(at)))
        pg, r = table[b, lost[b] // page].cuda(), torch.from_numpy(lost[b] % page).cuda()
        cache.k_pages.view(torch.uint8)[pg, :, r] = one
        sc = cache.scales[..., 0]
        sc[pg, :, r] = float("inf")
    s = kc.Shape.make(batch, hq, hkv, d, 1, n)
    lse = torch.empty(batch, hq, device="cuda")
    ws = kc.Workspace(s, (kc.OP_SPARSE_DECODE_Q8,))
    o = kc.sparse_decode_q8(s, q, cache, _i(rows), kv_lens=_i(lens), lse=lse, ws=ws)
    torch.cuda.synchronize()
    assert ws.error() == 0
    kval, vval, sc = held(cache, kind)
    o, lse, qd = o.view(batch, hq, d).double().cpu().numpy(), lse.double().cpu().numpy(), q.view(batch, hq, d).double().cpu().numpy()
    v_top, s_top = np.nanmax(np.abs(vval)), np.abs(sc[..., 1]).max()
    for b in range(0, batch, 7):
        keep = np.setdiff1d(np.arange(lens[b]), lost[b])
        for h in range(hq):
            if len(keep) == 0:
                assert np.isnan(o[b, h]).all() and lse[b, h] == -math.inf   # 0 / 0, log 0
                continue
            pg, r = np.array(rows[b])[keep // page], keep % page
            k = kval[pg, h // 2, r] * sc[pg, h // 2, r, 0][:, None]
            v = vval[pg, h // 2, r] * sc[pg, h // 2, r, 1][:, None]
            want, wl, mv, mqk = Q.attend(qd[b, h:h + 1], k, v)
            err = np.abs(o[b, h] - want[0])
            assert (err <= attention_bound(torch.bfloat16, d, lens[b], want[0], mv[0], mqk, v_top, s_top)).all(), (b, h)
            assert abs(lse[b, h] - wl[0]) <= lse_bound(d, lens[b], wl[0], mqk), (b, h)
