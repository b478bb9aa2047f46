"""The 8-bit paged KV cache's operators: what is timed, on which sizes, and their plain forms.

Four operators, which a decode step of a Kascade stack runs one after the other: page tables and slot maps from
request lengths, the append that quantises new K and V rows into pages, attention of one query token over the
cache (an anchor's index lists, or every key), and the gather that hands the cache's rows to selection and prefill.

A cache is k and v pages [num_pages, Hkv, P, d] of 8-bit values (e4m3 or int8) and scales
[num_pages, Hkv, P / S, 2] in fp32: one (K, V) pair for each S consecutive rows of a page and head.
"""
import math
import random

import torch

own = False   # False: the plain forms below; True: the framework's calls

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32,
         "e4m3": torch.float8_e4m3fn, "int8": torch.int8}
TOP = {"e4m3": 448.0, "int8": 127.0}
E_MIN, E_MAX = -100, 122   # exponents a block's scale may take
POOL = 3   # pages beside those that the requests hold


def listed():
    return [
        # one decode step of eight 64K sequences: a slot each, now and then a page
        dict(name="tables_step_b8", op="tables", batch=8, page=64, kv_max=65536, new_max=1, step=True),
        # admission of a batch of prompts beside running requests, ragged
        dict(name="tables_prompts_b256", op="tables", batch=256, page=64, kv_max=4096, new_max=2048, step=False),
        # the largest batch of requests, pages of 16, chunks of up to 512 tokens
        dict(name="tables_chunks_b2048", op="tables", batch=2048, page=16, kv_max=8192, new_max=509, step=False),
        # the rows of a decode step of eight sequences
        dict(name="append_step_b8", op="append", batch=8, kv_max=65536, new_max=1, hkv=8, d=128, page=64, block=64,
             cache="e4m3", dtype="bf16", step=True),
        # a 32K prompt's K and V of one Llama-shaped layer
        dict(name="append_prompt_32k", op="append", batch=1, kv_max=0, new_max=32768, hkv=8, d=128, page=64, block=64,
             cache="e4m3", dtype="bf16", step=False),
        # ragged chunks behind running contexts, int8 with small blocks, fp32 rows of 64
        dict(name="append_chunks_int8", op="append", batch=13, kv_max=3001, new_max=517, hkv=2, d=64, page=32, block=16,
             cache="int8", dtype="fp32", step=False),
        # the smallest stack: one layer's reuse attention over 10 % of 2048 keys
        dict(name="decode_b1_h8_n2k", op="decode", batch=1, hq=8, hkv=2, d=64, n_ctx=2048, num=10, den=100, mode=0,
             page=64, block=64, cache="e4m3", q="bf16", ragged=False),
        # Llama-shaped reuse layer, batch 1, 32K keys
        dict(name="decode_llama8b_n32k", op="decode", batch=1, hq=32, hkv=8, d=128, n_ctx=32768, num=10, den=100,
             mode=0, page=64, block=64, cache="e4m3", q="bf16", ragged=False),
        # eight sequences of 64K, 10 % lists
        dict(name="decode_llama8b_b8_n64k", op="decode", batch=8, hq=32, hkv=8, d=128, n_ctx=65536, num=10, den=100,
             mode=0, page=64, block=64, cache="e4m3", q="bf16", ragged=False),
        # dense attention of a ragged batch up to 64K (no index lists), int8, fp16 queries
        dict(name="decode_dense_b8_n64k", op="decode", batch=8, hq=32, hkv=8, d=128, n_ctx=65535, num=0, den=1, mode=0,
             page=128, block=32, cache="int8", q="fp16", ragged=True),
        # rows of one long-prompt sequence for a rolling chunk
        dict(name="gather_b1_n5000", op="gather", batch=1, hkv=8, d=128, n_ctx=5000, page=64, block=64, cache="e4m3",
             out="bf16", ragged=True),
        # every row of eight 32K sequences for an anchor layer's selection
        dict(name="gather_b8_n32k", op="gather", batch=8, hkv=8, d=128, n_ctx=32768, page=128, block=32, cache="int8",
             out="bf16", ragged=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(["tables", "append", "decode", "decode", "gather"])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "tables":
        step = rng.random() < 0.4
        new = 1 if step else _log(rng, 2, 1024)
        batch = _log(rng, 1, min(2048, 1024 * 1024 // new))
        return dict(op=op, batch=batch, page=page, kv_max=_log(rng, 16, 65536 if batch < 256 else 8192), new_max=new,
                    step=step)
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8])
    block = 1 << rng.randint(0, page.bit_length() - 1)
    cache = rng.choice(["e4m3", "int8"])
    if op == "append":
        step = rng.random() < 0.5
        batch = _log(rng, 1, 64)
        new = 1 if step else _log(rng, 2, 32768 // batch)
        block = max(block, 4)
        return dict(op=op, batch=batch, kv_max=_log(rng, 16, 8192), new_max=new, hkv=hkv, d=d, page=page, block=block,
                    cache=cache, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]), step=step)
    if op == "gather":
        out = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        return dict(op=op, batch=_log(rng, 1, 4 if out == "fp32" else 8), hkv=hkv, d=d, n_ctx=_log(rng, 100, 32768),
                    page=page, block=block, cache=cache, out=out, ragged=rng.random() < 0.5)
    num, den = rng.choice([(5, 100), (10, 100), (20, 100), (0, 1)])
    mode = rng.choice([0, 0, 1]) if num else 0
    return dict(op=op, batch=_log(rng, 1, 8 if num and not mode else 3), hq=hkv * rng.choice([1, 2] if mode else [1, 2, 4, 4, 8]),
                hkv=hkv, d=d, n_ctx=_log(rng, 100, 65535), num=num, den=den, mode=mode, page=page, block=block,
                cache=cache, q=rng.choice(["bf16", "bf16", "fp16"]), ragged=rng.random() < 0.5)


# ---------------------------------------------------------------- sizes

def _lens(c, most):
    """Context lengths of a ragged batch: evenly spread up to `most` (the order is the seed's)."""
    if not c.get("ragged", True):
        return [most] * c["batch"]
    return [max(1, most * (i + 1) // c["batch"]) for i in range(c["batch"])]


def _requests(c):
    """(tokens held, tokens new) of each request, in an order that the seed shuffles."""
    n = c["batch"]
    kv = [c["kv_max"] * (2 * i + 1) // (2 * n) for i in range(n)]
    new = [1] * n if c["step"] else [c["new_max"] * (n - i) // n for i in range(n)]
    return list(zip(kv, new))


def _lists(c):
    return c["hq"] if c["mode"] == 1 else c["hkv"]


def _count(c, n):
    return -(-c["num"] * n // c["den"]) if c["num"] else n


def work(c):
    if c["op"] == "tables":
        r = _requests(c)
        pages = sum(-(-(a + b) // c["page"]) - -(-a // c["page"]) for a, b in r)
        cap = c["batch"] * c["new_max"]
        # lengths and free pages in; table entries, lengths, offsets and slots out
        return {"bytes": 4 * (2 * c["batch"] + pages + pages + 2 * c["batch"] + 1 + cap + 2), "flops": 0}
    if c["op"] == "append":
        t = sum(b for _, b in _requests(c))
        blocks = sum((a + b - 1) // c["block"] - a // c["block"] + 1 for a, b in _requests(c) if b)
        w = TYPES[c["dtype"]].itemsize
        return {"bytes": 2 * t * c["hkv"] * c["d"] * (w + 1) + blocks * c["hkv"] * 16 + 4 * t,
                "flops": 4 * t * c["hkv"] * c["d"]}
    lens = _lens(c, c["n_ctx"])
    pages = sum(-(-n // c["page"]) for n in lens)
    if c["op"] == "gather":
        w = TYPES[c["out"]].itemsize
        blocks = sum(-(-n // c["block"]) for n in lens)
        return {"bytes": 2 * sum(lens) * c["hkv"] * c["d"] * (w + 1) + blocks * c["hkv"] * 8 + 4 * pages,
                "flops": 2 * sum(lens) * c["hkv"] * c["d"]}
    keys = sum(_count(c, n) for n in lens)   # of one list
    blocks = sum(min(_count(c, n), -(-n // c["block"])) for n in lens)
    heads = _lists(c)                        # rows are read once for each list that names them
    rows = heads if c["num"] else c["hkv"]
    return {"bytes": keys * rows * (2 * c["d"] + (4 if c["num"] else 0)) + blocks * rows * 8 + 4 * pages
            + c["batch"] * c["hq"] * (4 * c["d"] + 4), "flops": 4 * keys * c["hq"] * c["d"]}


# ---------------------------------------------------------------- inputs

def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _pow2(amax, cache):
    """The smallest power of two s with amax <= top s, by the exponent and fraction of amax."""
    m, e = torch.frexp(amax.double())        # amax = m 2^e, m in [0.5, 1)
    top_m, top_e = math.frexp(TOP[cache])
    e = e - top_e + (m > top_m).to(e.dtype)
    e = torch.where(amax > 0, e, torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX)
    return torch.ldexp(torch.ones_like(m), e)


def _to8(y, cache):
    """fp32 values rounded to the cache's type, saturated."""
    if cache == "e4m3":
        return y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return torch.nan_to_num(y, nan=0.0, posinf=127.0, neginf=-127.0).round().clamp(-127, 127).to(torch.int8)


def _cache_rows(c, g, num_pages):
    """One tensor's pages and block scales: normal rows, every 37th an outlier, as long contexts have them."""
    x = torch.randn(num_pages, c["hkv"], c["page"], c["d"], generator=g, device=DEV)
    x[:, :, ::37] *= 3.0
    xb = x.view(num_pages, c["hkv"], c["page"] // c["block"], c["block"], c["d"])
    s = _pow2(xb.abs().amax((3, 4)), c["cache"]).float()
    x8 = _to8(xb.div_(s[..., None, None]), c["cache"]).view(x.shape)
    return x8, s


def _paged(c, g, lens):
    """A cache that holds `lens` tokens of each request on shuffled pages, and its page table."""
    per = [-(-n // c["page"]) for n in lens]
    total = sum(per) + POOL
    k8, ks = _cache_rows(c, g, total)
    v8, vs = _cache_rows(c, g, total)
    table = torch.full((len(lens), max(per) + 1), -1, dtype=torch.int32)
    order = torch.randperm(total, generator=g, device=DEV).cpu().int()
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
    return dict(k=k8, v=v8, scales=torch.stack([ks, vs], -1).contiguous(), table=table.to(DEV), free=order[at:].to(DEV))


def prepare(c, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 17)
    rng = random.Random(int(seed) * 104729 + 5)
    s = dict(case=c)
    if c["op"] in ("tables", "append"):
        reqs = _requests(c)
        rng.shuffle(reqs)
        page = c["page"]
        per = [-(-(a + b) // page) for a, b in reqs]
        held = [-(-a // page) for a, _ in reqs]
        s.update(kv=_ints([a for a, _ in reqs]), new=_ints([b for _, b in reqs]))
        total, width = sum(per) + POOL, max(per) + 2
        order = torch.randperm(total, generator=g, device=DEV).int()
        ids = order.cpu().tolist()
        rows, at = [], 0
        for h in held:
            rows.append(ids[at:at + h] + [-1] * (width - h))
            at += h
        s.update(table=_ints(rows), free=order[at:].contiguous(), cap=c["batch"] * c["new_max"])
        if c["op"] == "append":
            # the step's slots, as the tables give them, and K, V as views of the layer's fused projection
            slots, nxt = [], at
            for (a, b), h, row in zip(reqs, held, rows):
                for i in range(h, -(-(a + b) // page)):
                    row[i] = ids[nxt]
                    nxt += 1
                slots += [row[p // page] * page + p % page for p in range(a, a + b)]
            t, h = len(slots), c["hkv"]
            qkv = torch.randn(t, 3, h, c["d"], generator=g, device=DEV)
            qkv[::29] *= 4.0
            qkv = qkv.to(TYPES[c["dtype"]])
            k8, ks = _cache_rows(c, g, total)
            v8, vs = _cache_rows(c, g, total)
            s.update(slots=_ints(slots), x=qkv[:, 1], y=qkv[:, 2], k=k8, v=v8,
                     scales=torch.stack([ks, vs], -1).contiguous())
    else:
        lens = _lens(c, c["n_ctx"])
        rng.shuffle(lens)
        s.update(_paged(c, g, lens), lens=_ints(lens))
        if c["op"] == "gather":
            shape = (c["batch"], c["hkv"], c["n_ctx"], c["d"])
            s.update(out_k=torch.zeros(shape, dtype=TYPES[c["out"]], device=DEV),
                     out_v=torch.zeros(shape, dtype=TYPES[c["out"]], device=DEV))
        else:
            s["q"] = (1.5 * torch.randn(c["batch"], c["hq"], 1, c["d"], generator=g, device=DEV)).to(TYPES[c["q"]])
            s["idx"] = s["map"] = None
            if c["num"]:
                n_lists, kk = _lists(c), _count(c, c["n_ctx"])
                idx = torch.full((c["batch"], n_lists, kk), -1, dtype=torch.int32, device=DEV)
                for b, n in enumerate(lens):   # ascending lists of distinct keys, then -1
                    k = _count(c, n)
                    pick = torch.rand(n_lists, n, generator=g, device=DEV).topk(k).indices
                    idx[b, :, :k] = pick.sort().values.int()
                s["idx"] = idx
                s["map"] = _ints([rng.randrange(n_lists) for _ in range(n_lists)])
    if own:
        from sparse_attention_long_anchor_b200 import kascade as kc
        if c["op"] != "tables":
            s["cache"] = kc.Q8Cache(s["k"], s["v"], s["scales"])
        if c["op"] == "decode":
            dt = {"bf16": kc.DTYPE_BF16, "fp16": kc.DTYPE_F16}[c["q"]]
            s["shape"] = kc.Shape.make(c["batch"], c["hq"], c["hkv"], c["d"], 1, c["n_ctx"],
                                       (c["num"], c["den"]) if c["num"] else (1, 1), mode=c["mode"], dtype=dt)
            s["ws"] = kc.Workspace(s["shape"], (kc.OP_SPARSE_DECODE_Q8,))
    return s


# ---------------------------------------------------------------- the operators

def run(s):
    if own:
        from sparse_attention_long_anchor_b200 import kascade as kc
        return _OWN[s["case"]["op"]](kc, s)
    return _PLAIN[s["case"]["op"]](s)


def _own_tables(kc, s):
    lens, offsets, slots, info = kc.page_tables(s["case"]["page"], s["kv"], s["new"], s["free"], s["table"], s["cap"])
    return s["table"], lens, offsets, slots, info


def _own_append(kc, s):
    kc.q8_append(s["cache"], s["x"], s["y"], s["slots"])
    return s["k"], s["v"], s["scales"]


def _own_decode(kc, s):
    c = s["case"]
    lse = torch.empty(c["batch"], c["hq"], device=DEV)
    o = kc.sparse_decode_q8(s["shape"], s["q"], s["cache"], s["table"], s["idx"], s["map"], kv_lens=s["lens"],
                            lse=lse, ws=s["ws"])
    return o, lse


def _own_gather(kc, s):
    return kc.q8_gather(s["cache"], s["table"], s["case"]["n_ctx"], s["lens"], k=s["out_k"], v=s["out_v"])


_OWN = dict(tables=_own_tables, append=_own_append, decode=_own_decode, gather=_own_gather)


def _plain_tables(s):
    page, cap = s["case"]["page"], s["cap"]
    kv, new, free, table = s["kv"].long(), s["new"].long(), s["free"].long(), s["table"].clone()
    n, width = table.shape
    first = (kv + page - 1) // page
    need = (kv + new + page - 1) // page - first
    zero = torch.zeros(1, dtype=torch.long, device=DEV)
    at, pg = torch.cat([zero, new.cumsum(0)]), torch.cat([zero, need.cumsum(0)])
    ok = (kv >= 0).all() & (new >= 0).all() & (kv + new <= width * page).all() & (at[-1] <= cap) & (pg[-1] <= free.numel())
    col = torch.arange(width, device=DEV)[None]
    rank = col - first[:, None]
    fresh = (rank >= 0) & (rank < need[:, None]) & ok
    taken = free[(pg[:-1, None] + rank).clamp(0, max(0, free.numel() - 1))] if free.numel() else torch.zeros_like(rank)
    table = torch.where(fresh, taken.int(), table)
    t = torch.arange(cap, device=DEV)
    b = torch.searchsorted(at[1:].contiguous(), t, right=True).clamp(max=n - 1)
    pos = (kv[b] + t - at[b]).clamp(0, width * page - 1)
    slot = table[b, pos // page].long() * page + pos % page
    slots = torch.where((t < at[-1]) & ok, slot, -1).int()
    lens = torch.where(ok, kv + new, kv).int()
    info = torch.where(ok, torch.stack([pg[-1], at[-1]]), torch.tensor([-1, 0], device=DEV)).int()
    return table, lens, torch.where(ok, at, 0).int(), slots, info


def _plain_append(s):
    c = s["case"]
    block, cache = c["block"], c["cache"]
    slots = s["slots"].long()
    blk = slots // block
    lead = torch.cat([torch.ones(1, dtype=torch.bool, device=DEV), blk[1:] != blk[:-1]])
    run_of = lead.cumsum(0) - 1              # the run of each token: neighbours in one block
    starts = slots[lead]
    n, per = starts.numel(), c["page"] // block
    page, in_page = starts // c["page"], starts % c["page"] // block
    offset = starts % block                  # rows of the block that were there before
    scales = s["scales"].view(-1, c["hkv"], per, 2).clone()
    outs = []
    for which, (x, pages) in enumerate(((s["x"], s["k"]), (s["y"], s["v"]))):
        x = x.float()
        amax = torch.where(x.isfinite(), x.abs(), 0.0).amax(-1)
        most = torch.zeros(n, c["hkv"], device=DEV).scatter_reduce_(0, run_of[:, None].expand(-1, c["hkv"]), amax, "amax")
        new = _pow2(most, cache).float()
        old = scales[page, :, in_page, which]
        new = torch.where(offset[:, None] > 0, torch.maximum(old, new), new)
        scales[page, :, in_page, which] = new
        p = pages.view(torch.uint8).view(-1, c["hkv"], per, block, c["d"]).clone()
        rows = p[page, :, in_page]           # [runs, heads, block, d]
        wide = rows.view(TYPES[cache]).float() * (old / new)[..., None, None]
        before = torch.arange(block, device=DEV)[None, :] < offset[:, None]
        grown = before[:, None, :, None] & (new > old)[..., None, None]
        p[page, :, in_page] = torch.where(grown, _to8(wide, cache).view(torch.uint8), rows)
        p = p.view(-1, c["hkv"], c["page"], c["d"])
        p[slots // c["page"], :, slots % c["page"]] = _to8(x / new[run_of][..., None], cache).view(torch.uint8)
        outs.append(p.view(TYPES[cache]))
    return outs[0], outs[1], scales.view(s["scales"].shape)


def _rows(s, keys, heads):
    """Row numbers of `keys` [B, L, n] for kv heads `heads` [L] in the pages taken as one list of rows."""
    page, hkv = s["case"]["page"], s["case"]["hkv"]
    table = s["table"].long()
    pg = torch.gather(table[:, None].expand(-1, keys.shape[1], -1), 2, keys // page)
    return (pg * hkv + heads[None, :, None]) * page + keys % page


def _dequantised(s, pages, which, rows):
    c = s["case"]
    x = pages.view(torch.uint8).view(-1, c["d"])[rows].view(TYPES[c["cache"]]).float()
    return x * s["scales"].view(-1, 2)[:, which][rows // c["block"]][..., None]


def _plain_decode(s):
    c = s["case"]
    bsz, hq, hkv, d, group = c["batch"], c["hq"], c["hkv"], c["d"], c["hq"] // c["hkv"]
    n_lists = _lists(c)
    lens = s["lens"].long()
    if c["num"]:
        keys = s["idx"].long()[:, s["map"].long()]
        count = (c["num"] * lens + c["den"] - 1) // c["den"]
    else:
        keys = torch.arange(c["n_ctx"], device=DEV).expand(bsz, n_lists, -1)
        count = lens
    n = keys.shape[-1]
    live = torch.arange(n, device=DEV)[None] < count[:, None]
    keys = torch.where(live[:, None], keys, 0)
    heads = torch.arange(n_lists, device=DEV) // (n_lists // hkv)
    rows = _rows(s, keys, heads)
    q = s["q"].float().view(bsz, n_lists, hq // n_lists, d)
    scores = torch.matmul(q, _dequantised(s, s["k"], 0, rows).transpose(-1, -2)) / math.sqrt(d)
    scores = scores.masked_fill(~live[:, None, None], float("-inf"))
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, _dequantised(s, s["v"], 1, rows)) / total
    return o.view(bsz, hq, 1, d).to(s["q"].dtype), (top + total.log()).view(bsz, hq)


def _plain_gather(s):
    c = s["case"]
    lens = s["lens"].long()
    keys = torch.arange(c["n_ctx"], device=DEV).expand(c["batch"], c["hkv"], -1)
    live = keys < lens[:, None, None]
    rows = _rows(s, torch.where(live, keys, 0), torch.arange(c["hkv"], device=DEV))
    return [torch.where(live[..., None], _dequantised(s, pages, which, rows).to(out.dtype), out)
            for which, (pages, out) in enumerate(((s["k"], s["out_k"]), (s["v"], s["out_v"])))]


_PLAIN = dict(tables=_plain_tables, append=_plain_append, decode=_plain_decode, gather=_plain_gather)


# ---------------------------------------------------------------- in 64 bits

def _nearest8(y, cache):
    """Doubles to the nearest value of the 8-bit type, ties to even, by the spacing of the values around each."""
    if cache == "int8":
        return torch.clamp(torch.round(torch.nan_to_num(y, nan=0.0)), -127.0, 127.0)
    _, e = torch.frexp(y)
    step = torch.ldexp(torch.ones_like(y), (e - 1).clamp(min=-6) - 3)
    return torch.clamp(torch.round(y / step) * step, -448.0, 448.0)


def _scale_of(most, cache):
    """The block scale of a largest magnitude, by trying exponents around its logarithm."""
    if most <= 0.0:
        return 2.0 ** E_MIN
    e = math.floor(math.log2(most / TOP[cache])) - 1
    while most > TOP[cache] * 2.0 ** e:
        e += 1
    return 2.0 ** min(max(e, E_MIN), E_MAX)


def exact(c, seed):
    if c["op"] == "tables":
        return None                          # whole numbers only
    s = prepare(c, seed)
    if c["op"] == "append":
        return _exact_append(c, s)
    ids, lens = s["table"].cpu().tolist(), s["lens"].cpu().tolist()

    def held(pages, which, b, h, n):
        """Head h's first n rows of request b, in doubles."""
        pg = torch.tensor(ids[b][:-(-n // c["page"])], device=DEV)
        x = pages[pg, h].double().reshape(-1, c["d"])[:n]
        sc = s["scales"][pg, h, :, which].double().repeat_interleave(c["block"], 1).reshape(-1)[:n]
        return x * sc[:, None]

    if c["op"] == "gather":
        shape = (c["batch"], c["hkv"], c["n_ctx"], c["d"])
        outs = [torch.zeros(shape, dtype=torch.float64, device=DEV) for _ in range(2)]
        for b, n in enumerate(lens):
            for h in range(c["hkv"]):
                for which, pages in enumerate((s["k"], s["v"])):
                    outs[which][b, h, :n] = held(pages, which, b, h, n)
        return outs
    o = torch.zeros(c["batch"], c["hq"], 1, c["d"], dtype=torch.float64, device=DEV)
    lse = torch.zeros(c["batch"], c["hq"], dtype=torch.float64, device=DEV)
    heads_map = s["map"].cpu().tolist() if c["num"] else None
    group = c["hq"] // c["hkv"]
    for b, n in enumerate(lens):
        for h in range(c["hkv"]):
            k, v = held(s["k"], 0, b, h, n), held(s["v"], 1, b, h, n)
            for qh in range(h * group, (h + 1) * group):
                kk, vv = k, v
                if c["num"]:
                    entry = heads_map[qh if c["mode"] == 1 else h]
                    pick = s["idx"][b, entry, :_count(c, n)].long()
                    kk, vv = k[pick], v[pick]
                x = (kk @ s["q"][b, qh, 0].double()) / math.sqrt(c["d"])
                lse[b, qh] = torch.logsumexp(x, 0)
                o[b, qh, 0] = torch.exp(x - lse[b, qh]) @ vv
    return o, lse


def _exact_append(c, s):
    slots = s["slots"].cpu().tolist()
    runs, i = [], 0
    while i < len(slots):
        j = i + 1
        while j < len(slots) and slots[j] // c["block"] == slots[i] // c["block"]:
            j += 1
        runs.append((i, j))
        i = j
    if len(runs) * c["hkv"] > 12000:
        return None                          # too many blocks for this way of going through them
    k, v, scales = s["k"].double().cpu(), s["v"].double().cpu(), s["scales"].double().cpu()
    for which, (x, pages) in enumerate(((s["x"], k), (s["y"], v))):
        x = x.double().cpu()
        for i, j in runs:
            page, row = divmod(slots[i], c["page"])
            cell, offset = divmod(row, c["block"])
            most = x[i:j].abs().amax((0, 2)).tolist()
            for h in range(c["hkv"]):
                new, old = _scale_of(most[h], c["cache"]), float(scales[page, h, cell, which])
                if offset:
                    new = max(new, old)
                    if new > old:
                        pages[page, h, row - offset:row] = _nearest8(pages[page, h, row - offset:row] * (old / new), c["cache"])
                scales[page, h, cell, which] = new
                pages[page, h, row:row + j - i] = _nearest8(x[i:j, h] / new, c["cache"])
    whole = c["cache"] == "int8"
    return (None if whole else k), (None if whole else v), scales
