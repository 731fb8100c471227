"""The grouped-query cache operators as a decode loop calls them: what is timed and what their answers are.

Three operators share one paged cache of separate K and V rows ([pages, KV heads, page_size, head_dim], a page table
of [request rows, logical pages]): the write of new rows, the attention of one new token per request over its cached
rows (with the weight that every row received, where the caller accumulates it), and the eviction of the rows that
received least.  ``own`` chooses between the plain torch form and the library's entry points.
"""
import math

import torch

own = False

_KINDS = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
_GOLDEN = 0.6180339887498949


# ---------------------------------------------------------------- cases
def _decode(name, **kw):
    c = {"op": "decode", "q": "bf16", "kv": "bf16", "heads": 32, "kv_heads": 8, "dim": 128, "page": 256, "batch": 1,
         "lo": 1, "hi": 1, "window": 0, "sink": False, "weights": False, "token_major": False}
    return {"name": name, **c, **kw}


def _store(name, **kw):
    c = {"op": "store", "q": "bf16", "kv": "bf16", "kv_heads": 8, "dim": 128, "page": 256, "batch": 1, "tokens": 1,
         "start": 0, "tracked": False}
    return {"name": name, **c, **kw}


def _evict(name, **kw):
    c = {"op": "evict", "kv": "bf16", "kv_heads": 8, "dim": 128, "page": 256, "batch": 1, "lo": 2, "hi": 2, "keep": 1,
         "first": 0, "recent": 0, "aged": False}
    return {"name": name, **c, **kw}


def listed():
    return [
        # one user, a few hundred cached tokens: the launch latency of a decode step
        _decode("decode_one_short", lo=333, hi=333),
        # a serving batch of mixed lengths, the usual decode step
        _decode("decode_batch", batch=32, lo=2048, hi=32768),
        # two very long contexts: the split over the cache's length carries it
        _decode("decode_long", heads=64, batch=2, lo=131072, hi=131071 + 64, sink=True),
        # a large batch over a cache held in 8 bits
        _decode("decode_e4m3", kv="e4m3", heads=32, kv_heads=4, batch=64, lo=1024, hi=16384),
        # a decode step that also accumulates the weight each cached row receives
        _decode("decode_weights", batch=16, lo=2048, hi=16384, weights=True),
        # a small model: one query head per KV head, 64 wide, f16, small pages, ragged short lengths, sliding window
        _decode("decode_heads64_f16", q="f16", kv="f16", heads=16, kv_heads=16, dim=64, page=16, batch=48, lo=1,
                hi=2000, window=1024, token_major=True),
        # the write of a decode step: one new token per request
        _store("store_step", batch=64, tokens=1, start=1023, tracked=True),
        # the write of a prompt chunk, packed to 8 bits
        _store("store_prompt_e4m3", kv="e4m3", batch=64, tokens=1024, start=500, tracked=True),
        # a full cache gives up one row per head after each decode step
        _evict("evict_step", batch=64, lo=2049, hi=2049, keep=2048, first=4, recent=128, aged=True),
        # caches with a bound, trimmed every few hundred steps
        _evict("evict_trim_e4m3", kv="e4m3", batch=32, lo=4200, hi=5120, keep=4096, first=4, recent=256, aged=True),
        # long prompts cut to the rows worth keeping
        _evict("evict_prompt", batch=8, lo=20000, hi=32768, keep=4096, first=4, recent=512),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "decode", "store", "evict", "evict"])
    kv = rng.choice(["bf16", "bf16", "f16", "e4m3"])
    q = kv if kv != "e4m3" else rng.choice(["bf16", "f16"])
    dim = rng.choice([64, 128, 128, 256])
    hkv = rng.choice([1, 2, 3, 4, 8, 8, 16])
    page = rng.choice([16, 32, 64, 128, 256, 256])
    row = hkv * dim * (1 if kv == "e4m3" else 2) * 2
    if op == "decode":
        batch = _spread(rng, 1, 128)
        hi = _spread(rng, 1, max(2, min(131072, int(1.2e9 / (row * batch)))))
        lo = rng.choice([1, hi // 4 + 1, hi])
        group = rng.choice([1, 2, 4, 5, 7, 8, 8, 12, 16])
        return {"op": op, "q": q, "kv": kv, "heads": group * hkv, "kv_heads": hkv, "dim": dim, "page": page,
                "batch": batch, "lo": lo, "hi": hi, "window": rng.choice([0, 0, 0, hi // 2 + 1, 128]),
                "sink": rng.random() < 0.5, "weights": rng.random() < 0.4, "token_major": rng.random() < 0.3}
    if op == "store":
        batch = _spread(rng, 1, 128)
        return {"op": op, "q": q, "kv": kv, "kv_heads": hkv, "dim": dim, "page": page, "batch": batch,
                "tokens": _spread(rng, 1, max(2, min(4096, int(2e8 / (row * batch))))), "start": rng.randrange(0, 3000),
                "tracked": rng.random() < 0.5}
    batch = _spread(rng, 1, 64)
    hi = _spread(rng, 40, max(64, min(100000, int(5e8 / (row * batch)))))
    keep = max(1, int(hi * rng.choice([0.1, 0.5, 0.9, 0.99])))
    return {"op": op, "kv": kv, "kv_heads": hkv, "dim": dim, "page": page, "batch": batch, "lo": max(1, hi - hi // 5),
            "hi": hi, "keep": keep, "first": min(4, keep // 4), "recent": min(128, keep // 4),
            "aged": rng.random() < 0.5}


def _lens(case):
    """The batch's cached lengths: spread evenly over lo .. hi, in an order that the seed shuffles."""
    lo, hi, n = case["lo"], case["hi"], case["batch"]
    return [lo + int((hi - lo + 1) * ((0.31 + i * _GOLDEN) % 1.0)) for i in range(n)]


def _attended(case):
    w = case["window"]
    return [min(n, w) if w else n for n in _lens(case)]


# ---------------------------------------------------------------- inputs
def _rows(shape, kind, gen):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float16 if kind != "bf16" else torch.bfloat16)
    return x.to(_KINDS[kind])


def _cache(case, slots, gen):
    """K and V pools whose pages belong to the requests in random order, with a few pages that belong to nobody."""
    pages = -(-slots // case["page"])
    total = case["batch"] * pages + 3
    shape = (total, case["kv_heads"], case["page"], case["dim"])
    if case.get("token_major"):
        shape = (total, case["page"], case["kv_heads"], case["dim"])
    k, v = _rows(shape, case["kv"], gen), _rows(shape, case["kv"], gen)
    if case.get("token_major"):
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    order = torch.randperm(total, generator=gen, device="cuda")[: case["batch"] * pages]
    st = {"k": k, "v": v, "table": order.view(case["batch"], pages).to(torch.int32)}
    if case["kv"] == "e4m3":
        st["k_scale"] = 0.02 + 0.03 * torch.rand(case["kv_heads"], generator=gen, device="cuda")
        st["v_scale"] = 0.02 + 0.03 * torch.rand(case["kv_heads"], generator=gen, device="cuda")
        if case["op"] == "decode":   # codes around 1 stand for values around 1
            st["k_scale"], st["v_scale"] = st["k_scale"] * 25, st["v_scale"] * 25
    return st


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    b, hkv, dim = case["batch"], case["kv_heads"], case["dim"]
    if case["op"] == "decode":
        st = _cache(case, case["hi"], gen)
        lens = torch.tensor(_lens(case), dtype=torch.int32, device="cuda")
        st["lens"] = lens[torch.randperm(b, generator=gen, device="cuda")].contiguous()
        st["query"] = _rows((b, case["heads"], dim), case["q"], gen)
        st["sink"] = torch.randn(case["heads"], generator=gen, device="cuda") if case["sink"] else None
        st["weights"] = None
        if case["weights"]:
            width = st["table"].shape[1] * case["page"]
            st["weights"] = torch.rand(b, hkv, width, generator=gen, device="cuda")
            st["weights_out"] = torch.zeros_like(st["weights"])
        st["out"] = torch.empty_like(st["query"])
        st["lse"] = torch.empty(b, case["heads"], device="cuda")
        st["max_len"] = case["hi"]
    elif case["op"] == "store":
        slots = case["start"] + case["tokens"]
        st = _cache(case, slots, gen)
        n = b * case["tokens"]
        # K and V as the projection leaves them: one row of K and V heads per token
        st["kv_new"] = _rows((n, 2 * hkv, dim), case["q"], gen)
        req = torch.arange(b, device="cuda").repeat_interleave(case["tokens"])
        slot = torch.arange(case["start"], slots, device="cuda").repeat(b)
        st["req"], st["slots"] = req.to(torch.int32), slot.to(torch.int32)
        if case["tracked"]:
            width = st["table"].shape[1] * case["page"]
            st["weights"] = torch.rand(b, hkv, width, generator=gen, device="cuda")
            st["positions"] = torch.randint(0, 1 << 20, (b, hkv, width), generator=gen, device="cuda", dtype=torch.int32)
            st["token_positions"] = torch.randint(0, 1 << 20, (n,), generator=gen, device="cuda", dtype=torch.int32)
    else:
        st = _cache(case, case["hi"], gen)
        lens = torch.tensor(_lens(case), dtype=torch.int32, device="cuda")
        st["lens"] = lens[torch.randperm(b, generator=gen, device="cuda")].contiguous()
        width = st["table"].shape[1] * case["page"]
        # a few rows received nothing at all, most little, some much
        w = torch.exp(2.0 * torch.randn(b, hkv, width, generator=gen, device="cuda"))
        st["weights"] = w * (torch.rand(b, hkv, width, generator=gen, device="cuda") > 0.02)
        place = torch.arange(width, device="cuda").expand(b, hkv, width)
        if case["aged"]:   # after earlier evictions: any cached row may stand in any slot
            place = torch.rand(b, hkv, width, generator=gen, device="cuda")
            place = place.masked_fill(torch.arange(width, device="cuda") >= st["lens"][:, None, None], 2.0)
            place = 3 * place.argsort(dim=-1).argsort(dim=-1)
            st["seen"] = 3 * st["lens"]
        else:
            st["seen"] = st["lens"].clone()
        st["positions"] = place.to(torch.int32).contiguous()
        st["weights_out"] = torch.zeros_like(st["weights"])
        st["positions_out"] = torch.zeros_like(st["positions"])
        st["lens_out"] = torch.zeros_like(st["lens"])
        st["max_len"] = case["hi"]
    st["case"] = dict(case)
    return st


# ---------------------------------------------------------------- one pass
def _handle(st):
    """The cache descriptor and the workspace that a program keeps beside its pools."""
    from hybrid_sparse_mqa_gb300 import attn
    if "cache" not in st:
        c = st["case"]
        cache = attn.make_gqa_cache(st["k"], st["v"], st["table"], k_scale=st.get("k_scale"), v_scale=st.get("v_scale"))
        size = 0
        if c["op"] == "decode":
            size = attn.dsv4_gqa_decode_workspace_size(cache, c["batch"], c["heads"], st["max_len"], c["weights"])
        elif c["op"] == "evict":
            size = attn.dsv4_gqa_evict_workspace_size(cache, c["batch"], st["max_len"], c["keep"])
        st["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        st["cache"] = cache
    return attn, st["cache"]


def run(st):
    return {"decode": _run_decode, "store": _run_store, "evict": _run_evict}[st["case"]["op"]](st)


def _run_decode(st):
    c = st["case"]
    if own:
        attn, cache = _handle(st)
        attn.dsv4_gqa_decode(st["query"], st["lens"], cache, sink=st["sink"], window=c["window"],
                             max_len=st["max_len"], weights=st["weights"], weights_out=st.get("weights_out"),
                             out=st["out"], lse=st["lse"], workspace=st["workspace"])
        return [st["out"], st["lse"]] + ([st["weights_out"]] if c["weights"] else [])
    b, h, d = st["query"].shape
    hkv, ps = c["kv_heads"], c["page"]
    pages = -(-st["max_len"] // ps)
    table = st["table"][:, :pages].long()
    k = st["k"][table].transpose(1, 2).reshape(b, hkv, pages * ps, d).float()
    v = st["v"][table].transpose(1, 2).reshape(b, hkv, pages * ps, d).float()
    if "k_scale" in st:
        k, v = k * st["k_scale"][:, None, None], v * st["v_scale"][:, None, None]
    slot = torch.arange(pages * ps, device="cuda")
    n = st["lens"][:, None].long()
    seen = slot < n
    if c["window"]:
        seen = seen & (slot >= n - c["window"])
    seen = seen[:, None, None, :]
    v = v.masked_fill(~seen[:, 0, 0, :][:, None, :, None], 0.0)
    q = st["query"].float().view(b, hkv, h // hkv, d)
    s = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    s = s.masked_fill(~seen, -math.inf)
    top = s.amax(dim=-1, keepdim=True)
    if st["sink"] is not None:
        sink = st["sink"].view(1, hkv, h // hkv, 1)
        top = torch.maximum(top, sink)
    top = top.clamp_min(-1e30)
    p = torch.exp(s - top)
    total = p.sum(dim=-1, keepdim=True)
    if st["sink"] is not None:
        total = total + torch.exp(sink - top)
    p = p / total.clamp_min(1e-38)
    out = torch.matmul(p, v).reshape(b, h, d).to(st["query"].dtype)
    lse = (top + torch.log(total)).reshape(b, h)
    if not c["weights"]:
        return [out, lse]
    w_out = st["weights_out"]
    width = pages * ps
    got = st["weights"][:, :, :width] + p.sum(dim=2)
    live = (slot < n)[:, None, :]
    w_out[:, :, :width] = torch.where(live, got, w_out[:, :, :width])
    return [out, lse, w_out]


def _run_store(st):
    c = st["case"]
    hkv = c["kv_heads"]
    k_new, v_new = st["kv_new"][:, :hkv], st["kv_new"][:, hkv:]
    if own:
        attn, cache = _handle(st)
        attn.dsv4_gqa_store(k_new, v_new, st["req"], st["slots"], cache, weights=st.get("weights"),
                            positions=st.get("positions"), token_positions=st.get("token_positions"))
    else:
        req, slot = st["req"].long(), st["slots"].long()
        page, off = st["table"][req, slot // c["page"]].long(), slot % c["page"]
        if c["kv"] == "e4m3":
            k_new = (k_new.float() / st["k_scale"][:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
            v_new = (v_new.float() / st["v_scale"][:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
            st["k"].view(torch.uint8)[page, :, off] = k_new.view(torch.uint8)
            st["v"].view(torch.uint8)[page, :, off] = v_new.view(torch.uint8)
        else:
            st["k"][page, :, off] = k_new
            st["v"][page, :, off] = v_new
        if c["tracked"]:
            st["weights"][req, :, slot] = 0.0
            st["positions"][req, :, slot] = st["token_positions"][:, None].expand(-1, hkv)
    return [st["k"], st["v"]] + ([st["weights"], st["positions"]] if c["tracked"] else [])


def _run_evict(st):
    c = st["case"]
    keep = c["keep"]
    if own:
        attn, cache = _handle(st)
        attn.dsv4_gqa_evict(st["lens"], cache, st["weights"], keep, seq_lens=st["seen"], positions=st["positions"],
                            first=c["first"], recent=c["recent"], max_len=st["max_len"], weights_out=st["weights_out"],
                            positions_out=st["positions_out"], lens_out=st["lens_out"], workspace=st["workspace"])
        return [st["lens_out"], st["weights_out"], st["positions_out"], st["k"], st["v"]]
    width = st["max_len"]
    b, hkv = st["weights"].shape[:2]
    w, pos = st["weights"][:, :, :width], st["positions"][:, :, :width]
    slot = torch.arange(width, device="cuda")
    n = st["lens"].long()[:, None, None]
    live = (slot < n).expand(b, hkv, width)
    guarded = live & ((pos < c["first"]) | (pos >= st["seen"][:, None, None] - c["recent"]))
    w = w.masked_fill(torch.isnan(w), -math.inf)
    # rank: guarded rows, then the heavier row, then the lower slot
    order = w.argsort(dim=-1, descending=True, stable=True)
    kind = 2 * guarded.to(torch.int32) + live.to(torch.int32)
    second = kind.gather(-1, order).argsort(dim=-1, descending=True, stable=True)
    order = order.gather(-1, second)
    kept = torch.zeros_like(live).scatter_(-1, order[..., :keep], True) & live
    hole, mover = live & ~kept & (slot < keep) & (n > keep), kept & (slot >= keep)
    at_hole, at_mover = hole.nonzero(), mover.nonzero()     # both by request, head, slot: as many of each per head
    bi, hi, dst, src = at_hole[:, 0], at_hole[:, 1], at_hole[:, 2], at_mover[:, 2]
    ps = c["page"]
    to, of = st["table"][bi, dst // ps].long(), st["table"][bi, src // ps].long()
    k, v = (x.view(torch.uint8) if c["kv"] == "e4m3" else x for x in (st["k"], st["v"]))
    k[to, hi, dst % ps] = k[of, hi, src % ps]
    v[to, hi, dst % ps] = v[of, hi, src % ps]
    stays = slot < n.clamp_max(keep)
    for_out = ((st["weights"], st["weights_out"]), (st["positions"], st["positions_out"]))
    (wi, wo), (pi, po) = for_out
    wo[:, :, :width] = torch.where(stays, wi[:, :, :width], wo[:, :, :width])
    po[:, :, :width] = torch.where(stays, pi[:, :, :width], po[:, :, :width])
    wo[bi, hi, dst] = wi[bi, hi, src]
    po[bi, hi, dst] = pi[bi, hi, src]
    st["lens_out"].copy_(st["lens"].clamp_max(keep))
    return [st["lens_out"], wo, po, st["k"], st["v"]]


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    es = 1 if case["kv"] == "e4m3" else 2
    hkv, d = case["kv_heads"], case["dim"]
    if case["op"] == "decode":
        rows = sum(_attended(case))
        b, h = case["batch"], case["heads"]
        byts = rows * hkv * d * es * 2 + b * h * d * 2 * 2 + b * h * 4 + b * 4
        byts += 4 * sum(-(-n // case["page"]) for n in _attended(case))
        if case["weights"]:
            byts += 8 * hkv * sum(_lens(case))
        return {"bytes": byts, "flops": 4 * rows * h * d}
    if case["op"] == "store":
        n = case["batch"] * case["tokens"]
        byts = n * hkv * d * 2 * (2 + es) + 8 * n
        if case["tracked"]:
            byts += n * 4 + n * hkv * 8
        return {"bytes": byts, "flops": n * hkv * d * 2 if es == 1 else 0}
    keep, byts = case["keep"], 0.0
    for n in _lens(case):
        byts += hkv * 8.0 * n + 8
        moved = 0.0
        if n > keep:
            moved = keep * (n - keep) / n
            if not case["aged"]:   # the newest rows stand behind the bound and all move
                free = n - case["first"] - case["recent"]
                late = min(case["recent"], n - keep)
                moved = late + (keep - case["first"] - case["recent"]) * max(0, n - keep - late) / max(1, free)
        byts += hkv * (moved * d * es * 2 * 2 + 8.0 * min(n, keep))
    return {"bytes": byts, "flops": 0}


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    return {"decode": _exact_decode, "store": _exact_store, "evict": _exact_evict}[case["op"]](case, st)


def _request_rows(st, case, pool, b, n):
    """The first n rows of request b, [KV heads, n, dim] in 64 bits."""
    where = st["table"][b, : -(-n // case["page"])].long()
    return torch.cat(list(st[pool][where].double()), dim=1)[:, :n]


def _exact_decode(case, st):
    hkv, group, d = case["kv_heads"], case["heads"] // case["kv_heads"], case["dim"]
    out = torch.zeros(st["query"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(out.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    mass = st["weights_out"].double() if case["weights"] else None
    for b, n in enumerate(st["lens"].tolist()):
        first = max(0, n - case["window"]) if case["window"] else 0
        k, v = (_request_rows(st, case, x, b, n)[:, first:] for x in ("k", "v"))
        if mass is not None:
            mass[b, :, :n] = st["weights"][b, :, :n].double()
        for g in range(hkv):
            mine = slice(g * group, (g + 1) * group)
            logits = st["query"][b, mine].double() @ k[g].T / math.sqrt(d)
            if case["kv"] == "e4m3":
                logits = logits * st["k_scale"][g].double()
            every = logits
            if st["sink"] is not None:
                every = torch.cat([logits, st["sink"][mine].double()[:, None]], dim=1)
            lse[b, mine] = torch.logsumexp(every, dim=1)
            prob = torch.exp(logits - lse[b, mine][:, None])
            o = prob @ v[g]
            out[b, mine] = o * st["v_scale"][g].double() if case["kv"] == "e4m3" else o
            if mass is not None:
                mass[b, g, first:n] += prob.sum(dim=0)
    return [out, lse] + ([mass] if mass is not None else [])


def _exact_store(case, st):
    hkv, ps = case["kv_heads"], case["page"]
    got = []
    for pool, new in (("k", st["kv_new"][:, :hkv]), ("v", st["kv_new"][:, hkv:])):
        x = new.double()
        if case["kv"] == "e4m3":
            x = (x / st[pool + "_scale"].double()[None, :, None]).clamp(-448.0, 448.0)
        whole = st[pool].double()
        for b in range(case["batch"]):
            at = range(b * case["tokens"], (b + 1) * case["tokens"])
            s = torch.arange(case["start"], case["start"] + case["tokens"], device="cuda")
            whole[st["table"][b].long()[s // ps], :, s % ps] = x[at.start: at.stop]
        got.append(whole)
    if not case["tracked"]:
        return got
    w, p = st["weights"].double(), st["positions"].clone()
    for b in range(case["batch"]):
        mine = st["token_positions"][b * case["tokens"]: (b + 1) * case["tokens"]]
        w[b, :, case["start"]: case["start"] + case["tokens"]] = 0.0
        p[b, :, case["start"]: case["start"] + case["tokens"]] = mine
    return got + [w, p]


def _exact_evict(case, st):
    keep, ps = case["keep"], case["page"]
    if case["batch"] * case["kv_heads"] > 600:
        return None
    w, pos, table = (st[x].cpu() for x in ("weights", "positions", "table"))
    w_out, p_out = st["weights_out"].double().cpu(), st["positions_out"].clone().cpu()
    k, v = st["k"].double(), st["v"].double()
    lens = st["lens"].tolist()
    for b, n in enumerate(lens):
        seen = int(st["seen"][b])
        for g in range(case["kv_heads"]):
            m = min(n, keep)
            w_out[b, g, :m], p_out[b, g, :m] = w[b, g, :m].double(), pos[b, g, :m]
            if n <= keep:
                continue
            at = pos[b, g, :n]
            score = w[b, g, :n].double().nan_to_num(nan=-math.inf, posinf=math.inf, neginf=-math.inf)
            safe = (at < case["first"]) | (at >= seen - case["recent"])
            value, index = torch.sort(torch.where(safe, math.inf, score), descending=True, stable=True)
            stay = torch.zeros(n, dtype=torch.bool)
            stay[index[:keep]] = True
            goes = torch.nonzero(stay[keep:])[:, 0] + keep
            into = torch.nonzero(~stay[:keep])[:, 0]
            w_out[b, g, into], p_out[b, g, into] = w[b, g, goes].double(), pos[b, g, goes]
            row = table[b].long()
            to, of = row[into // ps].cuda(), row[goes // ps].cuda()
            k[to, g, (into % ps).cuda()] = k[of, g, (goes % ps).cuda()]
            v[to, g, (into % ps).cuda()] = v[of, g, (goes % ps).cuda()]
    return [torch.tensor(lens, dtype=torch.int32).clamp_max(keep), w_out, p_out, k, v]
