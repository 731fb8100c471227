"""The 4-bit grouped-query cache as a decode loop uses it, and the reading back of a cache's rows: what is timed and
what their answers are.

A 4-bit row holds e2m1 codes, two to a byte (the even dim in the low half), and an e4m3 scale for every 16 of them in
pools of their own: value = code * block scale * the head's fp32 scale.  Three operators: the attention of one new token
per request over such a cache, the quantising write (a pass writes new rows and reads back what the cache now stands
for, as the attention inside a prompt's chunk does), and the reading back of rows, of any cache type, to 16 bits.
``own`` chooses between the plain torch form and the library's entry points.
"""
import math

import torch

own = False

_KINDS = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
_CODES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
_GOLDEN = 0.6180339887498949


# ---------------------------------------------------------------- cases
def _decode(name, **kw):
    c = {"op": "decode", "q": "bf16", "kv": "e2m1", "heads": 32, "kv_heads": 8, "dim": 128, "page": 256, "batch": 1,
         "lo": 1, "hi": 1, "window": 0, "sink": False, "weights": False, "token_major": False, "scaled": False}
    return {"name": name, **c, **kw}


def _rows_of(name, op, **kw):
    c = {"op": op, "q": "bf16", "kv": "e2m1", "kv_heads": 8, "dim": 128, "page": 256, "batch": 1, "tokens": 1,
         "start": 0, "token_major": False, "scaled": False}
    return {"name": name, **c, **kw}


def listed():
    return [
        # one user, a few hundred cached tokens: the launch latency of a decode step
        _decode("decode4_one_short", lo=333, hi=333),
        # a serving batch of mixed lengths, the usual decode step
        _decode("decode4_batch", batch=32, lo=2048, hi=32768),
        # two very long contexts, 8 query heads per KV head: the split over the cache's length carries it
        _decode("decode4_long", heads=64, batch=2, lo=131072, hi=131071 + 64, sink=True, scaled=True),
        # a step that also accumulates the weight each cached row receives, f16
        _decode("decode4_weights_f16", q="f16", batch=16, lo=2048, hi=16384, weights=True),
        # wide heads, 16 query heads for each of two KV heads
        _decode("decode4_heads256", heads=32, kv_heads=2, dim=256, batch=64, lo=1024, hi=16384, scaled=True),
        # a small model: one query head per KV head, 64 wide, f16, small token-major pages, ragged lengths, a window
        _decode("decode4_heads64_f16", q="f16", heads=16, kv_heads=16, dim=64, page=16, batch=48, lo=1, hi=2000,
                window=1024, token_major=True),
        # a decode step's write: one new token per request
        _rows_of("store4_step", "store", batch=64, tokens=1, start=1023),
        # a chunk of a few prompts: a ragged number of tokens that begins inside a page
        _rows_of("store4_chunk_f16", "store", q="f16", batch=7, tokens=333, start=77, scaled=True, dim=64, page=64),
        # long prompts at once
        _rows_of("store4_prompt", "store", batch=64, tokens=1024, start=500, scaled=True),
        # one request's short prefix, read for the attention of its next prompt chunk
        _rows_of("load4_short", "load", tokens=777),
        # the prefixes of a whole batch
        _rows_of("load4_prefix", "load", batch=32, tokens=4096, scaled=True),
        # the same of an 8-bit cache with token-major pages, to f16
        _rows_of("load_e4m3", "load", kv="e4m3", q="f16", batch=16, tokens=4001, token_major=True, scaled=True),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "decode", "store", "store", "load", "load"])
    kv = rng.choice(["e2m1", "e2m1", "bf16", "f16", "e4m3"]) if op == "load" else "e2m1"
    q = kv if kv in ("bf16", "f16") else rng.choice(["bf16", "f16"])
    dim = rng.choice([64, 128, 128, 256])
    hkv = rng.choice([1, 2, 3, 4, 8, 8, 16])
    page = rng.choice([16, 32, 64, 128, 256, 256])
    row = hkv * dim * 2                      # values of K and V
    case = {"op": op, "q": q, "kv": kv, "kv_heads": hkv, "dim": dim, "page": page,
            "token_major": rng.random() < 0.3, "scaled": kv in ("e2m1", "e4m3") and rng.random() < 0.5}
    if op == "decode":
        batch = _spread(rng, 1, 128)
        hi = _spread(rng, 1, max(2, min(131072, int(6e8 / (row * batch)))))
        group = rng.choice([1, 2, 4, 5, 7, 8, 8, 12, 16])
        return {**case, "heads": group * hkv, "batch": batch, "lo": rng.choice([1, hi // 4 + 1, hi]), "hi": hi,
                "window": rng.choice([0, 0, 0, hi // 2 + 1, 128]), "sink": rng.random() < 0.5,
                "weights": rng.random() < 0.3}
    batch = _spread(rng, 1, 128)
    return {**case, "batch": batch, "tokens": _spread(rng, 1, max(2, min(4096, int(1.2e8 / (row * batch))))),
            "start": rng.randrange(0, 3000)}


def _lens(case):
    """The batch's cached lengths: spread evenly over lo .. hi, in an order that the seed shuffles."""
    lo, hi, n = case["lo"], case["hi"], case["batch"]
    return [lo + int((hi - lo + 1) * ((0.31 + i * _GOLDEN) % 1.0)) for i in range(n)]


def _attended(case):
    w = case["window"]
    return [min(n, w) if w else n for n in _lens(case)]


# ---------------------------------------------------------------- inputs
def _pool(case, pages, width, gen, kind):
    """[pages, KV heads, page, width]: codes of normal values (the eight sizes are then about equally frequent), block
    scales of values around 1, or the values themselves."""
    order = (pages, case["page"], case["kv_heads"], width) if case["token_major"] else \
        (pages, case["kv_heads"], case["page"], width)
    if kind == "codes":
        x = torch.randint(0, 256, order, generator=gen, device="cuda", dtype=torch.uint8)
    elif kind == "blocks":
        x = (0.2 + 0.3 * torch.rand(order, generator=gen, device="cuda", dtype=torch.float16)).to(torch.float8_e4m3fn)
    else:
        x = torch.randn(order, generator=gen, device="cuda", dtype=torch.bfloat16 if kind == "bf16" else torch.float16)
        x = x.to(_KINDS[kind])
    return x.transpose(1, 2) if case["token_major"] else x


def _cache(case, slots, gen):
    """K and V pools whose pages belong to the requests in random order, with a few pages that belong to nobody."""
    pages = -(-slots // case["page"])
    total = case["batch"] * pages + 3
    st = {}
    for name in ("k", "v"):
        if case["kv"] == "e2m1":
            st[name] = _pool(case, total, case["dim"] // 2, gen, "codes")
            st[name + "_blocks"] = _pool(case, total, case["dim"] // 16, gen, "blocks")
        else:
            st[name] = _pool(case, total, case["dim"], gen, case["kv"])
        if case["scaled"]:   # calibrated factors, as a bf16 checkpoint holds them
            f = 0.5 + torch.rand(case["kv_heads"], generator=gen, device="cuda")
            st[name + "_scale"] = f.to(torch.bfloat16).float()
    order = torch.randperm(total, generator=gen, device="cuda")[: case["batch"] * pages]
    st["table"] = order.view(case["batch"], pages).to(torch.int32)
    return st


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    b, hkv, dim = case["batch"], case["kv_heads"], case["dim"]
    kind = _KINDS[case["q"]]
    if case["op"] == "decode":
        st = _cache(case, case["hi"], gen)
        lens = torch.tensor(_lens(case), dtype=torch.int32, device="cuda")
        st["lens"] = lens[torch.randperm(b, generator=gen, device="cuda")].contiguous()
        st["query"] = torch.randn(b, case["heads"], dim, generator=gen, device="cuda").to(kind)
        st["sink"] = torch.randn(case["heads"], generator=gen, device="cuda") if case["sink"] else None
        st["weights"] = None
        if case["weights"]:
            width = st["table"].shape[1] * case["page"]
            st["weights"] = torch.rand(b, hkv, width, generator=gen, device="cuda")
            st["weights_out"] = torch.zeros_like(st["weights"])
        st["out"] = torch.empty_like(st["query"])
        st["lse"] = torch.empty(b, case["heads"], device="cuda")
        st["max_len"] = case["hi"]
    else:
        slots = case["start"] + case["tokens"]
        st = _cache(case, slots, gen)
        n = b * case["tokens"]
        if case["op"] == "store":
            # K and V as the projection leaves them, one row of K and V heads per token; some dims of a key are larger
            x = torch.randn(n, 2 * hkv, dim, generator=gen, device="cuda", dtype=torch.float16)
            loud = 1.0 + 3.0 * (torch.rand(hkv, dim, generator=gen, device="cuda") > 0.95)
            x[:, :hkv] *= loud
            st["kv_new"] = x.to(kind)
        req = torch.arange(b, device="cuda").repeat_interleave(case["tokens"])
        slot = torch.arange(case["start"], slots, device="cuda").repeat(b)
        st["req"], st["slots"] = req.to(torch.int32), slot.to(torch.int32)
        st["k_rows"] = torch.empty(n, hkv, dim, device="cuda", dtype=kind)
        st["v_rows"] = torch.empty_like(st["k_rows"])
    st["case"] = dict(case)
    return st


# ---------------------------------------------------------------- one pass
def _handle(st):
    """The cache descriptor and the workspace that a program keeps beside its pools."""
    from hybrid_sparse_mqa_gb300 import attn
    if "cache" not in st:
        c = st["case"]
        cache = attn.make_gqa_cache(st["k"], st["v"], st["table"], k_scale=st.get("k_scale"), v_scale=st.get("v_scale"),
                                    k_blocks=st.get("k_blocks"), v_blocks=st.get("v_blocks"))
        if c["op"] == "decode":
            size = attn.dsv4_gqa_decode_workspace_size(cache, c["batch"], c["heads"], st["max_len"], c["weights"])
            st["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        st["cache"] = cache
    return attn, st["cache"]


def run(st):
    return {"decode": _run_decode, "store": _run_store, "load": _run_load}[st["case"]["op"]](st)


def _widen(codes, blocks):
    """e2m1 codes [..., D / 2] and block scales [..., D / 16] to fp32 [..., D]."""
    size = torch.tensor(_CODES, device=codes.device)
    size = torch.cat([size, -size])
    x = torch.stack([codes & 15, codes >> 4], dim=-1).long()
    x = size[x].reshape(*blocks.shape, 16)
    return (x * blocks.float()[..., None]).flatten(-2)


def _values(st, pool, index):
    """fp32 values of a pool's rows at `index`, without the heads' scales."""
    x = st[pool][index]
    return _widen(x, st[pool + "_blocks"][index]) if st["case"]["kv"] == "e2m1" else x.float()


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
    k = _values(st, "k", table).transpose(1, 2).reshape(b, hkv, pages * ps, d)
    v = _values(st, "v", table).transpose(1, 2).reshape(b, hkv, pages * ps, d)
    slot = torch.arange(pages * ps, device="cuda")
    n = st["lens"][:, None].long()
    seen = slot < n
    if c["window"]:
        seen = seen & (slot >= n - c["window"])
    seen = seen[:, None, None, :]
    v = v.masked_fill(~seen.transpose(2, 3), 0.0)
    q = st["query"].float().view(b, hkv, h // hkv, d)
    if c["scaled"]:
        q = q * st["k_scale"][:, None, None]
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
    out = torch.matmul(p, v)
    if c["scaled"]:
        out = out * st["v_scale"][:, None, None]
    out = out.reshape(b, h, d).to(st["query"].dtype)
    lse = (top + torch.log(total)).reshape(b, h)
    if not c["weights"]:
        return [out, lse]
    w_out = st["weights_out"]
    width = pages * ps
    got = st["weights"][:, :, :width] + p.sum(dim=2)
    live = (slot < n)[:, None, :]
    w_out[:, :, :width] = torch.where(live, got, w_out[:, :, :width])
    return [out, lse, w_out]


def _place(st):
    """Page and slot in the page of every token."""
    slot = st["slots"].long()
    return st["table"][st["req"].long(), slot // st["case"]["page"]].long(), slot % st["case"]["page"]


def _quantise(x, scale):
    """Codes and block scales of fp32 rows [..., D]; scale [KV heads, 1] or a number."""
    x = x.unflatten(-1, (-1, 16))
    top = x.abs().amax(dim=-1)
    block = (top / (6.0 * scale)).clamp_max(448.0).to(torch.float8_e4m3fn)
    step = (block.float() * scale)[..., None]
    y = torch.where(step > 0, x / step, 0.0)
    size = y.abs()
    code = torch.zeros_like(size, dtype=torch.uint8)
    for at, even in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += size >= at if even else size > at        # a tie goes to the even code
    code = (code | torch.signbit(y).to(torch.uint8) << 3).flatten(-2)
    return code[..., ::2] | (code[..., 1::2] << 4), block


def _read(st, pool, out):
    page, off = _place(st)
    x = _values(st, pool, (page, slice(None), off))
    if st["case"]["scaled"]:
        x = x * st[pool + "_scale"][:, None]
    out.copy_(x)
    return out


def _run_store(st):
    c = st["case"]
    hkv = c["kv_heads"]
    new = {"k": st["kv_new"][:, :hkv], "v": st["kv_new"][:, hkv:]}
    if own:
        attn, cache = _handle(st)
        attn.dsv4_gqa_store(new["k"], new["v"], st["req"], st["slots"], cache)
        return list(attn.dsv4_gqa_load(st["req"], st["slots"], cache, k=st["k_rows"], v=st["v_rows"]))
    page, off = _place(st)
    for pool in ("k", "v"):
        codes, blocks = _quantise(new[pool].float(), st[pool + "_scale"][:, None] if c["scaled"] else 1.0)
        st[pool][page, :, off] = codes
        st[pool + "_blocks"].view(torch.uint8)[page, :, off] = blocks.view(torch.uint8)
    return [_read(st, "k", st["k_rows"]), _read(st, "v", st["v_rows"])]


def _run_load(st):
    if own:
        attn, cache = _handle(st)
        return list(attn.dsv4_gqa_load(st["req"], st["slots"], cache, k=st["k_rows"], v=st["v_rows"]))
    return [_read(st, "k", st["k_rows"]), _read(st, "v", st["v_rows"])]


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    hkv, d = case["kv_heads"], case["dim"]
    row = {"e2m1": d // 2 + d // 16, "e4m3": d}.get(case["kv"], 2 * d)
    if case["op"] == "decode":
        rows = sum(_attended(case))
        b, h = case["batch"], case["heads"]
        byts = rows * hkv * row * 2 + b * h * d * 2 * 2 + b * h * 4 + b * 4
        byts += 4 * sum(-(-n // case["page"]) for n in _attended(case))
        if case["weights"]:
            byts += 8 * hkv * sum(_lens(case))
        return {"bytes": byts, "flops": 4 * rows * h * d}
    n = case["batch"] * case["tokens"]
    if case["op"] == "load":
        return {"bytes": n * hkv * 2 * (row + 2 * d) + 8 * n, "flops": 2 * n * hkv * 2 * d if row < 2 * d else 0}
    # new rows in, the cache's rows out, what they stand for out
    return {"bytes": n * hkv * 2 * (2 * d + row + 2 * d) + 8 * n, "flops": 6 * n * hkv * 2 * d}


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    return {"decode": _exact_decode, "store": _exact_store, "load": _exact_load}[case["op"]](case, st)


def _double(st, case, pool, index):
    """The values that rows of a pool stand for, heads' scales included; KV heads come first in `index`'s result."""
    rows = st[pool][index]
    if case["kv"] == "e2m1":
        out = torch.empty(*rows.shape[:-1], case["dim"], dtype=torch.float64, device="cuda")
        for half in (0, 1):
            code = (rows >> (4 * half)) & 15
            e, m = ((code >> 1) & 3).double(), (code & 1).double()
            size = torch.where(e == 0, 0.5 * m, (1.0 + 0.5 * m) * 2.0 ** (e - 1.0))
            out[..., half::2] = torch.where(code >= 8, -size, size)
        rows = out * st[pool + "_blocks"][index].double().repeat_interleave(16, dim=-1)
    else:
        rows = rows.double()
    return rows


def _exact_decode(case, st):
    hkv, group, d = case["kv_heads"], case["heads"] // case["kv_heads"], case["dim"]
    out = torch.zeros(st["query"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(out.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    mass = st["weights_out"].double() if case["weights"] else None
    for b, n in enumerate(st["lens"].tolist()):
        first = max(0, n - case["window"]) if case["window"] else 0
        where = st["table"][b, : -(-n // case["page"])].long()
        k, v = (_double(st, case, pool, where).transpose(0, 1).flatten(1, 2)[:, first:n] for pool in ("k", "v"))
        if mass is not None:
            mass[b, :, :n] = st["weights"][b, :, :n].double()
        for g in range(hkv):
            mine = slice(g * group, (g + 1) * group)
            logits = st["query"][b, mine].double() @ k[g].T / math.sqrt(d)
            if case["scaled"]:
                logits = logits * st["k_scale"][g].double()
            every = logits
            if st["sink"] is not None:
                every = torch.cat([logits, st["sink"][mine].double()[:, None]], dim=1)
            lse[b, mine] = torch.logsumexp(every, dim=1)
            prob = torch.exp(logits - lse[b, mine][:, None])
            o = prob @ v[g]
            out[b, mine] = o * st["v_scale"][g].double() if case["scaled"] else o
            if mass is not None:
                mass[b, g, first:n] += prob.sum(dim=0)
    return [out, lse] + ([mass] if mass is not None else [])


def _nearest(x, grid):
    """The grid's nearest value to each x >= 0 (ascending grid; a tie goes to the even place)."""
    at = torch.searchsorted(grid, x).clamp(1, len(grid) - 1)
    lo, hi = grid[at - 1], grid[at]
    up = (x - lo > hi - x) | ((x - lo == hi - x) & (at % 2 == 0))
    return torch.where(up, hi, lo)


def _exact_store(case, st):
    hkv = case["kv_heads"]
    codes = torch.tensor(_CODES, dtype=torch.float64, device="cuda")
    every = torch.arange(127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()   # 0 .. 448
    got = []
    for pool, new in (("k", st["kv_new"][:, :hkv]), ("v", st["kv_new"][:, hkv:])):
        x = new.double().unflatten(-1, (-1, 16))
        scale = st[pool + "_scale"].double()[:, None] if case["scaled"] else torch.ones(1, 1, device="cuda")
        step = _nearest(x.abs().amax(dim=-1) / 6.0 / scale, every) * scale
        size = torch.where(step[..., None] > 0, x.abs() / step[..., None], 0.0)
        got.append((torch.sign(x) * _nearest(size, codes) * step[..., None]).flatten(-2))
    return got


def _exact_load(case, st):
    ps, t = case["page"], case["tokens"]
    slots = torch.arange(case["start"], case["start"] + t, device="cuda")
    got = []
    for pool in ("k", "v"):
        x = [_double(st, case, pool, (st["table"][b].long()[slots // ps], slice(None), slots % ps))
             for b in range(case["batch"])]
        x = torch.cat(x)
        got.append(x * st[pool + "_scale"].double()[:, None] if case["scaled"] else x)
    return got
