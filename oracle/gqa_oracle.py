"""Float64 oracle of the grouped-query cache operators (include/dsv4gqa.h):
plain numpy loops over requests and heads, written from the formulas.  Test
infrastructure only; it shares no code with the CUDA path.

A cache is a dict: k, v [pages, KV heads, page_size, head_dim] (float64 values
as stored; codes' values for e4m3), table [rows, logical pages], k_scale,
v_scale [KV heads] or None.
"""
from __future__ import annotations

import numpy as np

ERR_REQ_ROW, ERR_STORE_ROW, ERR_GQA_PAGE, ERR_GQA_LENGTH, ERR_LOAD_ROW = 0x40, 0x80, 0x200, 0x400, 0x800

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([(m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 7) for e in range(16) for m in range(8)][:127])


def _nearest(grid, x):
    """Index of the ascending grid's value nearest to x >= 0 (ties to the even index, saturating)."""
    i = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo, hi = x - grid[i - 1], grid[i] - x
    return np.where((lo < hi) | ((lo == hi) & (i % 2 == 1)), i - 1, i)


def e2m1_pack(x, scale):
    """(codes, block scales) of rows x [..., D]: bytes [..., D / 2] and e4m3 codes [..., D / 16], as the write defines
    them: quotients in fp32, then the nearest value.  scale: fp32, broadcast against [..., D / 16]."""
    x = np.asarray(x, np.float32)
    x = x.reshape(*x.shape[:-1], -1, 16)
    scale = np.asarray(scale, np.float32)
    nan = np.isnan(x).any(-1)
    top = np.abs(np.where(np.isnan(x), 0, x)).max(-1)
    with np.errstate(over="ignore", divide="ignore", invalid="ignore"):
        block = _nearest(E4M3, (top / (np.float32(6) * scale)).astype(np.float64)).astype(np.uint8)
        step = (E4M3[block].astype(np.float32) * scale)[..., None]
        q = np.where(step > 0, x / step, np.float32(0))
        size = np.where(np.isnan(q), 0.0, np.abs(q).astype(np.float64))
    code = _nearest(E2M1, size).astype(np.uint8) | (np.signbit(x) & (step > 0)).astype(np.uint8) << 3
    code[nan] = 0
    block = np.where(nan, 0x7f, block).astype(np.uint8)
    code = code.reshape(*code.shape[:-2], -1)
    return code[..., ::2] | code[..., 1::2] << 4, block


def e2m1_values(codes, blocks):
    """Float64 values [..., D] of bytes [..., D / 2] and block scales' e4m3 codes [..., D / 16] (no head's scale)."""
    codes, blocks = np.asarray(codes), np.asarray(blocks)
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*blocks.shape, 16)
    s = np.where(blocks & 127 == 127, np.nan, E4M3[np.minimum(blocks & 127, 126)]) * np.where(blocks & 128, -1.0, 1.0)
    x = E2M1[c & 7] * np.where(c & 8, -1.0, 1.0) * s[..., None]
    return x.reshape(*blocks.shape[:-1], -1)


def gqa_load(req_rows, slots, cache):
    """(k, v, error bits): float64 [n, KV heads, D] of what the named slots stand for, heads' scales included."""
    table, ps = cache["table"], cache["k"].shape[2]
    n, err = len(slots), 0
    k, v = (np.zeros((n, cache["k"].shape[1], cache["k"].shape[3])) for _ in range(2))
    for i, (r, s) in enumerate(zip(req_rows, slots)):
        page = table[r, s // ps] if 0 <= r < table.shape[0] and 0 <= s < table.shape[1] * ps else -1
        if not 0 <= page < cache["k"].shape[0]:
            err = ERR_LOAD_ROW
            continue
        for out, pool in ((k, "k"), (v, "v")):
            scale = cache[pool + "_scale"]
            out[i] = cache[pool][page, :, s % ps] * (1.0 if scale is None else np.asarray(scale)[:, None])
    return k, v, err


def _request(lens, req, b, rows, max_len):
    """(row, cached rows, error bits) of request b."""
    n, row, err = int(lens[b]), b if req is None else int(req[b]), 0
    if n < 0 or n > max_len:
        err |= ERR_GQA_LENGTH
        n = min(max(n, 0), max_len)
    if not 0 <= row < rows:
        err |= ERR_REQ_ROW if n else 0
        row, n = 0, 0
    return row, n, err


def gqa_decode(q, lens, cache, *, max_len, scale, window=0, sink=None, req=None, weights=None, weights_out=None,
               decay=1.0):
    """(out, lse, weights_out, error bits, spread): spread holds what a
    tolerance needs: per head the largest sum |q||k| scale of a score, the sum
    p |v| of every output value, the largest |v| over the sum of exp(s - max),
    and per request the number of rows."""
    batch, heads, dim = q.shape
    hkv, ps = cache["k"].shape[1], cache["k"].shape[2]
    group = heads // hkv
    out = np.zeros(q.shape)
    lse = np.full((batch, heads), -np.inf)
    mag, soft, tail, rows = np.zeros((batch, heads)), np.zeros(q.shape), np.zeros((batch, heads)), np.zeros(batch, int)
    wo = None if weights is None else np.array(weights_out, dtype=np.float64)
    wslack = None if weights is None else np.zeros_like(wo)
    errs, sums = 0, {}
    for b in range(batch):
        row, n, err = _request(lens, req, b, cache["table"].shape[0], max_len)
        errs |= err
        rows[b] = n
        lo = max(0, n - window) if window else 0
        slots = np.arange(lo, n)
        page = cache["table"][row][slots // ps] if n else np.zeros(0, int)
        good = (page >= 0) & (page < cache["k"].shape[0])
        if not good.all():
            errs |= ERR_GQA_PAGE
        slots, page = slots[good], page[good]
        if wo is not None and n:
            got = sums.setdefault(row, [0, np.zeros(wo.shape[1:]), np.zeros(wo.shape[1:])])
            got[0] = max(got[0], n)
        for i in range(heads):
            h = i // group
            k = cache["k"][page, h, slots % ps]
            v = cache["v"][page, h, slots % ps]
            ks = 1.0 if cache["k_scale"] is None else float(cache["k_scale"][h])
            vs = 1.0 if cache["v_scale"] is None else float(cache["v_scale"][h])
            s = scale * ks * (k @ q[b, i])
            sk = -np.inf if sink is None else float(sink[i])
            every = np.append(s, sk)
            top = every.max()
            if top == -np.inf:
                continue
            if sk == np.inf:
                lse[b, i] = np.inf
                continue
            total = np.exp(every - top).sum()
            p = np.exp(s - top) / total
            out[b, i] = vs * (p @ v)
            lse[b, i] = top + np.log(total)
            if len(s):
                mag[b, i] = scale * ks * (np.abs(k) @ np.abs(q[b, i])).max()
                soft[b, i] = vs * (p @ np.abs(v))
                tail[b, i] = vs * np.abs(v).max() / total * len(s)
            if wo is not None and len(s):
                sums[row][1][h, slots] += p
                sums[row][2][h, slots] += p * (1.0 + mag[b, i])
    for row, (n, add, slack) in ({} if wo is None else sums).items():
        wo[row, :, :n] = decay * weights[row, :, :n].astype(np.float64) + add[:, :n]
        wslack[row] = slack
    return out, lse, wo, errs, {"mag": mag, "soft": soft, "tail": tail, "rows": rows, "wslack": wslack}


def gqa_evict(lens, cache, weights, keep, *, max_len, first=0, recent=0, seq_lens=None, positions=None, req=None,
              weights_out=None, positions_out=None):
    """(lens_out, k, v, weights_out, positions_out, error bits), new arrays.
    cache's pools may be of any element type: rows are copied."""
    table, ps = cache["table"], cache["k"].shape[2]
    k, v = cache["k"].copy(), cache["v"].copy()
    wo = weights.copy() if weights_out is None else weights_out.copy()
    po = None if positions is None else (positions if positions_out is None else positions_out).copy()
    batch, errs, named = len(lens), 0, set()
    lens_out = np.zeros(batch, dtype=np.int32)
    for b in range(batch):
        row, n, err = _request(lens, req, b, table.shape[0], max_len)
        errs |= err
        lens_out[b] = min(n, keep)
        again = req is not None and row in named
        if n:
            named.add(row)
        if again and n:
            errs |= ERR_REQ_ROW
            continue
        for h in range(k.shape[1]):
            if n <= keep:
                wo[row, h, :n] = weights[row, h, :n]
                if po is not None:
                    po[row, h, :n] = positions[row, h, :n]
                continue
            at = np.arange(n) if positions is None else positions[row, h, :n].astype(np.int64)
            seen = n if seq_lens is None else int(seq_lens[b])
            safe = (at < first) | (at >= seen - recent)
            w = weights[row, h, :n].astype(np.float64)
            w = np.where(np.isnan(w), -np.inf, w)
            order = sorted(range(n), key=lambda s: (0, s) if safe[s] else (1, -w[s], s))
            stays = np.zeros(n, bool)
            stays[order[:keep]] = True
            holes = [s for s in range(keep) if not stays[s]]
            goes = [s for s in range(keep, n) if stays[s]]
            for s in range(keep):
                if stays[s]:
                    wo[row, h, s] = weights[row, h, s]
                    if po is not None:
                        po[row, h, s] = positions[row, h, s]
            for dst, src in zip(holes, goes):
                wo[row, h, dst] = weights[row, h, src]
                if po is not None:
                    po[row, h, dst] = positions[row, h, src]
                to, of = table[row, dst // ps], table[row, src // ps]
                if not (0 <= to < k.shape[0] and 0 <= of < k.shape[0]):
                    errs |= ERR_GQA_PAGE
                    continue
                k[to, h, dst % ps] = cache["k"][of, h, src % ps]
                v[to, h, dst % ps] = cache["v"][of, h, src % ps]
    return lens_out, k, v, wo, po, errs
