"""The grouped-query cache operators on the GPU against the float64 oracle.

Store and evict move and round values by rules that fix every bit, so they
are compared exactly.  Decode is compared element by element with a bound
built from its arithmetic, for n rows of which a head's scores are at most m
in magnitude before cancellation (m = scale * max_j sum |q||k_j|):
  score      fp32 accumulation of D products, two factors:  ds = (D + 8) 2^-23 m
  p          2^x of the score in fp32: relative 2 ds + 2^-20 (both sides of the quotient)
  P's rounding for the MMA: two 16-bit pieces leave 2^-16; one f16 (e4m3
             caches) 2^-11, plus 2^-25 of the largest p for the small ones
  sums       fp32 over n / 16 steps and the joins: (n / 16 + 64) 2^-23
  output     half a step of its type, relative
The bound on an output is c * sum p|v| + tail + half a step * |out|, with c the
sum of the relative terms above.
"""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import gqa_oracle as O

pytestmark = pytest.mark.gpu

BF, HF, F8 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def A():
    from hybrid_sparse_mqa_gb300 import build
    build.build()
    from hybrid_sparse_mqa_gb300 import attn
    attn.lib()
    attn.dsv4_attn_get_device_error()
    return attn


class Case:
    """A cache of `rows` request rows with room for `slots` slots each, in a
    pool of shuffled pages; rows that nobody owns hold NaN and infinities."""

    def __init__(self, kv=BF, q=None, hkv=2, dim=64, page=16, rows=3, slots=100, seed=0, token_major=False, spread=1.0):
        self.kv, self.qt = kv, q or (kv if kv != F8 else BF)
        self.hkv, self.dim, self.page = hkv, dim, page
        self.width = -(-slots // page)
        self.gen = torch.Generator().manual_seed(seed)
        pages = rows * self.width + 3
        order = torch.randperm(pages, generator=self.gen)
        self.table = order[: rows * self.width].view(rows, self.width).to(torch.int32).contiguous()
        k, v = (torch.randn(pages, hkv, page, dim, generator=self.gen) * spread for _ in range(2))
        wild = torch.tensor([math.nan, math.inf, -math.inf, 3e4])
        for x in (k, v):
            x[order[rows * self.width:]] = wild[torch.randint(0, 4, x[:1].shape, generator=self.gen)]
        if kv == F8:
            k, v = k.nan_to_num(nan=math.nan, posinf=448, neginf=-448), v.nan_to_num(nan=math.nan, posinf=448, neginf=-448)
        self.k, self.v = self._lay(k.to(kv), token_major), self._lay(v.to(kv), token_major)
        self.ks = self.vs = None
        if kv == F8:
            self.ks, self.vs = (0.5 + torch.rand(hkv, generator=self.gen) for _ in range(2))

    @staticmethod
    def _lay(x, token_major):
        return x.transpose(1, 2).contiguous().transpose(1, 2) if token_major else x

    def poison(self, lens, rows=None):
        """NaN and infinities behind every request's last row."""
        for b, n in enumerate(lens):
            r = b if rows is None else rows[b]
            for s in range(n, self.width * self.page):
                p, o = int(self.table[r, s // self.page]), s % self.page
                bad = torch.tensor([math.nan, 448.0 if self.kv == F8 else math.inf])[s % 2].to(self.kv)
                for x in (self.k, self.v):
                    (x.view(torch.uint8) if self.kv == F8 else x)[p, :, o] = \
                        bad.view(torch.uint8) if self.kv == F8 else bad

    def query(self, batch, heads, spread=1.0):
        return (torch.randn(batch, heads, self.dim, generator=self.gen) * spread).to(self.qt)

    def cuda(self):
        for name in ("k", "v", "table", "ks", "vs"):
            x = getattr(self, name)
            setattr(self, name + "_d", None if x is None else self._keep_strides(x))
        return self

    @staticmethod
    def _keep_strides(x):
        if x.dim() == 4 and not x.is_contiguous():
            return x.transpose(1, 2).cuda().transpose(1, 2)
        return x.cuda()

    def handle(self, A):
        self.cuda()
        return A.make_gqa_cache(self.k_d, self.v_d, self.table_d, k_scale=self.ks_d, v_scale=self.vs_d)

    def oracle(self):
        return {"k": self.k.double().numpy(), "v": self.v.double().numpy(), "table": self.table.numpy(),
                "k_scale": None if self.ks is None else self.ks.double().numpy(),
                "v_scale": None if self.vs is None else self.vs.double().numpy()}


def check_decode(A, case, lens, heads, *, window=0, sink=None, req=None, weights=False, decay=1.0, spread=1.0,
                 max_len=None, scale=None, want_flags=0, q=None):
    cache = case.handle(A)
    batch = len(lens)
    q = case.query(batch, heads, spread) if q is None else q
    max_len = case.width * case.page if max_len is None else max_len
    lens_t = torch.tensor(lens, dtype=torch.int32)
    w = wo = None
    if weights:
        shape = (case.table.shape[0], case.hkv, case.width * case.page + 5)
        w = torch.rand(shape, generator=case.gen)
        wo = torch.full(shape, -7.0)
    kw = {} if scale is None else {"scale": scale}
    d = lambda x: None if x is None else x.cuda()      # noqa: E731
    w_d, wo_d = d(w), d(wo)
    out, lse = A.dsv4_gqa_decode(d(q), lens_t.cuda(), cache, sink=d(sink), window=window, max_len=max_len,
                                 req_pool_indices=None if req is None else torch.tensor(req, dtype=torch.int32).cuda(),
                                 weights=w_d, weights_out=wo_d, decay=decay, **kw)
    torch.cuda.synchronize()
    flags = A.dsv4_attn_get_device_error()
    ref, rlse, rw, err, sp = O.gqa_decode(
        q.double().numpy(), lens, case.oracle(), max_len=max_len, scale=1 / math.sqrt(case.dim) if scale is None else scale,
        window=window, sink=None if sink is None else sink.double().numpy(), req=req,
        weights=None if w is None else w.double().numpy(), weights_out=None if wo is None else wo.double().numpy(),
        decay=decay)
    assert flags == err == want_flags, (flags, err)
    half = torch.finfo(case.qt).eps / 2
    n = sp["rows"][:, None]
    ds = (case.dim + 8) * 2.0 ** -23 * sp["mag"]
    sums = (n / 16 + 64) * 2.0 ** -23
    rel = 2 * ds + 2.0 ** -20 + sums + (2.0 ** -11 if case.kv == F8 else 2.0 ** -16)
    tail = 2.0 ** -25 * sp["tail"]
    tiny = 2.0 ** -25 if case.qt == HF else 0.0
    tol = rel[..., None] * sp["soft"] + tail[..., None] + (half + 2.0 ** -22) * np.abs(ref) + tiny
    results, tracked = [(out, lse)], [wo_d]
    if weights:      # short lists go other ways without weights, and where request rows may repeat
        for named, kept in ((req, False), (list(range(batch)) if req is None else req, True)):
            extra = {"weights": w_d, "weights_out": d(wo), "decay": decay} if kept else {}
            results.append(A.dsv4_gqa_decode(
                d(q), lens_t.cuda(), cache, sink=d(sink), window=window, max_len=max_len,
                req_pool_indices=None if named is None else torch.tensor(named, dtype=torch.int32).cuda(), **extra, **kw))
            torch.cuda.synchronize()
            assert A.dsv4_attn_get_device_error() == want_flags
            tracked.append(extra.get("weights_out"))
    for o, l in results:
        e = np.abs(o.double().cpu().numpy() - ref)
        assert np.isfinite(o.double().cpu().numpy()).all()
        assert (e <= tol).all(), (float((e / np.maximum(tol, 1e-300)).max()), np.argwhere(e > tol)[:4].tolist())
        g = l.double().cpu().numpy()
        assert np.array_equal(np.isinf(g), np.isinf(rlse))
        fin = np.isfinite(rlse)
        assert (np.abs(g[fin] - rlse[fin]) <=
                (ds + 2.0 ** -20 + sums + np.abs(np.where(fin, rlse, 0)) * 2.0 ** -22)[fin]).all()
    for got in (x for x in tracked if x is not None):
        gw = got.double().cpu().numpy()
        tolw = sp["wslack"] * (2 * (case.dim + 8) * 2.0 ** -23 + 2.0 ** -19 + float(sums.max())) + np.abs(rw) * 2.0 ** -22
        assert (np.abs(gw - rw) <= tolw).all(), float((np.abs(gw - rw) / np.maximum(tolw, 1e-300)).max())
    return out, lse, wo_d


EDGE = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 97, 100]


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("kv,q", [(BF, BF), (HF, HF), (F8, BF), (F8, HF)])
def test_decode_types_dims_and_lengths(A, kv, q, dim, page):
    c = Case(kv=kv, q=q, dim=dim, page=page, rows=len(EDGE), slots=100, seed=dim + page)
    c.poison(EDGE)
    check_decode(A, c, EDGE, 8, weights=True, sink=torch.randn(8, generator=c.gen))


@pytest.mark.parametrize("group", [1, 3, 8, 9, 16, 17, 64])
@pytest.mark.parametrize("kv", [BF, F8])
def test_decode_groups(A, kv, group):
    c = Case(kv=kv, hkv=3, dim=128, rows=4, slots=300, seed=group)
    c.poison([300, 5, 0, 129])
    check_decode(A, c, [300, 5, 0, 129], 3 * group, weights=True, decay=0.75)


@pytest.mark.parametrize("group", [17, 32, 33, 48, 49, 64])
@pytest.mark.parametrize("kv,dim", [(BF, 64), (BF, 128), (HF, 256), (F8, 64), (F8, 128), (F8, 256)])
def test_decode_of_wide_groups_over_long_lists(A, kv, dim, group):
    # several passes over the cache: parts that end inside requests, shared rows, pages outside the pool
    lens = [2500, 0, 7, 1203, 40, 1]
    c = Case(kv=kv, hkv=2, dim=dim, rows=6, slots=2500, seed=group + dim, token_major=group % 2 == 1)
    c.poison(lens)
    c.table[3, 30:33] = torch.tensor([-1, 10 ** 6, c.k.shape[0]])
    sink = torch.randn(2 * group, generator=c.gen)
    check_decode(A, c, lens, 2 * group, weights=True, sink=sink, want_flags=O.ERR_GQA_PAGE)
    check_decode(A, c, [1203, 2500, 40, 0, 7, 1203], 2 * group, window=700, req=[0, 0, 3, 1, 2, 3], weights=True,
                 want_flags=O.ERR_GQA_PAGE)


@pytest.mark.parametrize("window", [1, 15, 16, 40, 64, 1000])
@pytest.mark.parametrize("kv,dim", [(BF, 64), (BF, 128), (F8, 64), (HF, 256)])
def test_decode_windows(A, kv, dim, window):
    lens = [0, 1, 16, 39, 40, 41, 80, 200]
    c = Case(kv=kv, dim=dim, rows=8, slots=200, seed=window)
    c.poison(lens)
    check_decode(A, c, lens, 4, window=window, weights=True, decay=0.5)


@pytest.mark.parametrize("kv,dim,token_major,page", [(BF, 128, True, 32), (F8, 64, True, 16), (F8, 128, False, 128),
                                                     (HF, 64, False, 1024), (BF, 256, True, 256)])
def test_decode_layouts_and_splits(A, kv, dim, token_major, page):
    # few segments, long: every request is cut over many CTAs
    c = Case(kv=kv, hkv=2, dim=dim, page=page, rows=3, slots=9000, seed=9, token_major=token_major)
    check_decode(A, c, [8999, 3, 5001], 10, weights=True, sink=torch.randn(10, generator=c.gen))


def test_decode_more_requests_than_threads(A):
    lens = [(37 * b) % 90 if b % 5 else 0 for b in range(300)]
    c = Case(rows=300, slots=90, seed=2)
    check_decode(A, c, lens, 4, weights=True)
    check_decode(A, c, [0] * 299 + [50], 4)
    check_decode(A, c, [0] * 300, 4, sink=torch.randn(4, generator=c.gen))


def test_decode_scores_that_keep_rising(A):
    # the running reference moves with almost every tile, and far
    for kv in (BF, F8):
        c = Case(kv=kv, hkv=1, dim=64, rows=2, slots=2000, seed=4)
        ramp = torch.linspace(-30, 30, c.width * 16).view(1, -1, 16, 1)
        k = c.k.float()
        k[c.table[0].long()] = (ramp.transpose(0, 1) * torch.ones(64) * 0.2)
        c.k = k.to(kv)
        check_decode(A, c, [2000, 1999], 8, weights=True, spread=1.5)


def test_decode_one_row_takes_all(A):
    # scores of some hundreds: every other weight underflows
    c = Case(hkv=2, dim=128, rows=3, slots=500, seed=5)
    check_decode(A, c, [500, 499, 1], 8, spread=30.0, weights=True)


@pytest.mark.parametrize("slots,lens", [(100, [100, 17]), (9000, [9000, 4001])])
def test_decode_of_scores_far_below_zero(A, slots, lens):
    # Every score is -2^109 (7 rows of 8) or -2^110: products and sums of powers of two are exact, so the equal ones
    # share the weight and the output is their values' mean: fp32 sums of 16-bit values, and half a step of bf16.
    c = Case(hkv=1, dim=64, rows=2, slots=slots, seed=7)
    c.k.fill_(-2.0 ** 53)
    c.k[:, :, ::8] *= 2
    q = torch.full((2, 8, 64), 2.0 ** 53, dtype=BF)
    out, lse = A.dsv4_gqa_decode(q.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), c.handle(A), scale=2.0 ** -3)
    assert A.dsv4_attn_get_device_error() == 0
    for b, n in enumerate(lens):
        s = np.array([x for x in range(n) if x % 8])
        v = c.v[c.table[b].long()[s // c.page], 0, s % c.page].double()
        tol = v.abs().mean(0) * ((n / 16 + 64) * 2.0 ** -23 + 2.0 ** -16) + v.mean(0).abs() * (2.0 ** -8 + 2.0 ** -22)
        assert ((out[b].double().cpu() - v.mean(0)).abs() <= tol).all()
        assert (lse[b].double().cpu() / -2.0 ** 109 - 1).abs().max() <= 4 * 2.0 ** -23


def test_decode_small_queries_of_an_e4m3_cache(A):
    # queries whose f16 value would be zero or infinite
    for spread in (1e-12, 1e25):
        c = Case(kv=F8, q=BF, hkv=2, dim=64, rows=2, slots=60, seed=6)
        check_decode(A, c, [60, 33], 4, spread=spread, scale=0.125 / spread)


@pytest.mark.parametrize("heads", [2, 8, 24])
@pytest.mark.parametrize("kv,dim", [(BF, 64), (BF, 128), (HF, 64), (HF, 128), (HF, 256)])
@pytest.mark.parametrize("slots,lens", [(100, [100, 1, 17]), (9000, [9000, 4001, 40])])
def test_decode_of_infinite_values(A, kv, dim, heads, slots, lens):
    # a value that overflowed when it was written: infinite where every infinity of the dim has one sign, NaN where
    # both signs or a NaN meet, and all other dims as if it were not there
    c = Case(kv=kv, hkv=2, dim=dim, rows=3, slots=slots, seed=dim + heads)
    q = c.query(3, heads)
    lens_t = torch.tensor(lens, dtype=torch.int32).cuda()
    plain = A.dsv4_gqa_decode(q.cuda(), lens_t, c.handle(A), max_len=slots)

    def put(b, h, s, d, x):
        c.v[int(c.table[b, s // c.page]), h, s % c.page, d] = x

    marks = {}                                    # (request, KV head, dim): what its outputs are
    for b, n in enumerate(lens):
        for h in range(2):
            for i in range(6):
                d = int(torch.randint(0, dim // 8, (1,), generator=c.gen)) * 8 + i
                for s in torch.randint(0, n, (1 + i,), generator=c.gen).tolist():
                    put(b, h, s, d, -math.inf if i % 2 else math.inf)
                marks[b, h, d] = -math.inf if i % 2 else math.inf
            put(b, h, n - 1, dim - 1, math.nan)
            marks[b, h, dim - 1] = math.nan
            put(b, h, 0, dim - 2, math.inf)
            put(b, h, n - 1, dim - 2, -math.inf)
            marks[b, h, dim - 2] = math.nan if n > 1 else -math.inf
    c.poison(lens)
    w = torch.zeros(3, 2, c.width * c.page).cuda()
    cache = c.handle(A)
    results = [A.dsv4_gqa_decode(q.cuda(), lens_t, cache, max_len=slots),
               A.dsv4_gqa_decode(q.cuda(), lens_t, cache, max_len=slots, weights=w,
                                 req_pool_indices=torch.arange(3, dtype=torch.int32).cuda())]
    assert A.dsv4_attn_get_device_error() == 0
    group = heads // 2
    for i, (out, lse) in enumerate(results):
        want = results[1][0].clone() if i else plain[0].clone()
        for (b, h, d), x in marks.items():
            want[b, h * group: (h + 1) * group, d] = x
        assert torch.equal(out.isnan(), want.isnan())
        assert torch.equal(out.nan_to_num(nan=0.0, posinf=math.inf, neginf=-math.inf),
                           want.nan_to_num(nan=0.0, posinf=math.inf, neginf=-math.inf))
        if i == 0:
            assert torch.equal(lse, plain[1])


@pytest.mark.parametrize("slots,lens", [(900, [900, 333]), (9000, [9000, 4001])])
@pytest.mark.parametrize("kv,q", [(BF, BF), (HF, HF), (F8, BF), (F8, HF)])
@pytest.mark.parametrize("below", [12, 18, 22, 26, 30])
def test_decode_of_many_rows_far_below_one(A, kv, q, below, slots, lens):
    # the first row takes nearly all the weight and has the value zero, so the output is the sum of thousands of weights
    # of about 2^-below.  The scores are exact (one nonzero product); p is 2^x of them: 2^-20, and its half step for
    # the MMA, which is 2^-17 of p (two pieces) or 2^-12 (one), and below f16's normal numbers 2^-36 of the largest p.
    c = Case(kv=kv, q=q, hkv=1, dim=64, rows=2, slots=slots, seed=below)
    c.ks = c.vs = None
    k, v = torch.zeros(c.k.shape), torch.ones(c.v.shape)
    k[..., 0] = -below
    v[:, :, ::3, 1::2] = 0.5
    for b in range(2):
        k[int(c.table[b, 0]), :, 0] = 0.0
        v[int(c.table[b, 0]), :, 0] = 0.0
    c.k, c.v = k.to(kv), v.to(kv)
    assert torch.equal(c.k.float(), k)
    query = torch.zeros(2, 8, 64)
    query[:, :, 0] = 1.0
    scale = 0.71                                      # weights of 2^-1.024 below
    out, lse = A.dsv4_gqa_decode(query.to(q).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), c.handle(A),
                                 scale=scale, max_len=slots)
    assert A.dsv4_attn_get_device_error() == 0
    p = math.exp(-float(np.float32(scale)) * below)
    for b, n in enumerate(lens):
        rows = c.v.double()[c.table[b].long()].transpose(1, 2).reshape(-1, 64)[1:n]
        total = 1 + (n - 1) * p
        ref = rows.sum(0) * p / total
        exponents = below * 2.0 ** -23                # the rounding of the score and of its difference from the reference
        rel = 2.0 ** -19 + 4 * exponents + (n / 16 + 64) * 2.0 ** -23 + (2.0 ** -17 if kv != F8 else 2.0 ** -12)
        tol = ref * (rel + torch.finfo(q).eps / 2) + (0 if kv == BF else (n - 1) * 2.0 ** -36 / total)
        if q == HF:
            tol = tol + 2.0 ** -25                    # an output below f16's normal numbers
        assert ((out[b].double().cpu() - ref).abs() <= tol).all(), float(((out[b].double().cpu() - ref).abs() / tol).max())
        assert (lse[b].double().cpu() - math.log(total)).abs().max() <= 2.0 ** -19 + (n / 16 + 64) * 2.0 ** -23 + 2.0 ** -20


@pytest.mark.parametrize("scale", [0.71, 0.9, 1.3, 1.7, 2.2])
@pytest.mark.parametrize("kv,q", [(BF, BF), (HF, HF), (F8, HF)])
def test_decode_of_values_that_cancel(A, kv, q, scale):
    # half the rows have the value 1 and half -1, with weights that differ little, so that the rounding of P shows
    # beside the output's: 2^-17 of the sum of all weights at most (two pieces), while one f16 would leave up to 2^-12
    c = Case(kv=kv, q=q, hkv=1, dim=64, rows=1, slots=640, seed=3)
    c.ks = c.vs = None
    k, v = torch.zeros(c.k.shape), torch.ones(c.v.shape)
    k[:, :, ::2, 0], k[:, :, 1::2, 0] = 1.0, 0.9375
    v[:, :, 1::2] = -1.0
    c.k, c.v = k.to(kv), v.to(kv)
    query = torch.zeros(1, 8, 64)
    query[:, :, 0] = 1.0
    out, _ = A.dsv4_gqa_decode(query.to(q).cuda(), torch.tensor([640], dtype=torch.int32).cuda(), c.handle(A),
                               scale=scale, max_len=640)
    x = float(np.float32(scale))
    ref = (math.exp(x) - math.exp(0.9375 * x)) / (math.exp(x) + math.exp(0.9375 * x))
    # (sums as above; the scores are exact up to their rounding, 2^-23 of 4 log2 units)
    tol = 2.0 ** -17 + 2.0 ** -19 + 2.0 ** -20 + (640 / 16 + 64) * 2.0 ** -23 + ref * torch.finfo(q).eps / 2
    assert float((out.double() - ref).abs().max()) <= tol


@pytest.mark.parametrize("kv,q", [(BF, BF), (HF, HF), (F8, BF), (F8, HF)])
@pytest.mark.parametrize("step", [1, 2, 4, 8, 16, 32])
@pytest.mark.parametrize("sign", [1, -1])
def test_decode_of_scores_whose_spacing_is_coarse(A, kv, q, step, sign):
    # scores of step * (2^23 + i) log2 units, exact in fp32 and `step` apart, rising by one from tile to tile: what is
    # added to or taken from such a score is rounded to that spacing too
    c = Case(kv=kv, q=q, hkv=1, dim=64, rows=1, slots=400, seed=step)
    c.ks = c.vs = None
    i = (torch.arange(400) // 48).float()                    # i = 0 .. 8
    query = torch.zeros(1, 8, 64)
    query[:, :, 0], query[:, :, 1] = 2.0 ** 15, 1.0
    k = torch.zeros(400, 64)
    k[:, 0], k[:, 1] = sign * 256.0, i
    pages = c.table[0].long()
    kk = c.k.float()
    kk[pages] = k.view(-1, 16, 64)[:, None]
    c.k = kk.to(kv)
    assert torch.equal(c.k.float()[pages, 0].view(400, 64), k)
    log2e = np.float32(1.4426950408889634)
    scale = np.float32(step / 1.4426950408889634)
    near = [np.nextafter(scale, np.float32(0)), scale, np.nextafter(scale, np.float32(1e9))]
    scale = float([x for x in near if np.float32(x * log2e) == step][0])
    v = c.v.double()[pages, 0].view(400, 64)
    cache, n, w = c.handle(A), torch.tensor([400], dtype=torch.int32).cuda(), torch.zeros(1, 1, 400).cuda()
    p = torch.exp2(step * (i - i.max()).double())
    p /= p.sum()
    # (2^x: 2^-20, sums of 400 rows, pieces of P; a weight below 2^-36 of the largest may be lost beside f16)
    rel = 2.0 ** -20 + (400 / 16 + 64) * 2.0 ** -23 + (2.0 ** -12 if kv == F8 and q == BF else 2.0 ** -17)
    tol = (p @ v.abs()) * rel + (p @ v).abs() * (torch.finfo(q).eps / 2 + 2.0 ** -22) + \
        400 * 2.0 ** -36 * v.abs().max() + (2.0 ** -25 if q == HF else 0)
    for kw in ({}, {"weights": w, "req_pool_indices": torch.zeros(1, dtype=torch.int32).cuda()}):
        out, lse = A.dsv4_gqa_decode(query.to(q).cuda(), n, cache, scale=scale, max_len=400, **kw)
        assert ((out[0].double().cpu() - p @ v).abs() <= tol).all()
        assert float((lse.double().cpu() / (sign * step * 2.0 ** 23 * math.log(2)) - 1).abs().max()) <= 2.0 ** -19
    # (no bound on the weights: they are 2^(score - lse), and an fp32 lse of this size is rounded to the same spacing,
    # which is a factor of up to 2^(step / 2))
    assert A.dsv4_attn_get_device_error() == 0


def test_decode_sinks(A):
    c = Case(rows=3, slots=60, seed=7)
    for value in (-math.inf, -100.0, 0.0, 60.0, math.inf):
        check_decode(A, c, [60, 0, 7], 4, sink=torch.full((4,), value), weights=True)


def test_decode_request_rows_in_any_order_and_padding(A):
    c = Case(rows=6, slots=80, seed=8)
    # rows 4 and 1; a padded entry whose row is not one
    check_decode(A, c, [70, 0, 33], 4, req=[4, 99, 1], weights=True)
    check_decode(A, c, [70, 20, 33], 4, req=[4, -1, 1], weights=True, want_flags=O.ERR_REQ_ROW)


def test_decode_requests_that_share_a_row(A):
    c = Case(rows=4, slots=90, seed=10)
    check_decode(A, c, [80, 45, 0, 60, 88], 4, req=[2, 2, 2, 1, 2], weights=True, decay=0.25)


def test_decode_lengths_out_of_range(A):
    c = Case(rows=3, slots=96, seed=11)
    check_decode(A, c, [100, -4, 50], 4, max_len=90, weights=True, want_flags=O.ERR_GQA_LENGTH)


def test_decode_pages_outside_the_pool(A):
    c = Case(rows=3, slots=160, seed=12)
    c.table[0, 2], c.table[1, 0], c.table[2, 9] = -1, c.k.shape[0], 2 ** 30
    c.table[2, 1:] = -1
    check_decode(A, c, [160, 30, 16], 4, weights=True, want_flags=O.ERR_GQA_PAGE)
    c.table[0, :] = -1                       # not one readable row
    check_decode(A, c, [160, 0, 16], 4, weights=True, want_flags=O.ERR_GQA_PAGE)


def test_decode_strided_queries(A):
    c = Case(hkv=2, dim=64, rows=3, slots=50, seed=13)
    cache = c.handle(A)
    wide = torch.randn(3, 8 + 4, 64, generator=c.gen).to(BF).cuda()      # q, k and v of a projection
    q = wide[:, :8]
    lens = torch.tensor([50, 20, 31], dtype=torch.int32).cuda()
    out, lse = A.dsv4_gqa_decode(q, lens, cache)
    out2, lse2 = A.dsv4_gqa_decode(q.contiguous(), lens, cache)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    with pytest.raises(A.Dsv4Error):
        A.dsv4_gqa_decode(wide.transpose(1, 2)[:, :8].transpose(1, 2)[:, :, :64][:, ::2], lens, cache)


def test_decode_is_reproducible_and_in_place_equals_out_of_place(A):
    c = Case(kv=F8, hkv=4, dim=128, rows=5, slots=3000, seed=14)
    cache = c.handle(A)
    lens = torch.tensor([3000, 10, 1777, 0, 2048], dtype=torch.int32).cuda()
    q = c.query(5, 16).cuda()
    w = torch.rand(5, 4, 3008, generator=c.gen).cuda()
    got = []
    for _ in range(3):
        wo = torch.full_like(w, 3.0)
        out, lse = A.dsv4_gqa_decode(q, lens, cache, weights=w, weights_out=wo, decay=0.9)
        got.append((out.clone(), lse.clone(), wo))
    for o, l, x in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(l, got[0][1]) and torch.equal(x, got[0][2])
    inplace = w.clone()
    A.dsv4_gqa_decode(q, lens, cache, weights=inplace, decay=0.9)
    for b, n in enumerate(lens.tolist()):
        assert torch.equal(inplace[b, :, :n], got[0][2][b, :, :n])
        assert torch.equal(inplace[b, :, n:], w[b, :, n:]) and bool((got[0][2][b, :, n:] == 3.0).all())


def test_decode_in_a_graph_and_on_streams(A):
    c = Case(hkv=2, dim=128, rows=4, slots=2000, seed=15)
    cache = c.handle(A)
    q = c.query(4, 8).cuda()
    lens = torch.tensor([2000, 3, 700, 0], dtype=torch.int32).cuda()
    w = torch.zeros(4, 2, 2000).cuda()
    A.dsv4_gqa_decode(q, lens, cache, weights=w.clone())
    wo = torch.zeros_like(w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = A.dsv4_gqa_decode(q, lens, cache, weights=w, weights_out=wo)
    A.dsv4_gqa_decode(q, lens, cache)
    short = torch.cuda.CUDAGraph()
    with torch.cuda.graph(short):
        res = A.dsv4_gqa_decode(q, lens, cache)
    for now in ([2000, 3, 700, 0], [1, 1999, 0, 64], [0, 0, 0, 0]):
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        q.copy_(c.query(4, 8))
        wo.fill_(-1.0)
        graph.replay()
        torch.cuda.synchronize()
        x = torch.full_like(w, -1.0)
        o2, l2 = A.dsv4_gqa_decode(q, lens, cache, weights=w, weights_out=x)
        assert torch.equal(out, o2) and torch.equal(lse, l2) and torch.equal(wo, x)
        plain = A.dsv4_gqa_decode(q, lens, cache)
        short.replay()
        torch.cuda.synchronize()
        assert torch.equal(res[0], plain[0]) and torch.equal(res[1], plain[1])
    # two calls at once, each with its own workspace
    lens.copy_(torch.tensor([2000, 3, 700, 0], dtype=torch.int32))
    want = A.dsv4_gqa_decode(q, lens, cache)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams * 4:
        with torch.cuda.stream(s):
            got.append(A.dsv4_gqa_decode(q, lens, cache))
    s = torch.cuda.Stream()
    got.append(A.dsv4_gqa_decode(q, lens, cache, stream=s))
    torch.cuda.synchronize()
    for o, l in got:
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])


def test_calls_on_two_streams_without_workspaces(A):
    # a call on the current stream gives its scratch back when it returns, with its kernels still queued; the next
    # call, on another stream and of the same sizes, must not get it
    sets = []
    for i in range(2):
        c = Case(hkv=8, dim=128, page=64, rows=4, slots=20000, seed=80 + i)
        w = torch.rand(4, 8, 20032, generator=c.gen).cuda()
        lens = torch.tensor([20000, 7, 15000 - i, 19999], dtype=torch.int32).cuda()
        sets.append((c.handle(A), c.query(4, 16).cuda(), lens, w, c))
    s = torch.cuda.Stream()
    keep = 3000

    def call(i, stream, kept):
        cache, q, lens, w, c = sets[i]
        if kept == "evict":
            return [A.dsv4_gqa_evict(lens, cache, w, keep, weights_out=kept_out[i], stream=stream), kept_out[i]]
        wo = kept_out[i]
        return list(A.dsv4_gqa_decode(q, lens, cache, weights=w if kept else None, weights_out=wo if kept else None,
                                      stream=stream)) + [wo]

    for kept in (False, True, "evict"):
        pools = [(c.k_d.clone(), c.v_d.clone()) for *_, c in sets]
        kept_out = [torch.zeros_like(sets[i][3]) for i in range(2)]
        want = []
        for i in range(2):
            want.append([x.clone() for x in call(i, None, kept)])
            torch.cuda.synchronize()
        moved = [(c.k_d.clone(), c.v_d.clone()) for *_, c in sets]
        for _ in range(4):
            for (*_, c), (k, v) in zip(sets, pools):
                c.k_d.copy_(k)
                c.v_d.copy_(v)
            kept_out = [torch.zeros_like(sets[i][3]) for i in range(2)]
            torch.cuda.synchronize()
            got = [call(0, None, kept), call(1, s, kept)]
            torch.cuda.synchronize()
            for x, y in zip(got, want):
                assert all(torch.equal(p, r) for p, r in zip(x, y))
            for (*_, c), (k, v) in zip(sets, moved):
                assert np.array_equal(_bits(c.k_d), _bits(k)) and np.array_equal(_bits(c.v_d), _bits(v))
    assert A.dsv4_attn_get_device_error() == 0


def test_decode_of_nothing(A):
    c = Case(rows=2, slots=32)
    cache = c.handle(A)
    out, lse = A.dsv4_gqa_decode(c.query(0, 4).cuda(), torch.zeros(0, dtype=torch.int32).cuda(), cache)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)


def test_decode_offsets_beyond_32_bits(A):
    # a pool of 5 GB whose pages in use lie at its end
    pages = 160000
    k = torch.zeros(pages, 1, 128, 128, dtype=BF, device="cuda")
    v = torch.zeros_like(k)
    c = Case(hkv=1, dim=128, page=128, rows=2, slots=300, seed=16)
    own = c.table.long().flatten()
    k[pages - 1 - own.cuda()] = c.k[own].cuda()
    v[pages - 1 - own.cuda()] = c.v[own].cuda()
    lens = torch.tensor([300, 129], dtype=torch.int32).cuda()
    q = c.query(2, 8).cuda()
    far = A.make_gqa_cache(k, v, (pages - 1 - c.table.cuda()).to(torch.int32))
    out, lse = A.dsv4_gqa_decode(q, lens, far)
    want, wl = A.dsv4_gqa_decode(q, lens, c.handle(A))
    assert torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("lens", [[90000, 1, 88001], [60000, 0, 120001], [3, 5, 40]])
def test_decode_of_long_lists(A, lens):
    # enough tiles (16 slots each; over 64 for each of 1216 warps) that shares are claimed while the kernel runs; and
    # short lists in the same room.
    # Definition in 64 bits on the GPU; nothing may depend on who claims what.
    rows, hkv, heads, dim, page = 3, 8, 16, 128, 256
    width = -(-120001 // page)
    gen = torch.Generator(device="cuda").manual_seed(77)
    shape = (rows * width, hkv, page, dim)
    k, v = (torch.randn(shape, generator=gen, device="cuda", dtype=BF) for _ in range(2))
    table = torch.randperm(rows * width, generator=gen, device="cuda").view(rows, width).to(torch.int32)
    cache = A.make_gqa_cache(k, v, table)
    q = torch.randn(rows, heads, dim, generator=gen, device="cuda", dtype=BF)
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    w = torch.zeros(rows, hkv, width * page, device="cuda")
    got = []
    for _ in range(3):
        wo = torch.full_like(w, -1.0)
        out, lse = A.dsv4_gqa_decode(q, n, cache, weights=w, weights_out=wo)
        plain = A.dsv4_gqa_decode(q, n, cache)
        assert torch.equal(out, plain[0]) and torch.equal(lse, plain[1])
        got.append((out, lse, wo))
    assert A.dsv4_attn_get_device_error() == 0
    for x in got[1:]:
        assert all(torch.equal(p, r) for p, r in zip(x, got[0]))
    out, lse, wo = got[0]
    for b, m in enumerate(lens):
        assert bool((wo[b, :, m:] == -1.0).all())
        if m == 0:
            assert bool((out[b] == 0).all()) and bool(torch.isinf(lse[b]).all())
            continue
        for h in range(hkv):
            kk, vv = (x[table[b].long(), h].reshape(-1, dim)[:m].double() for x in (k, v))
            qq = q[b, 2 * h: 2 * h + 2].double()
            s = qq @ kk.T / math.sqrt(dim)
            ref_lse = torch.logsumexp(s, dim=1)
            p = torch.exp(s - ref_lse[:, None])
            ref = p @ vv
            mag = float((qq.abs() @ kk.abs().T).max()) / math.sqrt(dim)
            ds, sums = (dim + 8) * 2.0 ** -23 * mag, (m / 16 + 64) * 2.0 ** -23
            # (sums: as above; they grow with the rows of one share, not with m, but the bound need not be tight)
            tol = (2 * ds + 2.0 ** -20 + 2.0 ** -16 + sums) * (p @ vv.abs()) + (2.0 ** -8 + 2.0 ** -22) * ref.abs()
            assert bool(((out[b, 2 * h: 2 * h + 2].double() - ref).abs() <= tol).all())
            assert float((lse[b, 2 * h: 2 * h + 2].double() - ref_lse).abs().max()) <= ds + sums + 2.0 ** -18
            tw = p.sum(0) * (2 * ds + 2.0 ** -19 + sums)
            assert bool(((wo[b, h, :m].double() - p.sum(0)).abs() <= tw + 1e-12).all())


LONG = {
    # kv, q, head_dim, query heads per KV head, KV heads, page, window, lengths: so many tiles that shares are claimed
    "e4m3_64": (F8, BF, 64, 4, 8, 256, 0, [400000, 7, 250001]),
    "e4m3_64_f16": (F8, HF, 64, 10, 8, 64, 0, [350000, 300123]),
    "e4m3_128": (F8, BF, 128, 8, 8, 128, 0, [170000, 0, 160001]),
    "e4m3_256_wide": (F8, BF, 256, 16, 4, 256, 0, [200000, 130001]),
    "bf16_256": (BF, BF, 256, 2, 4, 256, 0, [100000, 1, 70001]),
    "f16_256_wide": (HF, HF, 256, 12, 2, 1024, 0, [200000, 130001]),
    "f16_128_groups": (HF, HF, 128, 17, 4, 16, 0, [120000, 50001, 33]),
    "bf16_64_window": (BF, BF, 64, 1, 16, 32, 5000, [5000 + 150 * i * (i % 3 > 0) + 7 * i for i in range(40)]),
    "bf16_128_many": (BF, BF, 128, 3, 8, 64, 0, [(9000 + 137 * i) * (i % 7 > 0) for i in range(37)]),
}


@pytest.mark.parametrize("name", sorted(LONG))
def test_decode_of_long_lists_of_every_shape(A, name):
    # claimed shares of every type, width and group size, compared with the definition in 64 bits (bounds as above);
    # with weights and without, bit for bit the same in every call
    kv, qt, dim, group, hkv, page, window, lens = LONG[name]
    rows, heads = len(lens), group * hkv
    row_bytes, fp8 = dim * (1 if kv == F8 else 2), kv == F8
    tile = max(16, 4096 // row_bytes)
    chunks = -(-group // (16 if group > 8 else 8))
    tiles = sum((n - 1) // tile - (max(0, n - window) if window else 0) // tile + 1 for n in lens if n) * hkv * chunks
    assert tiles >= 64 * 4 * (152 if row_bytes > 256 else 304)          # 64 per resident warp
    width = -(-max(lens) // page)
    gen = torch.Generator(device="cuda").manual_seed(len(name))
    pages = sum(-(-n // page) for n in lens)
    k, v = (torch.randn(pages, hkv, page, dim, generator=gen, device="cuda", dtype=BF).to(kv) for _ in range(2))
    order, table, at = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32), [], 0
    for n in lens:                              # (a table wider than a request's pages names none behind them)
        mine = order[at: at - (-n // page)]
        at += mine.numel()
        table.append(torch.nn.functional.pad(mine, (0, width - mine.numel()), value=-1))
    table = torch.stack(table)
    ks, vs = ((0.5 + torch.rand(hkv, generator=gen, device="cuda")) if fp8 else None for _ in range(2))
    cache = A.make_gqa_cache(k, v, table, k_scale=ks, v_scale=vs)
    q = torch.randn(rows, heads, dim, generator=gen, device="cuda", dtype=BF).to(qt)
    sink = torch.randn(heads, generator=gen, device="cuda")
    n_d = torch.tensor(lens, dtype=torch.int32).cuda()
    w = torch.zeros(rows, hkv, width * page, device="cuda")
    got = []
    for _ in range(3):
        wo = torch.full_like(w, -1.0)
        out, lse = A.dsv4_gqa_decode(q, n_d, cache, sink=sink, window=window, weights=w, weights_out=wo)
        plain = A.dsv4_gqa_decode(q, n_d, cache, sink=sink, window=window)
        assert torch.equal(out, plain[0]) and torch.equal(lse, plain[1])
        got.append((out, lse, wo))
    assert A.dsv4_attn_get_device_error() == 0
    for x in got[1:]:
        assert all(torch.equal(p, r) for p, r in zip(x, got[0]))
    out, lse, wo = got[0]
    piece = 2.0 ** -17 if not (fp8 and qt == BF) else 2.0 ** -12
    for b, m in enumerate(lens):
        assert bool((wo[b, :, m:] == -1.0).all())
        lo = max(0, m - window) if window else 0
        if m == 0:
            # (lse = sink, by way of log2 units: two fp32 products, 2^-24 each, by factors off by 2^-25 each)
            assert bool((out[b] == 0).all()) and bool(((lse[b] - sink).abs() <= 2.0 ** -22 * sink.abs()).all())
            continue
        for h in range(hkv):
            here = table[b, : -(-m // page)].long()
            kk, vv = ((x.view(torch.uint8)[here, h].view(F8) if fp8 else x[here, h]).reshape(-1, dim)[lo:m].double()
                      for x in (k, v))
            mine = slice(group * h, group * (h + 1))
            factor = (float(ks[h]) if fp8 else 1.0) / math.sqrt(dim)
            vmul = float(vs[h]) if fp8 else 1.0
            s = q[b, mine].double() @ kk.T * factor
            mag = float((q[b, mine].double().abs() @ kk.abs().T).max()) * factor
            ref_lse = torch.logaddexp(torch.logsumexp(s, dim=1), sink[mine].double())
            p = torch.exp(s - ref_lse[:, None])
            ref, soft = p @ vv * vmul, p @ vv.abs() * vmul
            ds, sums = (dim + 8) * 2.0 ** -23 * mag, ((m - lo) / 16 + 64) * 2.0 ** -23
            tail = 0 if kv == BF else p.max(dim=1, keepdim=True).values * (m - lo) * 2.0 ** -36 * float(vv.abs().max()) * vmul
            tol = (2 * ds + 2.0 ** -20 + piece + sums) * soft + tail + (torch.finfo(qt).eps / 2 + 2.0 ** -22) * ref.abs()
            if qt == HF:
                tol = tol + 2.0 ** -25
            assert bool(((out[b, mine].double() - ref).abs() <= tol).all())
            assert float((lse[b, mine].double() - ref_lse).abs().max()) <= ds + sums + 2.0 ** -18
            tw = p.sum(0) * (2 * ds + 2.0 ** -19 + sums)
            assert bool(((wo[b, h, lo:m].double() - p.sum(0)).abs() <= tw + 1e-12).all())
            assert bool((wo[b, h, :lo] == 0).all())


def test_long_lists_at_once_and_in_graphs(A):
    # two calls with claims on two streams: each grid's CTAs come and go as the other leaves room, so a CTA may take
    # over one that would have been resident; results stay bit for bit those of a call alone
    rows, hkv, heads, dim, page, n = 2, 8, 8, 128, 256, 90000
    width = -(-n // page)
    gen = torch.Generator(device="cuda").manual_seed(78)
    sets = []
    for i in range(2):
        k, v = (torch.randn(rows * width, hkv, page, dim, generator=gen, device="cuda", dtype=HF) for _ in range(2))
        table = torch.randperm(rows * width, generator=gen, device="cuda").view(rows, width).to(torch.int32)
        cache = A.make_gqa_cache(k, v, table)
        q = torch.randn(rows, heads, dim, generator=gen, device="cuda", dtype=HF)
        lens = torch.tensor([n, n - 777 * i - 1], dtype=torch.int32).cuda()
        sets.append((cache, q, lens, A.dsv4_gqa_decode(q, lens, cache)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(8):
        got = []
        for s, (cache, q, lens, _) in zip(streams, sets):
            with torch.cuda.stream(s):
                for _ in range(3):
                    got.append(A.dsv4_gqa_decode(q, lens, cache))
        torch.cuda.synchronize()
        for i, (out, lse) in enumerate(got):
            want = sets[i // 3][3]
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    graphs = []
    for cache, q, lens, _ in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = A.dsv4_gqa_decode(q, lens, cache)
        graphs.append((g, res))
    for _ in range(4):
        for s, (g, _) in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for (_, res), (_, _, _, want) in zip(graphs, sets):
            assert torch.equal(res[0], want[0]) and torch.equal(res[1], want[1])
    assert A.dsv4_attn_get_device_error() == 0


_CAPTURE = """
import torch
from hybrid_sparse_mqa_gb300 import attn as A
BF, F8 = torch.bfloat16, torch.float8_e4m3fn
gen = torch.Generator(device="cuda").manual_seed(1)
def rand(*shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=BF)
def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")
pages, hkv, page, dim = 40, 2, 256, {dim}
k, v = (rand(pages, hkv, page, dim).to({kv}) for _ in range(2))
cache = A.make_gqa_cache(k, v, torch.arange(pages, device="cuda", dtype=torch.int32).view(2, 20))
bits = lambda x: x.view(torch.uint8).clone()
q, wide, lens = rand(2, 4, dim), rand(2, 32, dim), ints(5000, 4000)
w, rows = torch.rand(2, hkv, 20 * page, device="cuda"), ints(1, 0)
new, slots = rand(2, 2 * hkv, dim), ints(5000, 4000)
calls = dict(
    long=lambda: A.dsv4_gqa_decode(q, lens, cache),
    kept=lambda: A.dsv4_gqa_decode(q, lens, cache, weights=w, weights_out=torch.zeros_like(w), req_pool_indices=rows),
    wide=lambda: A.dsv4_gqa_decode(wide, lens, cache), wide_short=lambda: A.dsv4_gqa_decode(wide, lens, cache, max_len=100),
    evict=lambda: [A.dsv4_gqa_evict(lens, cache, w, 1000, weights_out=torch.zeros_like(w)), bits(k), bits(v)],
)
# one short call of each function, of the forms with the fewest launches, is what was made before the captures
A.dsv4_gqa_decode(q, ints(3, 2), cache, max_len=100)
A.dsv4_gqa_store(new[:, :hkv], new[:, hkv:], ints(0, 1), slots, cache)
A.dsv4_gqa_evict(ints(3, 2), cache, w, 100, max_len=100)
A.dsv4_attn_get_device_error()
k0, v0 = bits(k), bits(v)
graphs = dict()
for name, call in calls.items():
    graphs[name] = (torch.cuda.CUDAGraph(), None)
    with torch.cuda.graph(graphs[name][0]):
        got = call()
    graphs[name] = (graphs[name][0], got)
for name, call in calls.items():
    for again in range(2):
        k.view(torch.uint8).copy_(k0), v.view(torch.uint8).copy_(v0)
        graphs[name][0].replay()
        torch.cuda.synchronize()
        first = [x.clone() for x in graphs[name][1]]
        k.view(torch.uint8).copy_(k0), v.view(torch.uint8).copy_(v0)
        assert all(torch.equal(x, y) for x, y in zip(first, call())), name
# (wide_short: lengths above max_len)
assert A.dsv4_attn_get_device_error() in (0, A.DEV_ERR["GQA_LENGTH"])
print("captured")
"""


@pytest.mark.parametrize("kv,dim", [("BF", 64), ("BF", 128), ("BF", 256), ("F8", 64), ("F8", 128), ("F8", 256)])
def test_captures_after_one_call_of_each_function(A, kv, dim):
    # in a process of its own: what an earlier test has launched is loaded already
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", _CAPTURE.format(kv=kv, dim=dim)], cwd=root, capture_output=True, text=True,
                         timeout=300)
    assert run.returncode == 0 and "captured" in run.stdout, run.stderr[-2000:]


def test_claims_that_are_given_up(A):
    # with one look for each answer, warps give up while theirs is on its way: the call ends and says so, and the next
    # one is right
    rows, hkv, heads, dim, page, n = 2, 8, 8, 128, 256, 90000
    width = -(-n // page)
    gen = torch.Generator(device="cuda").manual_seed(79)
    k, v = (torch.randn(rows * width, hkv, page, dim, generator=gen, device="cuda", dtype=BF) for _ in range(2))
    table = torch.arange(rows * width, device="cuda").view(rows, width).to(torch.int32)
    cache = A.make_gqa_cache(k, v, table)
    q = torch.randn(rows, heads, dim, generator=gen, device="cuda", dtype=BF)
    lens = torch.tensor([n, n - 5], dtype=torch.int32).cuda()
    want = A.dsv4_gqa_decode(q, lens, cache)
    assert A.dsv4_attn_get_device_error() == 0
    for _ in range(3):
        try:
            A.lib().dsv4_gqa_test_claim_limits(0, 1)
            A.dsv4_gqa_decode(q, lens, cache)
        finally:
            A.lib().dsv4_gqa_test_claim_limits(-1, -1)
        assert A.dsv4_attn_get_device_error() == A.DEV_ERR["TIMEOUT"]
        got = A.dsv4_gqa_decode(q, lens, cache)
        assert A.dsv4_attn_get_device_error() == 0
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ---------------------------------------------------------------- store
def _bits(x):
    x = x.detach().cpu()
    return x.contiguous().view(torch.uint8 if x.element_size() == 1 else torch.int16).numpy()


def _store_reference(case, k, v, req, slots):
    """The pools after the write, and the error bits (float32 quotients, the type's own rounding)."""
    got, err = [], 0
    for pool, x, scale in ((case.k, k, case.ks), (case.v, v, case.vs)):
        p = _bits(pool).copy()
        for i, (r, s) in enumerate(zip(req, slots)):
            if not (0 <= r < case.table.shape[0] and 0 <= s < case.width * case.page):
                err |= O.ERR_STORE_ROW
                continue
            page = int(case.table[r, s // case.page])
            if not 0 <= page < pool.shape[0]:
                err |= O.ERR_STORE_ROW
                continue
            row = x[i]
            if case.kv == F8:
                row = (row.float() / scale[:, None]).clamp(-448, 448).to(F8)
            p[page, :, s % case.page] = _bits(row)
        got.append(p)
    return got, err


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("kv,q", [(BF, BF), (HF, HF), (F8, BF), (F8, HF)])
@pytest.mark.parametrize("token_major", [False, True])
def test_store_matches(A, kv, q, dim, token_major):
    c = Case(kv=kv, q=q, hkv=3, dim=dim, rows=4, slots=70, seed=dim, token_major=token_major)
    cache = c.handle(A)
    n = 41
    cells = torch.randperm(4 * 70, generator=c.gen)[:n]
    req, slots = (cells // 70).to(torch.int32), (cells % 70).to(torch.int32)
    wide = torch.randn(n, 6, dim, generator=c.gen).to(q)
    wide[3] *= 1e4 if q == HF else 1e30                        # saturates
    wide[4] = 0.0
    wide[5, :, ::2] = -0.0
    wide[6, :, :8] = torch.tensor([1e-8, -1e-8, 2e-3, -2e-3, 464.0, -464.0, 1.0625, 6e-5]).to(q)
    k, v = wide[:, :3], wide[:, 3:]
    w, pos = torch.rand(4, 3, 80, generator=c.gen), torch.randint(0, 99, (4, 3, 80), generator=c.gen, dtype=torch.int32)
    tp = torch.randint(0, 1 << 30, (n,), generator=c.gen, dtype=torch.int32)
    w_d, pos_d, wide_d = w.cuda(), pos.cuda(), wide.cuda()
    A.dsv4_gqa_store(wide_d[:, :3], wide_d[:, 3:], req.cuda(), slots.cuda(), cache, weights=w_d, positions=pos_d,
                     token_positions=tp.cuda())
    torch.cuda.synchronize()
    assert A.dsv4_attn_get_device_error() == 0
    want, err = _store_reference(c, k, v, req.tolist(), slots.tolist())
    assert err == 0
    assert np.array_equal(_bits(c.k_d), want[0]) and np.array_equal(_bits(c.v_d), want[1])
    w[req.long(), :, slots.long()] = 0.0
    pos[req.long(), :, slots.long()] = tp[:, None].expand(-1, 3)
    assert torch.equal(w_d.cpu(), w) and torch.equal(pos_d.cpu(), pos)


@pytest.mark.parametrize("q", [BF, HF])
def test_store_rounds_every_value_as_the_quotient_does(A, q):
    # every value of the input's type, against scales that are not powers of two,
    # among them the first ones that are divided by instead of multiplied
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(q)
    x = torch.cat([bits, torch.zeros(-len(bits) % 128, dtype=q)]).view(-1, 1, 128)
    n = x.shape[0]
    edges = (2.0 ** -60, 1.3 * 2.0 ** 60, 1e-30) if q == BF else (2.0 ** -23, 127.0, 127.1, 1e-8)
    for scale in (1.0, 0.02173, 3.7e-3, 1.4142135, 97.3, 1023.7) + edges:
        c = Case(kv=F8, q=q, hkv=1, dim=128, rows=1, slots=n, page=256)
        c.ks = torch.tensor([scale])
        c.vs = torch.tensor([scale * 1.09])
        cache = c.handle(A)
        A.dsv4_gqa_store(x.cuda(), x.cuda(), torch.zeros(n, dtype=torch.int32).cuda(),
                         torch.arange(n, dtype=torch.int32).cuda(), cache)
        want, _ = _store_reference(c, x, x, [0] * n, list(range(n)))
        for got, ref in ((c.k_d, want[0]), (c.v_d, want[1])):
            g = _bits(got)
            nan = (ref & 0x7F) == 0x7F                 # (a NaN's sign is not a value)
            assert np.array_equal((g & 0x7F) == 0x7F, nan) and np.array_equal(g[~nan], ref[~nan]), scale


def test_store_of_values_without_a_code(A):
    # infinities saturate, NaN stays NaN; no scale means one
    x = torch.zeros(1, 1, 64)
    x[0, 0, :4] = torch.tensor([math.inf, -math.inf, math.nan, 3e38])
    c = Case(kv=F8, hkv=1, rows=1, slots=16)
    c.ks = c.vs = None
    cache = c.handle(A)
    zero = torch.zeros(1, dtype=torch.int32).cuda()
    A.dsv4_gqa_store(x.to(BF).cuda(), x.to(BF).cuda(), zero, zero, cache)
    row = c.k_d[int(c.table[0, 0]), 0, 0].float().cpu()
    assert row[:2].tolist() == [448.0, -448.0] and bool(torch.isnan(row[2])) and row[3] == 448.0
    assert bool((row[4:] == 0).all())


def test_store_reports_rows_without_a_place(A):
    c = Case(hkv=2, rows=3, slots=64, seed=21)
    c.table[1, 2], c.table[2, 0] = -1, c.k.shape[0]
    cache = c.handle(A)
    req = [0, -1, 3, 1, 2, 0, 0, 1]
    slots = [5, 0, 0, 40, 3, -1, 64, 10]
    x = torch.randn(8, 4, 64, generator=c.gen).to(BF)
    w = torch.full((3, 2, 64), 5.0).cuda()
    A.dsv4_gqa_store(x[:, :2].cuda(), x[:, 2:].cuda(), torch.tensor(req, dtype=torch.int32).cuda(),
                     torch.tensor(slots, dtype=torch.int32).cuda(), cache, weights=w)
    torch.cuda.synchronize()
    flags = A.dsv4_attn_get_device_error()
    want, err = _store_reference(c, x[:, :2], x[:, 2:], req, slots)
    assert flags == err == O.ERR_STORE_ROW
    assert np.array_equal(_bits(c.k_d), want[0]) and np.array_equal(_bits(c.v_d), want[1])
    assert sorted(torch.nonzero(w.cpu() == 0).tolist()) == [[0, 0, 5], [0, 1, 5], [1, 0, 10], [1, 1, 10]]
    # a slot that the tracking arrays are too narrow for has no place either
    narrow = torch.full((3, 2, 8), 5.0).cuda()
    before = _bits(c.k_d)
    one = torch.zeros(1, dtype=torch.int32).cuda()
    A.dsv4_gqa_store(x[:1, :2].cuda(), x[:1, 2:].cuda(), one, one + 9, cache, weights=narrow)
    assert A.dsv4_attn_get_device_error() == O.ERR_STORE_ROW
    assert np.array_equal(before, _bits(c.k_d)) and bool((narrow == 5.0).all())
    A.dsv4_gqa_store(x[:0, :2].cuda(), x[:0, 2:].cuda(), one[:0], one[:0], cache)
    assert A.dsv4_attn_get_device_error() == 0


# ---------------------------------------------------------------- evict
def check_evict(A, c, lens, keep, *, first=0, recent=0, seen=None, positions=None, req=None, w=None, max_len=None,
                want_flags=0, inplace=False):
    cache = c.handle(A)
    slots = c.width * c.page
    rows = c.table.shape[0]
    w = torch.rand(rows, c.hkv, slots + 3, generator=c.gen) if w is None else w
    max_len = slots if max_len is None else max_len
    fill = None if inplace else torch.full_like(w, -3.0)
    pfill = None if inplace or positions is None else torch.full_like(positions, -3)
    d = lambda x: None if x is None else x.cuda()       # noqa: E731
    i32 = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32)      # noqa: E731
    w_d, wo_d, p_d, po_d, lens_d = d(w), d(fill), d(positions), d(pfill), d(i32(lens))
    got = A.dsv4_gqa_evict(lens_d, cache, w_d, keep, seq_lens=d(i32(seen)), positions=p_d, first=first, recent=recent,
                           req_pool_indices=d(i32(req)), max_len=max_len, weights_out=wo_d, positions_out=po_d,
                           lens_out=lens_d if inplace else None)
    torch.cuda.synchronize()
    flags = A.dsv4_attn_get_device_error()
    cache64 = {"k": _bits(c.k), "v": _bits(c.v), "table": c.table.numpy()}
    n_out, k, v, wo, po, err = O.gqa_evict(
        lens, cache64, w.numpy(), keep, max_len=max_len, first=first, recent=recent, seq_lens=seen,
        positions=None if positions is None else positions.numpy(), req=req,
        weights_out=None if fill is None else fill.numpy(), positions_out=None if pfill is None else pfill.numpy())
    assert flags == err == want_flags, (flags, err)
    assert got.cpu().tolist() == n_out.tolist()
    assert np.array_equal((w_d if inplace else wo_d).cpu().numpy(), wo, equal_nan=True)
    if positions is not None:
        assert np.array_equal((p_d if inplace else po_d).cpu().numpy(), po)
    assert np.array_equal(_bits(c.k_d), k) and np.array_equal(_bits(c.v_d), v)
    return cache


def _positions(c, seen, lens):
    """Distinct positions below seen[b] in every request's slots, in any order."""
    slots = c.width * c.page
    p = torch.zeros(c.table.shape[0], c.hkv, slots + 3, dtype=torch.int32)
    for r, (n, top) in enumerate(zip(lens, seen)):
        for h in range(c.hkv):
            p[r, h, :n] = torch.randperm(top, generator=c.gen)[:n].to(torch.int32)
    return p


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("kv,dim,token_major", [(BF, 64, False), (HF, 128, True), (F8, 64, False), (F8, 256, True)])
def test_evict_matches(A, kv, dim, token_major, inplace):
    lens = [0, 1, 39, 40, 41, 57, 100, 128]
    c = Case(kv=kv, hkv=3, dim=dim, rows=8, slots=128, seed=dim, token_major=token_major)
    seen = [n + 30 for n in lens]
    check_evict(A, c, lens, 40, first=3, recent=10, seen=seen, positions=_positions(c, seen, lens), inplace=inplace)


@pytest.mark.parametrize("keep", [1, 2, 31, 32, 33, 64, 99, 100, 127, 128])
def test_evict_bounds(A, keep):
    c = Case(hkv=2, rows=3, slots=128, seed=keep)
    check_evict(A, c, [128, 100, 33], keep)
    check_evict(A, c, [128, 100, 33], keep, recent=keep)
    check_evict(A, c, [128, 100, 33], keep, first=keep)


@pytest.mark.parametrize("rows,slots,keep", [(1, 5000, 4999), (1, 9000, 100), (2, 40000, 20000), (1, 70000, 64000),
                                             (20, 5000, 2500), (1, 420000, 1000)])
def test_evict_long_rows(A, rows, slots, keep):
    # clusters of 1 to 8 CTAs; the longest row does not fit their shared memory
    c = Case(hkv=1, rows=rows, slots=slots, page=1024, seed=slots)
    w = torch.rand(rows, 1, c.width * c.page + 3, generator=c.gen)
    w = torch.where(torch.rand(w.shape, generator=c.gen) < 0.3, torch.round(w * 50) / 50, w)     # many equal ones
    check_evict(A, c, [slots - 17 * r for r in range(rows)], keep, first=2, recent=60, w=w)


def test_evict_equal_and_special_weights(A):
    c = Case(hkv=2, rows=4, slots=300, seed=31)
    for kind in range(4):
        w = torch.zeros(4, 2, 304 + 3)
        if kind == 1:
            w[:] = torch.tensor([0.0, -0.0, 1e-45, -1e-45, math.inf, -math.inf, math.nan, 3e38])[
                torch.randint(0, 8, w.shape, generator=c.gen)]
        if kind == 2:
            w[:] = math.nan
        if kind == 3:
            w = -torch.rand(w.shape, generator=c.gen)
        check_evict(A, c, [300, 299, 120, 150], 128, w=w, recent=20)
        check_evict(A, c, [300, 299, 297, 296], 296, w=w, recent=20)       # one to four rows too many
        check_evict(A, c, [300, 298, 120, 150], 296, w=w, recent=296, inplace=True)


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("kv,dim,token_major", [(BF, 64, False), (HF, 256, True), (F8, 64, True), (F8, 128, False)])
def test_evict_a_step_of_a_full_cache(A, kv, dim, token_major, inplace):
    # no request can be more than four rows over the bound
    c = Case(kv=kv, hkv=3, dim=dim, rows=9, slots=140, seed=dim, token_major=token_major)
    lens = [132, 131, 130, 129, 128, 100, 1, 0, 132]
    seen = [n + 50 for n in lens]
    pos = _positions(c, seen, lens)
    check_evict(A, c, lens, 128, max_len=132, inplace=inplace)
    check_evict(A, c, lens, 128, max_len=132, first=3, recent=20, seen=seen, positions=pos, inplace=inplace)
    check_evict(A, c, lens, 128, max_len=132, recent=128, inplace=inplace)
    check_evict(A, c, [132, 3, 140, 0, 129], 128, req=[8, 40, 0, 77, 0], max_len=132, inplace=inplace,
                want_flags=O.ERR_REQ_ROW | O.ERR_GQA_LENGTH)
    w = torch.zeros(9, 3, 147)
    w[:, :, ::3] = math.nan
    check_evict(A, c, lens, 128, max_len=132, w=w, inplace=inplace)
    c.table[0, 8], c.table[1, 0] = -1, 10 ** 6
    check_evict(A, c, lens, 128, max_len=132, w=w, inplace=inplace, want_flags=O.ERR_GQA_PAGE)


@pytest.mark.parametrize("slack", [2, 40])
def test_evict_with_new_lengths_in_place_of_the_tokens_seen(A, slack):
    # slack 2: one launch, whose CTAs read the tokens seen for every KV head
    rows, keep = 40, 128
    c = Case(hkv=8, dim=64, rows=rows, slots=keep + slack, seed=slack)
    lens = torch.full((rows,), keep + slack, dtype=torch.int32, device="cuda")
    w = torch.rand(rows, 8, keep + slack, generator=c.gen)
    results = []
    for same in (False, True):
        cache, w_d, seen = c.handle(A), w.cuda(), lens.clone()
        got = A.dsv4_gqa_evict(lens, cache, w_d, keep, seq_lens=seen, recent=30, max_len=keep + slack,
                               lens_out=seen if same else None)
        results.append((got, w_d[:, :, :keep], c.k_d, c.v_d))
    assert A.dsv4_attn_get_device_error() == 0
    for x, y in zip(*results):
        assert torch.equal(x.view(torch.int16) if x.dtype == BF else x, y.view(torch.int16) if y.dtype == BF else y)


def test_evict_a_step_of_long_caches(A):
    for slots in (5000, 12000, 30000, 40000):
        c = Case(hkv=2, rows=2, slots=slots, page=1024, seed=slots)
        check_evict(A, c, [slots, slots - 2], slots - 3, first=4, recent=100, max_len=slots)


def test_evict_rows_named_in_any_order_twice_or_not_at_all(A):
    c = Case(hkv=2, rows=5, slots=96, seed=32)
    check_evict(A, c, [90, 0, 70], 40, req=[3, 77, 0])
    check_evict(A, c, [90, 80, 0, 70], 40, req=[3, 3, 3, 0], want_flags=O.ERR_REQ_ROW)
    check_evict(A, c, [90, 20, 70], 40, req=[3, 5, 0], want_flags=O.ERR_REQ_ROW)


def test_evict_lengths_and_pages_out_of_range(A):
    c = Case(hkv=2, rows=3, slots=96, seed=33)
    check_evict(A, c, [200, -5, 60], 40, max_len=90, want_flags=O.ERR_GQA_LENGTH)
    c.table[0, 0], c.table[2, 3] = -1, 10 ** 6
    check_evict(A, c, [96, 30, 64], 40, want_flags=O.ERR_GQA_PAGE)


def test_evict_in_a_graph(A):
    c = Case(hkv=2, rows=3, slots=128, seed=34)
    cache = c.handle(A)
    w = torch.rand(3, 2, 128, generator=c.gen)
    lens = torch.tensor([128, 20, 100], dtype=torch.int32).cuda()
    wi, wo, n = w.cuda(), torch.zeros(3, 2, 128).cuda(), torch.zeros(3, dtype=torch.int32).cuda()
    k0, v0 = c.k_d.clone(), c.v_d.clone()
    A.dsv4_gqa_evict(lens, cache, wi, 64, weights_out=wo, lens_out=n)
    want = (_bits(c.k_d).copy(), _bits(c.v_d).copy(), wo.clone(), n.clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        A.dsv4_gqa_evict(lens, cache, wi, 64, weights_out=wo, lens_out=n)
    for _ in range(2):
        c.k_d.copy_(k0)
        c.v_d.copy_(v0)
        wo.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(_bits(c.k_d), want[0]) and np.array_equal(_bits(c.v_d), want[1])
        assert torch.equal(wo, want[2]) and torch.equal(n, want[3])


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("kv", [BF, F8])
def test_a_bounded_cache_over_many_steps(A, kv):
    """Write, attend, accumulate, evict: a decode loop whose caches never grow
    past a bound, every step against the oracle run on the same cache."""
    rows, hkv, heads, dim, bound = 3, 2, 8, 64, 48
    c = Case(kv=kv, hkv=hkv, dim=dim, rows=rows, slots=64, seed=40)
    cache = c.handle(A)
    w = torch.zeros(rows, hkv, 64).cuda()
    pos = torch.zeros(rows, hkv, 64, dtype=torch.int32).cuda()
    prompt = [40, 10, 47]
    lens = torch.tensor(prompt, dtype=torch.int32).cuda()
    seen = lens.clone()
    req = torch.arange(rows, dtype=torch.int32).cuda()
    for r, n in enumerate(prompt):          # the prompt rows are what the pool holds; their positions are their slots
        pos[r, :, :n] = torch.arange(n, dtype=torch.int32).cuda()
    for step in range(30):
        new = torch.randn(rows, 2 * hkv, dim, generator=c.gen).to(c.qt).cuda()
        q = c.query(rows, heads).cuda()
        A.dsv4_gqa_store(new[:, :hkv], new[:, hkv:], req, lens, cache, weights=w, positions=pos, token_positions=seen)
        lens += 1
        seen += 1
        before = w.clone()
        out, lse = A.dsv4_gqa_decode(q, lens, cache, weights=w, max_len=64)
        c.k, c.v = c.k_d.cpu(), c.v_d.cpu()
        ref, rlse, rw, err, _ = O.gqa_decode(q.double().cpu().numpy(), lens.tolist(), c.oracle(), max_len=64,
                                             scale=1 / math.sqrt(dim), weights=before.double().cpu().numpy(),
                                             weights_out=before.double().cpu().numpy())
        assert err == 0
        # scores of a few units over at most 64 rows: rounding of the output (2^-8) and, for
        # e4m3 caches, of P (2^-11) times values below 6
        assert np.abs(out.double().cpu().numpy() - ref).max() <= 2.0 ** -8 * np.abs(ref).max() + 6 * 1.5 * 2.0 ** -11
        assert np.abs(w.double().cpu().numpy() - rw).max() <= 1e-4
        pool = {"k": _bits(c.k), "v": _bits(c.v), "table": c.table.numpy()}
        n_out, k, v, wo, po, err = O.gqa_evict(lens.tolist(), pool, w.cpu().numpy(), bound, max_len=64, first=2,
                                               recent=8, seq_lens=seen.tolist(), positions=pos.cpu().numpy())
        A.dsv4_gqa_evict(lens, cache, w, bound, seq_lens=seen, positions=pos, first=2, recent=8, max_len=64,
                         lens_out=lens)
        assert err == 0 and A.dsv4_attn_get_device_error() == 0
        assert lens.tolist() == n_out.tolist() and max(n_out) <= bound
        assert np.array_equal(_bits(c.k_d), k) and np.array_equal(_bits(c.v_d), v)
        assert np.array_equal(w.cpu().numpy(), wo) and np.array_equal(pos.cpu().numpy(), po)
    # the first positions and the newest ones are all still there
    for r in range(rows):
        for h in range(hkv):
            left = set(pos[r, h, : int(lens[r])].tolist())
            top = int(seen[r])
            assert {0, 1} | set(range(top - 8, top)) <= left
