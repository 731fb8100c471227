"""The 4-bit grouped-query cache on the GPU against the float64 oracle: its write, its reading back, the attention over
it and its eviction.

Write, read-back and eviction move and round values by rules that fix every bit, so they are compared exactly.  Decode
is compared element by element with a bound built from its arithmetic, for n rows of which a head's scores are at most
m in magnitude before cancellation (m = scale * max_j sum |q||k_j|); codes times block scales are exact in f16:
  score      fp32 accumulation of D products, three factors:  ds = (D + 8) 2^-23 m
  p          2^x of the score in fp32: relative 2 ds + 2^-20 (both sides of the quotient)
  P's rounding for the MMA: one f16 (bf16 outputs) 2^-11, two (f16 outputs) 2^-16, plus 2^-36 of the largest p
  sums       fp32 over n / 16 steps and the joins: (n / 16 + 64) 2^-23
  output     half a step of its type, relative
"""
import math

import numpy as np
import pytest
import torch

from oracle import gqa_oracle as O
from tests._gqa4 import BF, F8, HF, Cache4, lay, pack, to_device

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def A():
    from hybrid_sparse_mqa_gb300 import build
    build.build()
    from hybrid_sparse_mqa_gb300 import attn
    attn.lib()
    attn.dsv4_attn_get_device_error()
    return attn


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


# ---------------------------------------------------------------- the write
def new_rows(n, hkv, dim, dtype, gen):
    """Rows of all sizes, with zero blocks, lone large values, both zeros and values next to the codes' borders."""
    x = torch.randn(n, hkv, dim, generator=gen) * torch.exp2(torch.randint(-6, 7, (n, hkv, 1), generator=gen).float())
    b = x.view(n, hkv, dim // 16, 16)
    b[torch.rand(b.shape[:3], generator=gen) < 0.05] = 0.0
    near = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.0, -0.0, -0.25, -5.0, 1e-6, -1e-6, 4.0, 3.0])
    pick = torch.rand(b.shape[:3], generator=gen) < 0.2
    step = torch.exp2(torch.randint(-5, 3, b.shape[:3], generator=gen).float())[..., None]
    b[pick] = (near * step)[pick]
    return x.to(dtype)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("q", [BF, HF])
@pytest.mark.parametrize("token_major", [False, True])
@pytest.mark.parametrize("scaled", [False, True])
def test_store_matches(A, q, dim, token_major, scaled):
    c = Cache4(q=q, hkv=3, dim=dim, page=32, rows=4, slots=150, seed=dim, token_major=token_major, scaled=scaled)
    cache = c.handle(A)
    n = 157
    x = new_rows(n, 6, dim, q, c.gen).cuda()
    k, v = x[:, ::2], x[:, 1::2]                                  # strided heads
    where = torch.randperm(4 * 150, generator=c.gen)[:n]
    req, slots = (where // 150).int(), (where % 150).int()
    w = torch.rand(4, 3, 160, generator=c.gen)
    pos = torch.randint(0, 1000, (4, 3, 160), generator=c.gen, dtype=torch.int32)
    tok = torch.randint(0, 1000, (n,), generator=c.gen, dtype=torch.int32)
    w_d, pos_d = w.cuda(), pos.cuda()
    A.dsv4_gqa_store(k, v, req.cuda(), slots.cuda(), cache, weights=w_d, positions=pos_d, token_positions=tok.cuda())
    assert A.dsv4_attn_get_device_error() == 0
    for new, codes, blocks, scale in ((k, c.k, c.kb, c.ks), (v, c.v, c.vb, c.vs)):
        got = pack(new.cpu(), scale)
        for i, (r, s) in enumerate(zip(req.tolist(), slots.tolist())):
            p = int(c.table[r, s // 32])
            codes[p, :, s % 32], blocks[p, :, s % 32] = got[0][i], got[1][i]
    for i, (r, s) in enumerate(zip(req.tolist(), slots.tolist())):
        w[r, :, s], pos[r, :, s] = 0.0, tok[i]
    for got, want in ((c.k_d, c.k), (c.v_d, c.v), (c.kb_d, c.kb), (c.vb_d, c.vb), (w_d, w), (pos_d, pos)):
        assert torch.equal(got.cpu(), want)                       # everything else is as it was


@pytest.mark.parametrize("q", [BF, HF])
@pytest.mark.parametrize("scale", [1.0, 0.37, 1 / 3, 2.0 ** -14, 15.9, 2.0 ** -20, 300.0, 2.0 ** -65, 2.0 ** 65])
def test_store_of_every_size(A, q, scale):
    # every 16-bit value beside each block maximum of its size; heads' scales inside and outside the range in which
    # quotients are had without dividing
    bits = torch.arange(0, 1 << 16, dtype=torch.int32).to(torch.int16)
    x = bits.view(q).float()
    x = x[torch.isfinite(x)]
    x = x[(x.abs() < 1e37)]
    n = x.numel() // 512
    x = torch.cat([x[torch.randperm(x.numel(), generator=torch.Generator().manual_seed(5))][: n * 512],
                   x[: n * 512]]).view(-1, 1, 64).to(q)
    n = x.shape[0]
    c = Cache4(q=q, hkv=1, dim=64, rows=1, slots=n, seed=1)
    c.ks = c.vs = torch.full((1,), scale)
    cache = c.handle(A)
    x = x.cuda()
    A.dsv4_gqa_store(x, -x, i32([0] * n), torch.arange(n, dtype=torch.int32).cuda(), cache)
    pages = c.table[0].long()
    for pool, blocks, new in ((c.k_d, c.kb_d, x), (c.v_d, c.vb_d, -x)):
        codes, scales = pack(new.cpu(), c.ks)
        assert torch.equal(blocks.cpu()[pages, 0].reshape(-1, 4)[:n], scales[:, 0])
        assert torch.equal(pool.cpu()[pages, 0].reshape(-1, 32)[:n], codes[:, 0])


def test_store_of_values_without_a_code(A):
    for q in (BF, HF):
        for scale in (1.0, 40.0, 1e-30):
            c = Cache4(q=q, hkv=1, dim=64, rows=1, slots=4, seed=2)
            c.ks = c.vs = torch.full((1,), scale)
            cache = c.handle(A)
            x = torch.zeros(4, 1, 64)
            x[0, 0, 3], x[0, 0, 20] = math.nan, math.inf
            x[1, 0, :16] = -math.inf
            x[1, 0, 17] = -math.nan
            x[2, 0, 5], x[2, 0, 6], x[2, 0, 33] = math.inf, 1.0, torch.finfo(q).smallest_normal
            x[3] = torch.finfo(q).max
            x = x.to(q)
            A.dsv4_gqa_store(x.cuda(), (-x).cuda(), i32([0] * 4), i32([0, 1, 2, 3]), cache)
            page = int(c.table[0, 0])
            for pool, blocks, new in ((c.k_d, c.kb_d, x), (c.v_d, c.vb_d, -x)):
                codes, scales = pack(new, c.ks)
                assert torch.equal(blocks.cpu()[page, 0, :4], scales[:, 0])
                assert torch.equal(pool.cpu()[page, 0, :4], codes[:, 0])
            k, _ = A.dsv4_gqa_load(i32([0, 0]), i32([0, 1]), cache)
            assert k[0, 0, :16].isnan().all() and not k[0, 0, 16:].isnan().any() and k[1, 0, 16:32].isnan().all()
            top = torch.tensor(6 * 448 * np.float32(scale), dtype=BF)
            assert (k[1, 0, :16].cpu() == -top).all() and k[0, 0, 20] == top


def test_rows_without_a_place(A):
    c = Cache4(hkv=2, dim=128, rows=2, slots=40, seed=3)
    c.table[1, 1] = -1
    c.table[1, 2] = 10 ** 6
    cache = c.handle(A)
    x = torch.ones(8, 2, 128, dtype=BF).cuda()
    req, slots = i32([0, -1, 2, 0, 0, 1, 1, 1]), i32([5, 0, 0, -1, 48, 20, 40, 3])
    A.dsv4_gqa_store(x, x, req, slots, cache)
    assert A.dsv4_attn_get_device_error() == O.ERR_STORE_ROW
    codes, blocks = pack(x.cpu(), c.ks)
    for r, s, i in ((0, 5, 0), (1, 3, 7)):
        p = int(c.table[r, 0])
        c.k[p, :, s], c.kb[p, :, s] = codes[i], blocks[i]
    assert torch.equal(c.k_d.cpu(), c.k) and torch.equal(c.kb_d.cpu(), c.kb)
    k, v = (torch.full((8, 2, 128), 7.0, dtype=BF).cuda() for _ in range(2))
    A.dsv4_gqa_load(req, slots, cache, k=k, v=v)
    assert A.dsv4_attn_get_device_error() == O.ERR_LOAD_ROW
    assert (k[1:7] == 0).all() and (v[1:7] == 0).all() and (k[[0, 7]] != 0).all()
    A.dsv4_gqa_load(req[:1], slots[:1], cache)
    assert A.dsv4_attn_get_device_error() == 0


# ---------------------------------------------------------------- the way back
class Plain:
    """A bf16, f16 or e4m3 cache with the fields of Cache4 that reading it back needs."""

    def __init__(self, kv, q, hkv, dim, page, rows, slots, seed, token_major):
        g = torch.Generator().manual_seed(seed)
        width = -(-slots // page)
        order = torch.randperm(rows * width + 2, generator=g)
        self.table = order[: rows * width].view(rows, width).to(torch.int32).contiguous()
        self.gen, self.page = g, page
        shape = (rows * width + 2, hkv, page, dim)
        self.k, self.v = (lay((torch.randn(shape, generator=g) * 3).to(kv), token_major) for _ in range(2))
        self.ks, self.vs = ((0.5 + torch.rand(hkv, generator=g) if kv == F8 else None) for _ in range(2))

    def handle(self, A):
        raw = [to_device(x.view(torch.uint8)).view(F8) if x.dtype == F8 else to_device(x) for x in (self.k, self.v)]
        return A.make_gqa_cache(*raw, self.table.cuda(), k_scale=to_device(self.ks), v_scale=to_device(self.vs))

    def oracle(self):
        return {"k": self.k.double().numpy(), "v": self.v.double().numpy(), "table": self.table.numpy(),
                "k_scale": None if self.ks is None else self.ks.double().numpy(),
                "v_scale": None if self.vs is None else self.vs.double().numpy()}


def twice_rounded(x, q):
    """Float64 x rounded to fp32 and then to q, as the library's product and its result are."""
    return torch.from_numpy(x).float().to(q)


@pytest.mark.parametrize("token_major", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("kv,q", [("e2m1", BF), ("e2m1", HF), (F8, BF), (F8, HF), (BF, BF), (HF, HF)])
def test_load_matches(A, kv, q, dim, token_major):
    make = dict(hkv=3, dim=dim, page=32, rows=4, slots=150, seed=dim, token_major=token_major)
    c = Cache4(q=q, wide_scales=True, **make) if kv == "e2m1" else Plain(kv, q, **make)
    cache = c.handle(A)
    for n in (1, 3, 33, 200):
        req = torch.randint(0, 4, (n,), generator=c.gen, dtype=torch.int32)
        slots = torch.randint(0, 150, (n,), generator=c.gen, dtype=torch.int32)
        want = [twice_rounded(x, q) for x in O.gqa_load(req.tolist(), slots.tolist(), c.oracle())[:2]]
        got = A.dsv4_gqa_load(req.cuda(), slots.cuda(), cache, dtype=q)
        both = torch.full((n, 6, dim), 7.0, dtype=q).cuda()       # K and V heads in turn, as a projection's rows
        A.dsv4_gqa_load(req.cuda(), slots.cuda(), cache, k=both[:, ::2], v=both[:, 1::2])
        rows = torch.full((2, 3, n, dim + 8), 7.0, dtype=q).cuda()     # heads first, padded rows
        A.dsv4_gqa_load(req.cuda(), slots.cuda(), cache, k=rows[0, :, :, :dim].transpose(0, 1),
                        v=rows[1, :, :, :dim].transpose(0, 1))
        for i in range(2):
            assert torch.equal(got[i].cpu(), want[i])
            assert torch.equal(both[:, i::2].cpu(), want[i])
            assert torch.equal(rows[i, :, :, :dim].transpose(0, 1).cpu(), want[i])
        assert (rows[..., dim:] == 7.0).all()
    assert A.dsv4_attn_get_device_error() == 0


def test_load_of_nothing_and_of_one_row_many_times(A):
    c = Cache4(hkv=1, dim=64, rows=1, slots=20)
    cache = c.handle(A)
    k, v = A.dsv4_gqa_load(i32([]), i32([]), cache)
    assert k.shape == v.shape == (0, 1, 64)
    k, v = A.dsv4_gqa_load(i32([0] * 1000), i32([7] * 1000), cache)
    assert (k == k[:1]).all() and (v == v[:1]).all()
    want = O.gqa_load([0], [7], c.oracle())
    assert torch.equal(k[:1].cpu(), twice_rounded(want[0], BF)) and torch.equal(v[:1].cpu(), twice_rounded(want[1], BF))


# ---------------------------------------------------------------- attention
def check_decode(A, case, lens, heads, *, window=0, sink=None, req=None, weights=False, decay=1.0, spread=1.0,
                 max_len=None, scale=None, want_flags=0):
    cache = case.handle(A)
    batch = len(lens)
    q = case.query(batch, heads, spread)
    max_len = case.width * case.page if max_len is None else max_len
    w = wo = None
    if weights:
        shape = (case.table.shape[0], case.hkv, case.width * case.page + 5)
        w, wo = torch.rand(shape, generator=case.gen), torch.full(shape, -7.0)
    real = 1 / math.sqrt(case.dim) if scale is None else scale
    ref, rlse, rw, err, sp = O.gqa_decode(
        q.double().numpy(), lens, case.oracle(), max_len=max_len, scale=real, window=window,
        sink=None if sink is None else sink.double().numpy(), req=req, weights=None if w is None else w.double().numpy(),
        weights_out=None if wo is None else wo.double().numpy(), decay=decay)
    d = lambda x: None if x is None else x.cuda()      # noqa: E731
    # short lists go other ways without weights, and where request rows are named
    ways = [(req, weights)]
    if weights:
        ways += [(req, False), (list(range(batch)) if req is None else req, True)]
    half = torch.finfo(case.qt).eps / 2
    ds = (case.dim + 8) * 2.0 ** -23 * sp["mag"]
    sums = (sp["rows"][:, None] / 16 + 64) * 2.0 ** -23
    rel = 2 * ds + 2.0 ** -20 + sums + (2.0 ** -11 if case.qt == BF else 2.0 ** -16)
    tol = rel[..., None] * sp["soft"] + 2.0 ** -36 * sp["tail"][..., None] + (half + 2.0 ** -22) * np.abs(ref) + \
        (2.0 ** -25 if case.qt == HF else 0.0)
    for named, kept in ways:
        wo_d = d(wo) if kept else None
        extra = {"weights": d(w), "weights_out": wo_d, "decay": decay} if kept else {}
        out, lse = A.dsv4_gqa_decode(d(q), i32(lens), cache, sink=d(sink), window=window, max_len=max_len, scale=real,
                                     req_pool_indices=None if named is None else i32(named), **extra)
        flags = A.dsv4_attn_get_device_error()
        assert flags == err == want_flags, (flags, err)
        o, g = out.double().cpu().numpy(), lse.double().cpu().numpy()
        assert np.isfinite(o).all()
        e = np.abs(o - ref)
        assert (e <= tol).all(), (float((e / np.maximum(tol, 1e-300)).max()), np.argwhere(e > tol)[:4].tolist())
        assert np.array_equal(np.isinf(g), np.isinf(rlse))
        fin = np.isfinite(rlse)
        assert (np.abs(g[fin] - rlse[fin]) <=
                (ds + 2.0 ** -20 + sums + np.abs(np.where(fin, rlse, 0)) * 2.0 ** -22)[fin]).all()
        if kept:
            gw = wo_d.double().cpu().numpy()
            tolw = sp["wslack"] * (2 * (case.dim + 8) * 2.0 ** -23 + 2.0 ** -19 + float(sums.max())) + np.abs(rw) * 2.0 ** -22
            assert (np.abs(gw - rw) <= tolw).all(), float((np.abs(gw - rw) / np.maximum(tolw, 1e-300)).max())


EDGE = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 97, 100]


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("q", [BF, HF])
def test_decode_types_dims_and_lengths(A, q, dim, page):
    c = Cache4(q=q, dim=dim, page=page, rows=len(EDGE), slots=100, seed=dim + page)
    c.poison(EDGE)
    check_decode(A, c, EDGE, 8, weights=True, sink=torch.randn(8, generator=c.gen))


@pytest.mark.parametrize("group", [1, 3, 8, 9, 16, 17, 64])
@pytest.mark.parametrize("q,dim", [(BF, 128), (HF, 64), (HF, 256), (BF, 256)])
def test_decode_groups(A, q, dim, group):
    c = Cache4(q=q, hkv=3, dim=dim, rows=4, slots=300, seed=group, scaled=group % 2 == 0)
    c.poison([300, 5, 0, 129])
    check_decode(A, c, [300, 5, 0, 129], 3 * group, weights=True, decay=0.75)


@pytest.mark.parametrize("window", [1, 15, 16, 40, 64, 1000])
@pytest.mark.parametrize("q,dim", [(BF, 64), (BF, 128), (HF, 256)])
def test_decode_windows(A, q, dim, window):
    lens = [0, 1, 16, 39, 40, 41, 80, 200]
    c = Cache4(q=q, dim=dim, rows=8, slots=200, seed=window)
    c.poison(lens)
    check_decode(A, c, lens, 4, window=window, weights=True, decay=0.5)


@pytest.mark.parametrize("q,dim,token_major,page", [(BF, 128, True, 32), (BF, 64, True, 16), (HF, 128, False, 128),
                                                    (HF, 64, False, 1024), (BF, 256, True, 256)])
def test_decode_layouts_and_splits(A, q, dim, token_major, page):
    # few segments, long: every request is cut over many CTAs
    c = Cache4(q=q, hkv=2, dim=dim, page=page, rows=3, slots=9000, seed=9, token_major=token_major)
    check_decode(A, c, [8999, 3, 5001], 10, weights=True, sink=torch.randn(10, generator=c.gen))


@pytest.mark.parametrize("group", [8, 16, 33])
@pytest.mark.parametrize("q,dim", [(BF, 64), (BF, 128), (HF, 128), (BF, 256)])
def test_decode_over_long_lists_with_missing_pages(A, q, dim, group):
    lens = [2500, 0, 7, 1203, 40, 1]
    c = Cache4(q=q, hkv=2, dim=dim, rows=6, slots=2500, seed=group + dim, token_major=group % 2 == 1)
    c.poison(lens)
    c.table[3, 30:33] = torch.tensor([-1, 10 ** 6, c.k.shape[0]])
    check_decode(A, c, lens, 2 * group, weights=True, sink=torch.randn(2 * group, generator=c.gen),
                 want_flags=O.ERR_GQA_PAGE)
    check_decode(A, c, [1203, 2500, 40, 0, 7, 1203], 2 * group, window=700, req=[0, 0, 3, 1, 2, 3], weights=True,
                 want_flags=O.ERR_GQA_PAGE)


@pytest.mark.parametrize("q", [BF, HF])
def test_decode_block_scales_of_all_sizes(A, q):
    for dim in (64, 128, 256):
        c = Cache4(q=q, dim=dim, rows=3, slots=200, seed=dim, wide_scales=True)
        c.kb[..., 1] = c.kb[..., 1] ^ 0x80           # a scale below zero counts as it stands
        c.vb[..., ::2, 2] = 0x7e                     # 448
        c.vb[..., 1::2, 3] = 0x01                    # the smallest
        c.poison([200, 77, 16])
        check_decode(A, c, [200, 77, 16], 8, weights=True)


@pytest.mark.parametrize("slots,lens", [(100, [100, 1, 17]), (9000, [9000, 4001, 40])])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_decode_of_blocks_without_a_value(A, dim, slots, lens):
    # a NaN block of an attended V row makes its 16 dims NaN and leaves the others as they are; of K, everything of the
    # KV head's queries
    c = Cache4(hkv=2, dim=dim, rows=3, slots=slots, seed=dim)
    q, n = c.query(3, 8).cuda(), i32(lens)
    plain = A.dsv4_gqa_decode(q, n, c.handle(A), max_len=slots)
    c.poison(lens)
    at = lambda b, s: (int(c.table[b, s // c.page]), s % c.page)      # noqa: E731
    for b, length in enumerate(lens):
        p, o = at(b, length // 2)
        c.vb[p, 1, o, dim // 16 - 1 - b] = 0x7f
    out, lse = A.dsv4_gqa_decode(q, n, c.handle(A), max_len=slots)
    assert torch.equal(lse, plain[1])
    for b in range(3):
        d = 16 * (dim // 16 - 1 - b)
        assert out[b, 4:, d: d + 16].isnan().all()
        out[b, 4:, d: d + 16] = plain[0][b, 4:, d: d + 16]
    assert torch.equal(out, plain[0])
    p, o = at(0, lens[0] - 1)
    c.kb[p, 0, o, 0] = 0xff
    out, lse = A.dsv4_gqa_decode(q, n, c.handle(A), max_len=slots)
    assert out[0, :4].isnan().all() and lse[0, :4].isnan().all() and torch.equal(lse[1:], plain[1][1:])
    assert A.dsv4_attn_get_device_error() == 0


def test_decode_small_and_large_queries(A):
    for spread in (1e-12, 1e25):
        c = Cache4(hkv=2, dim=64, rows=2, slots=60, seed=6)
        check_decode(A, c, [60, 33], 4, spread=spread, scale=0.125 / spread)


def test_decode_one_row_takes_all(A):
    c = Cache4(hkv=2, dim=128, rows=3, slots=500, seed=5)
    check_decode(A, c, [500, 499, 1], 8, spread=30.0, weights=True)


def test_decode_sinks_lengths_and_rows(A):
    c = Cache4(rows=6, slots=80, seed=8)
    for value in (-math.inf, -100.0, 0.0, 60.0, math.inf):
        check_decode(A, c, [80, 0, 7], 4, sink=torch.full((4,), value), weights=True)
    check_decode(A, c, [70, 0, 33], 4, req=[4, 99, 1], weights=True)
    check_decode(A, c, [70, 20, 33], 4, req=[4, -1, 1], weights=True, want_flags=O.ERR_REQ_ROW)
    check_decode(A, c, [81, -1, 33], 4, weights=True, want_flags=O.ERR_GQA_LENGTH)


def test_decode_offsets_beyond_32_bits(A):
    # codes and block scales far apart: pages of a pool larger than 4 GB, the request's at its end
    pages, page = 70000, 1024
    codes = torch.zeros(pages, 1, page, 64, dtype=torch.uint8, device="cuda")
    blocks = torch.zeros(pages, 1, page, 8, dtype=torch.uint8, device="cuda")
    gen = torch.Generator().manual_seed(1)
    few = Cache4(hkv=1, dim=128, page=page, rows=1, slots=2 * page, seed=1)
    table = torch.tensor([[pages - 1, pages - 3]], dtype=torch.int32)
    for i, p in enumerate(table[0].tolist()):
        codes[p], blocks[p] = few.k[int(few.table[0, i])].cuda(), few.kb[int(few.table[0, i])].cuda()
    cache = A.make_gqa_cache(codes, codes, table.cuda(), k_blocks=blocks.view(F8), v_blocks=blocks.view(F8),
                             k_scale=few.ks.cuda(), v_scale=few.ks.cuda())
    few.v, few.vb, few.vs = few.k, few.kb, few.ks
    q = torch.randn(1, 8, 128, generator=gen).to(BF).cuda()
    n = i32([2000])
    want = A.dsv4_gqa_decode(q, n, few.handle(A))
    got = A.dsv4_gqa_decode(q, n, cache)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    rows = torch.randn(3, 1, 128, generator=gen).to(BF).cuda()
    req, slots = i32([0, 0, 0]), i32([5, 1023, 1500])
    A.dsv4_gqa_store(rows, rows, req, slots, cache)
    got = A.dsv4_gqa_load(req, slots, cache)
    codes4, blocks4 = pack(rows.cpu(), few.ks)
    want = O.e2m1_values(codes4.numpy(), blocks4.numpy()) * few.ks.double().numpy()[:, None]
    assert torch.equal(got[0].cpu(), twice_rounded(want, BF)) and torch.equal(got[1], got[0])
    assert A.dsv4_attn_get_device_error() == 0


@pytest.mark.parametrize("lens", [[90000, 1, 88001], [60000, 0, 120001]])
@pytest.mark.parametrize("q,heads,dim", [(BF, 8, 128), (HF, 16, 64), (BF, 16, 256), (HF, 8, 128)])
def test_decode_of_long_lists(A, lens, q, heads, dim):
    # shares that are claimed, many pieces a segment; against the 64-bit form on the GPU
    page, rows, hkv = 256, 3, 4
    width = -(-max(lens) // page)
    gen = torch.Generator(device="cuda").manual_seed(dim + heads)
    pages = rows * width
    pool = {}
    for name in ("k", "v"):
        pool[name] = torch.randint(0, 256, (pages, hkv, page, dim // 2), generator=gen, device="cuda", dtype=torch.uint8)
        pool[name + "b"] = (0.2 + 0.3 * torch.rand(pages, hkv, page, dim // 16, generator=gen, device="cuda")).to(F8)
    table = torch.randperm(pages, generator=gen, device="cuda").view(rows, width).int()
    cache = A.make_gqa_cache(pool["k"], pool["v"], table, k_blocks=pool["kb"], v_blocks=pool["vb"])
    query = torch.randn(rows, hkv * heads, dim, generator=gen, device="cuda").to(q)
    outs = [A.dsv4_gqa_decode(query, i32(lens), cache) for _ in range(2)]
    assert A.dsv4_attn_get_device_error() == 0
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])      # bit for bit
    size = torch.tensor(O.E2M1, device="cuda")
    size = torch.cat([size, -size])
    half = torch.finfo(q).eps / 2
    for b, n in enumerate(lens):
        if n == 0:
            assert (outs[0][0][b] == 0).all()
            continue
        for h in range(hkv):
            kv = []
            for name in ("k", "v"):
                c = pool[name][table[b].long(), h].reshape(-1, dim // 2)[:n]
                x = size[torch.stack([c & 15, c >> 4], -1).long()].reshape(n, -1, 16)
                kv.append((x * pool[name + "b"][table[b].long(), h].reshape(-1, dim // 16)[:n].double()[..., None])
                          .flatten(1))
            mine = slice(h * heads, (h + 1) * heads)
            x = query[b, mine].double()
            s = x @ kv[0].T / math.sqrt(dim)
            p = torch.softmax(s, -1)
            ref = p @ kv[1]
            mag = (x.abs() @ kv[0].abs().T).amax(-1) / math.sqrt(dim)
            rel = 2 * (dim + 8) * 2.0 ** -23 * mag + 2.0 ** -20 + (n / 16 + 64) * 2.0 ** -23 + \
                (2.0 ** -11 if q == BF else 2.0 ** -16)
            tol = rel[:, None] * (p @ kv[1].abs()) + (half + 2.0 ** -22) * ref.abs() + 2.0 ** -25
            assert ((outs[0][0][b, mine].double() - ref).abs() <= tol).all()
            assert ((outs[0][1][b, mine].double() - torch.logsumexp(s, -1)).abs() <= rel + 2.0 ** -18).all()


# ---------------------------------------------------------------- eviction
@pytest.mark.parametrize("slack", [3, 60])
@pytest.mark.parametrize("dim,token_major", [(64, False), (128, True), (256, False)])
def test_evict_takes_block_scales_along(A, dim, token_major, slack):
    c = Cache4(hkv=3, dim=dim, rows=4, slots=150, seed=dim + slack, token_major=token_major)
    cache = c.handle(A)
    lens, keep = [150, 150 - slack, 149, 10], 150 - slack
    w = torch.rand(4, 3, 150, generator=c.gen)
    pos = torch.stack([torch.stack([torch.randperm(150, generator=c.gen) for _ in range(3)]) for _ in range(4)]).int()
    w_d, pos_d = w.cuda(), pos.cuda()
    n_out = A.dsv4_gqa_evict(i32(lens), cache, w_d, keep, positions=pos_d, seq_lens=i32([150] * 4), first=2, recent=5,
                             max_len=150)
    assert A.dsv4_attn_get_device_error() == 0
    for codes, blocks, dc, db in ((c.k, c.kb, c.k_d, c.kb_d), (c.v, c.vb, c.v_d, c.vb_d)):
        rows = torch.cat([codes, blocks], -1).numpy()              # whole rows, as the oracle copies them
        ref = O.gqa_evict(lens, {"k": rows, "v": rows, "table": c.table.numpy()}, w.numpy(), keep, max_len=150, first=2,
                          recent=5, positions=pos.numpy(), seq_lens=[150] * 4)
        assert np.array_equal(ref[1], torch.cat([dc, db], -1).cpu().numpy())
    assert n_out.tolist() == ref[0].tolist()
    for b, n in enumerate(ref[0].tolist()):
        assert np.array_equal(w_d[b, :, :n].cpu().numpy(), ref[3][b, :, :n])
        assert np.array_equal(pos_d[b, :, :n].cpu().numpy(), ref[4][b, :, :n])


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("q,dim", [(BF, 128), (HF, 64)])
def test_a_bounded_cache_over_many_steps(A, q, dim):
    # a prompt is written, read back, and then tokens are drafted one by one with the cache kept at its bound
    batch, hkv, heads, keep, page = 3, 2, 8, 40, 16
    c = Cache4(q=q, hkv=hkv, dim=dim, page=page, rows=batch, slots=64, seed=11)
    cache = c.handle(A)
    state = c.oracle()
    w, pos = torch.zeros(batch, hkv, 64), torch.zeros(batch, hkv, 64, dtype=torch.int32)
    w_d, pos_d = w.cuda(), pos.cuda()
    lens = [41, 30, 12]

    def put(x_k, x_v, req, slots, toks):
        A.dsv4_gqa_store(x_k.cuda(), x_v.cuda(), i32(req), i32(slots), cache, weights=w_d, positions=pos_d,
                         token_positions=i32(toks))
        for x, name, scale in ((x_k, "k", c.ks), (x_v, "v", c.vs)):
            vals = O.e2m1_values(*(y.numpy() for y in pack(x, scale)))
            for i, (r, s) in enumerate(zip(req, slots)):
                state[name][state["table"][r, s // page], :, s % page] = vals[i]
        for i, (r, s) in enumerate(zip(req, slots)):
            w[r, :, s], pos[r, :, s] = 0.0, toks[i]

    req = [b for b in range(batch) for _ in range(lens[b])]
    slots = [s for b in range(batch) for s in range(lens[b])]
    put(new_rows(len(req), hkv, dim, q, c.gen), new_rows(len(req), hkv, dim, q, c.gen), req, slots, slots)
    got = A.dsv4_gqa_load(i32(req), i32(slots), cache, dtype=q)
    want = O.gqa_load(req, slots, state)
    for x, y in zip(got, want):
        assert torch.equal(x.cpu(), twice_rounded(y, q))
    seen = list(lens)
    for step in range(8):
        x = new_rows(2 * batch, hkv, dim, q, c.gen)
        put(x[:batch], x[batch:], list(range(batch)), lens, seen)
        lens, seen = [n + 1 for n in lens], [n + 1 for n in seen]
        query = c.query(batch, heads, 0.5)
        before = w.double().numpy()
        ref, rlse, rw, err, sp = O.gqa_decode(query.double().numpy(), lens, state, max_len=64, scale=dim ** -0.5,
                                              weights=before, weights_out=before)
        out, lse = A.dsv4_gqa_decode(query.cuda(), i32(lens), cache, weights=w_d, max_len=64)
        ds = (dim + 8) * 2.0 ** -23 * sp["mag"]
        rel = 2 * ds + 2.0 ** -20 + 68 * 2.0 ** -23 + (2.0 ** -11 if q == BF else 2.0 ** -16)
        tol = rel[..., None] * sp["soft"] + (torch.finfo(q).eps / 2 + 2.0 ** -22) * np.abs(ref) + \
            2.0 ** -36 * sp["tail"][..., None] + 2.0 ** -25
        assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()
        tolw = sp["wslack"] * (2 * (dim + 8) * 2.0 ** -23 + 2.0 ** -19 + 68 * 2.0 ** -23) + np.abs(rw) * 2.0 ** -22
        assert (np.abs(w_d.double().cpu().numpy() - rw) <= tolw).all()
        w = w_d.cpu().clone()                    # the eviction goes by the weights as they are
        n_out = A.dsv4_gqa_evict(i32(lens), cache, w_d, keep, positions=pos_d, seq_lens=i32(seen), first=2, recent=4,
                                 max_len=64)
        ref = O.gqa_evict(lens, state, w.numpy(), keep, max_len=64, first=2, recent=4, positions=pos.numpy(),
                          seq_lens=seen)
        lens = n_out.tolist()
        assert lens == ref[0].tolist()
        state["k"], state["v"], w, pos = ref[1], ref[2], torch.from_numpy(ref[3]), torch.from_numpy(ref[4])
        for b, n in enumerate(lens):
            assert torch.equal(w_d[b, :, :n].cpu(), w[b, :, :n]) and torch.equal(pos_d[b, :, :n].cpu(), pos[b, :, :n])
        req = [b for b in range(batch) for _ in range(lens[b])]
        slots = [s for b in range(batch) for s in range(lens[b])]
        for x, y in zip(A.dsv4_gqa_load(i32(req), i32(slots), cache, dtype=q), O.gqa_load(req, slots, state)):
            assert torch.equal(x.cpu(), twice_rounded(y, q))
    assert A.dsv4_attn_get_device_error() == 0


def test_in_a_graph_and_on_streams(A):
    c = Cache4(hkv=2, dim=128, rows=3, slots=400, seed=12)
    cache = c.handle(A)
    lens, req, slots = i32([300, 5, 0]), i32([0, 1, 2]), i32([299, 4, 7])
    x = new_rows(6, 2, 128, BF, c.gen).cuda()
    q = c.query(3, 8).cuda()
    ws = torch.empty(A.dsv4_gqa_decode_workspace_size(cache, 3, 8, 400), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(3, 8, device="cuda")
    k, v = torch.empty(3, 2, 128, dtype=BF, device="cuda"), torch.empty(3, 2, 128, dtype=BF, device="cuda")

    def step(stream=None):
        A.dsv4_gqa_store(x[:3], x[3:], req, slots, cache, stream=stream)
        A.dsv4_gqa_load(req, slots, cache, k=k, v=v, stream=stream)
        A.dsv4_gqa_decode(q, lens, cache, max_len=400, out=out, lse=lse, workspace=ws, stream=stream)

    step()
    torch.cuda.synchronize()
    want = [y.clone() for y in (out, lse, k, v)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for y in (out, lse, k, v):
        y.fill_(3)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((out, lse, k, v), want))
    # other rows, lengths and values: read anew at every replay
    x.copy_(new_rows(6, 2, 128, BF, c.gen))
    lens.copy_(i32([123, 0, 8]))
    slots.copy_(i32([122, 17, 7]))
    graph.replay()
    torch.cuda.synchronize()
    got = [y.clone() for y in (out, lse, k, v)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((out, lse, k, v), got))
    side.wait_stream(torch.cuda.current_stream())
    other = A.dsv4_gqa_load(req, slots, cache, stream=side)
    side.synchronize()
    assert torch.equal(other[0], k) and torch.equal(other[1], v)
    assert A.dsv4_attn_get_device_error() == 0
