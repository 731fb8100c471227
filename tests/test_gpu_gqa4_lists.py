"""Attention over long lists of 4-bit rows (64 and 128 dims, up to 8 query heads per KV head), where tiles of 128 slots go
to the block-scaled tensor cores: borders of tiles and shares, references that move, sums that leave the accumulator,
queries of every kind, and captures.  The bound on errors is that of test_gpu_gqa4.check_decode.  Calls with weights that
name their request rows always take the list; the others do from some thousand rows on."""
import math

import pytest
import torch

from oracle import gqa_oracle as O
from tests._gqa4 import BF, F8, HF, Cache4
from tests.test_gpu_gqa4 import A, check_decode, i32  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page,token_major", [(16, False), (64, True), (1024, False)])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q", [BF, HF])
def test_borders_of_tiles(A, q, dim, page, token_major):  # noqa: F811
    lens = [127, 128, 129, 0, 255, 256, 257, 1, 383, 16]
    c = Cache4(q=q, hkv=2, dim=dim, page=page, rows=len(lens), slots=400, seed=page + dim, token_major=token_major)
    req = [7, 0, 3, 9, 1, 2, 8, 4, 5, 6]
    c.poison(lens, req)
    check_decode(A, c, lens, 10, weights=True, sink=torch.randn(10, generator=c.gen), req=req)


@pytest.mark.parametrize("window", [1, 100, 128, 129, 300])
@pytest.mark.parametrize("q,dim", [(BF, 128), (HF, 64), (HF, 128)])
def test_windows(A, q, dim, window):  # noqa: F811
    lens = [500, 128, 129, 300, 2, 428]
    c = Cache4(q=q, dim=dim, rows=6, slots=500, seed=window)
    req = [5, 4, 3, 2, 1, 0]
    c.poison(lens, req)
    check_decode(A, c, lens, 6, window=window, weights=True, decay=0.5, req=req)


@pytest.mark.parametrize("q,dim,group", [(BF, 128, 1), (HF, 128, 8), (BF, 64, 7)])
def test_more_segments_than_ctas(A, q, dim, group):  # noqa: F811
    # several segments to a share, many of them of one tile
    gen = torch.Generator().manual_seed(group)
    lens = [int(x) for x in torch.randint(0, 300, (70,), generator=gen)]
    c = Cache4(q=q, hkv=7, dim=dim, page=32, rows=70, slots=300, seed=dim + group)
    check_decode(A, c, lens, 7 * group, weights=True, req=[int(x) for x in torch.randperm(70, generator=gen)])


@pytest.mark.parametrize("q,dim,group", [(BF, 128, 8), (HF, 64, 1), (HF, 128, 3), (BF, 64, 8)])
def test_more_short_segments_than_ctas(A, q, dim, group):  # noqa: F811
    # a CTA each, in several waves, with weights and without
    gen = torch.Generator().manual_seed(group)
    lens = [int(x) for x in torch.randint(0, 700, (60,), generator=gen)]
    c = Cache4(q=q, hkv=6, dim=dim, page=16, rows=60, slots=700, seed=dim + group, token_major=True)
    c.poison(lens)
    check_decode(A, c, lens, 6 * group, weights=True, window=500, sink=torch.randn(6 * group, generator=c.gen))


@pytest.mark.parametrize("q,dim", [(BF, 128), (HF, 64)])
def test_references_that_move(A, q, dim):  # noqa: F811
    # scores that grow along the slots (most tiles move the reference, back and forth over tiles of both groups), then
    # shrink again; and one that jumps within a tile's last slots
    n = 6000
    c = Cache4(q=q, hkv=1, dim=dim, page=64, rows=2, slots=n, seed=dim)
    for r in range(2):
        for s in range(n):
            up = s if r == 0 else n - s
            code = 0x10 + up * 0x40 // n
            c.kb[int(c.table[r, s // 64]), :, s % 64] = code
    check_decode(A, c, [n, n], 8, weights=True, req=[1, 0], spread=2.0)


@pytest.mark.parametrize("q,dim", [(BF, 128), (HF, 128), (BF, 64)])
def test_one_request_over_all_ctas(A, q, dim):  # noqa: F811
    # 30000 rows of one KV head: a share for every tile; with weights, and missing pages among them
    c = Cache4(q=q, hkv=1, dim=dim, page=128, rows=1, slots=30000, seed=dim)
    c.table[0, 100] = -1
    c.table[0, 150:153] = 10 ** 7
    check_decode(A, c, [29999], 8, weights=True, want_flags=O.ERR_GQA_PAGE)


def test_sums_over_many_tiles(A):  # noqa: F811
    # enough rows that a share holds dozens of tiles; all values alike, so that a truncating sum would show its drift
    pages, page, hkv, dim, batch = 1200, 1024, 4, 128, 4
    codes = torch.full((pages, hkv, page, dim // 2), 0x55, dtype=torch.uint8, device="cuda")        # 3.0
    blocks = torch.full((pages, hkv, page, dim // 16), 0x39, dtype=torch.uint8, device="cuda")      # 1.125
    table = torch.arange(pages, dtype=torch.int32, device="cuda").view(batch, pages // batch)
    cache = A.make_gqa_cache(codes, codes, table, k_blocks=blocks.view(F8), v_blocks=blocks.view(F8))
    n = pages // batch * page
    for q in (BF, HF):
        query = torch.zeros(batch, 8 * hkv, dim, dtype=q, device="cuda")
        out, lse = A.dsv4_gqa_decode(query, i32([n, n - 5, n - 1000, 100000]), cache)
        # every weight 1: sums of the softmax exact to n < 2^24; n / 16 steps of the accumulator in pieces of 128
        want = 3.375
        assert float((out.double() - want).abs().max()) <= want * (2.0 ** -16 + torch.finfo(q).eps / 2)
        assert float((lse.double() - torch.tensor([n, n - 5, n - 1000, 100000.0]).double().log().cuda()[:, None]).abs().max()) < 1e-5
    assert A.dsv4_attn_get_device_error() == 0


@pytest.mark.parametrize("q", [BF, HF])
def test_queries_of_all_sizes(A, q):  # noqa: F811
    # dims of a head from its largest value down to nothing, signs, zeros, heads of zeros, subnormal heads
    c = Cache4(q=q, hkv=2, dim=128, rows=2, slots=9000, seed=3)
    size = torch.exp2(-torch.arange(128).float() / 4)
    plain = c.query
    def query(batch, heads, spread):                              # noqa: E306
        x = plain(batch, heads, spread).float() * size
        x[:, 1] = 0.0
        x[:, 2] *= 2.0 ** -20 if q == HF else 1e-30
        x[:, 3, ::2] = 0.0
        return x.to(q)
    c.query = query
    check_decode(A, c, [9000, 8111], 8, weights=True, sink=torch.zeros(8))


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("q", [BF, HF])
def test_queries_without_a_value(A, q, bad):  # noqa: F811
    c = Cache4(q=q, hkv=2, dim=128, rows=3, slots=9000, seed=4)
    x, n = c.query(3, 8).cuda(), i32([9000, 0, 4001])
    cache = c.handle(A)
    want = A.dsv4_gqa_decode(x, n, cache)
    x[:, 5, 77] = bad
    out, lse = A.dsv4_gqa_decode(x, n, cache)
    assert out[[0, 2], 5].isnan().all() and lse[[0, 2], 5].isnan().all() and (out[1] == 0).all() and lse[1, 5] == -math.inf
    others = [0, 1, 2, 3, 4, 6, 7]
    assert torch.equal(out[:, others], want[0][:, others]) and torch.equal(lse[:, others], want[1][:, others])
    assert A.dsv4_attn_get_device_error() == 0


def test_strided_queries_and_outputs_of_other_rows(A):  # noqa: F811
    c = Cache4(q=BF, hkv=3, dim=128, rows=4, slots=7000, seed=5)
    cache = c.handle(A)
    wide = torch.randn(4, 40, 128, generator=c.gen).to(BF).cuda()
    n = i32([7000, 3000, 0, 6999])
    want = A.dsv4_gqa_decode(wide[:, 3:18].contiguous(), n, cache)
    got = A.dsv4_gqa_decode(wide[:, 3:18], n, cache)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_streams_at_once(A):  # noqa: F811
    # calls that share the SMs and their tensor memory
    c = Cache4(q=BF, hkv=4, dim=128, rows=8, slots=12000, seed=6)
    cache = c.handle(A)
    x, n = c.query(8, 32).cuda(), i32([12000 - 700 * i for i in range(8)])
    want = A.dsv4_gqa_decode(x, n, cache)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for _ in range(6):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(A.dsv4_gqa_decode(x, n, cache))
    torch.cuda.synchronize()
    for out, lse in got:
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert A.dsv4_attn_get_device_error() == 0


def test_a_list_captured_after_a_short_call(A):  # noqa: F811
    # the first call of a format, type and width loads every kernel that later ones can take
    for q, dim in ((BF, 64), (HF, 128)):
        c = Cache4(q=q, hkv=2, dim=dim, rows=2, slots=9000, seed=7)
        cache = c.handle(A)
        x, n = c.query(2, 4).cuda(), i32([100, 50])
        A.dsv4_gqa_decode(x, n, cache, max_len=100)
        w = torch.rand(2, 2, cache._slots, device="cuda")
        keep = w.clone()
        size = A.dsv4_gqa_decode_workspace_size(cache, 2, 4, 9000, True)
        ws, out, lse = torch.empty(size, dtype=torch.uint8, device="cuda"), torch.empty_like(x), torch.empty(2, 4, device="cuda")
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            A.dsv4_gqa_decode(x, n, cache, max_len=9000, weights=w, out=out, lse=lse, workspace=ws)
        n.copy_(i32([9000, 777]))
        g.replay()
        torch.cuda.synchronize()
        first = w.clone()
        plain = A.dsv4_gqa_decode(x, n, cache, max_len=9000, weights=keep)
        assert torch.equal(out, plain[0]) and torch.equal(lse, plain[1]) and torch.equal(first, keep)
    assert A.dsv4_attn_get_device_error() == 0
