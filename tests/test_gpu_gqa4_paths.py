"""Attention over 4-bit rows on the kernel that each test names: a call that gives every segment a cluster is one launch,
one that shares out the list of tiles is two (with weights three), and every test asserts which of them its calls take.
With 64 and 128 dims and up to 8 query heads per KV head the list is that of the block-scaled tensor cores."""
import os
import subprocess
import sys

import pytest
import torch

from tests._gqa4 import BF, F8, HF, Cache4
from tests._launches import kernels
from tests.test_gpu_gqa4 import A, check_decode, i32  # noqa: F401

pytestmark = pytest.mark.gpu


def on_list(call):
    """call()'s result, after seeing that it takes the list."""
    got = call()
    assert kernels(call) == 2
    return got


def test_kernels_are_counted(A):  # noqa: F811
    c = Cache4(hkv=2, dim=128, rows=2, slots=9000, seed=1)
    cache, x, n = c.handle(A), c.query(2, 4).cuda(), i32([90, 17])
    w = torch.rand(2, 2, cache._slots, device="cuda")
    A.dsv4_gqa_decode(x, n, cache, max_len=90)
    assert kernels(lambda: A.dsv4_gqa_decode(x, n, cache, max_len=90)) == 1
    assert kernels(lambda: A.dsv4_gqa_decode(x, n, cache)) == 2
    assert kernels(lambda: A.dsv4_gqa_decode(x, n, cache, weights=w, weights_out=w)) == 3


def test_strided_queries_on_lists(A):  # noqa: F811
    for q, dim, slots in ((BF, 128, 9000), (HF, 64, 17000)):
        c = Cache4(q=q, hkv=3, dim=dim, rows=4, slots=slots, seed=5)
        cache = c.handle(A)
        wide = torch.randn(4, 40, dim, generator=c.gen).to(q).cuda()
        n, close = i32([slots, 3000, 0, slots - 1]), wide[:, 3:18].contiguous()
        want = on_list(lambda: A.dsv4_gqa_decode(close, n, cache))
        got = on_list(lambda: A.dsv4_gqa_decode(wide[:, 3:18], n, cache))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert A.dsv4_attn_get_device_error() == 0


def test_lists_on_streams_at_once(A):  # noqa: F811
    # calls that share the SMs and their tensor memory, each stream with a form of its own
    forms = []
    for q, dim, slots in ((BF, 128, 17000), (HF, 128, 17000), (BF, 64, 33000)):
        c = Cache4(q=q, hkv=4, dim=dim, page=64, rows=8, slots=slots, seed=6)
        cache, x, n = c.handle(A), c.query(8, 32).cuda(), i32([slots - 700 * i for i in range(8)])
        call = lambda x=x, n=n, cache=cache: A.dsv4_gqa_decode(x, n, cache)      # noqa: E731
        forms.append((torch.cuda.Stream(), call, on_list(call), []))
    torch.cuda.synchronize()
    for _ in range(8):
        for stream, call, _, got in forms:
            with torch.cuda.stream(stream):
                got.append(call())
    torch.cuda.synchronize()
    for _, _, want, got in forms:
        for out, lse in got:
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert A.dsv4_attn_get_device_error() == 0


def test_lists_beside_the_sparse_attention(A):  # noqa: F811
    # the draft's cache on one stream and the verified model's on another: both kernels use tensor memory
    from hybrid_sparse_mqa_gb300 import synth
    inp = synth.make_inputs(synth.Workload("beside", batch=8, heads=64, ratio=4, seq_lens=(900, 3000, 70, 5000, 2600, 4000, 1, 128),
                                           seed=5), device="cuda")
    c = Cache4(hkv=4, dim=128, page=64, rows=8, slots=17000, seed=6)
    cache, x, n = c.handle(A), c.query(8, 32).cuda(), i32([17000 - 900 * i for i in range(8)])
    calls = (lambda: A.dsv4_gqa_decode(x, n, cache), lambda: A.run_inputs(inp))
    want = (on_list(calls[0]), calls[1]())
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in calls], ([], [])
    for _ in range(20):
        for stream, call, mine in zip(streams, calls, got):
            with torch.cuda.stream(stream):
                mine.append(call())
    torch.cuda.synchronize()
    for first, mine in zip(want, got):
        for out, lse in mine:
            assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    assert A.dsv4_attn_get_device_error() == 0


@pytest.mark.parametrize("q", [BF, HF])
@pytest.mark.parametrize("dim,slots", [(64, 17000), (128, 9000)])
def test_blocks_without_a_value_on_lists(A, q, dim, slots):  # noqa: F811
    # NaN blocks behind the last rows change nothing; one of an attended V row makes its 16 dims NaN and leaves the others
    # as they are; of K, everything of the KV head's queries
    lens = [slots, slots // 2 + 1, 40]
    c = Cache4(q=q, hkv=2, dim=dim, page=64, rows=3, slots=slots, seed=dim)
    x, n = c.query(3, 8).cuda(), i32(lens)
    decode = lambda cache: on_list(lambda: A.dsv4_gqa_decode(x, n, cache, max_len=slots))      # noqa: E731
    plain = decode(c.handle(A))
    c.poison(lens)
    place = lambda b, s: (int(c.table[b, s // c.page]), s % c.page)      # noqa: E731
    for b, length in enumerate(lens):
        p, o = place(b, length // 2)
        c.vb[p, 1, o, b] = 0xff if b == 1 else 0x7f
    out, lse = decode(c.handle(A))
    assert torch.equal(lse, plain[1])
    for b in range(3):
        nan = slice(16 * b, 16 * b + 16)
        assert out[b, 4:, nan].isnan().all()
        out[b, 4:, nan] = plain[0][b, 4:, nan]
    assert torch.equal(out, plain[0])
    p, o = place(0, slots - 1)
    c.kb[p, 0, o, dim // 16 - 1] = 0xff
    out, lse = decode(c.handle(A))
    assert out[0, :4].isnan().all() and lse[0, :4].isnan().all() and torch.equal(lse[0, 4:], plain[1][0, 4:])
    assert torch.equal(lse[1:], plain[1][1:])
    assert A.dsv4_attn_get_device_error() == 0


@pytest.mark.parametrize("q", [BF, HF])
def test_signs_and_sizes_of_block_scales_on_lists(A, q):  # noqa: F811
    for dim, slots in ((64, 17000), (128, 9000)):
        c = Cache4(q=q, dim=dim, page=128, rows=2, slots=slots, seed=dim, wide_scales=True)
        c.kb[..., 1] = c.kb[..., 1] ^ 0x80
        c.vb[..., ::3, 2] = c.vb[..., ::3, 2] ^ 0x80
        c.vb[..., ::2, 3] = 0x7e                     # 448
        c.vb[..., 1::2, 0] = 0x01                    # the smallest
        x, n, cache = c.query(2, 8).cuda(), i32([slots, 4007]), c.handle(A)
        on_list(lambda: A.dsv4_gqa_decode(x, n, cache, max_len=slots))
        check_decode(A, c, [slots, 4007], 8, max_len=slots)


@pytest.mark.parametrize("dim", [64, 128])
def test_offsets_beyond_32_bits_on_lists(A, dim):  # noqa: F811
    # codes and, behind them in the same page, block scales of a pool larger than 4 GB; the request's pages at its end
    page, size = 1024, dim // 2 * 1024 + dim // 16 * 1024
    width = 9 if dim == 128 else 17
    pages = (1 << 32) // size + 2 * width + 8
    few = Cache4(hkv=1, dim=dim, page=page, rows=1, slots=width * page, seed=1)
    pool = torch.zeros(pages, size, dtype=torch.uint8, device="cuda")
    codes = pool[:, : dim // 2 * page].view(pages, 1, page, dim // 2)
    blocks = pool[:, dim // 2 * page:].view(pages, 1, page, dim // 16)
    table = torch.tensor([[pages - 1 - 2 * i for i in range(width)]], dtype=torch.int32)
    for i, p in enumerate(table[0].tolist()):
        codes[p], blocks[p] = few.k[int(few.table[0, i])].cuda(), few.kb[int(few.table[0, i])].cuda()
    assert int(table.min()) * size > 1 << 32
    cache = A.make_gqa_cache(codes, codes, table.cuda(), k_blocks=blocks.view(F8), v_blocks=blocks.view(F8),
                             k_scale=few.ks.cuda(), v_scale=few.ks.cuda())
    few.v, few.vb, few.vs = few.k, few.kb, few.ks
    x, n, small = few.query(1, 8).cuda(), i32([width * page - 100]), few.handle(A)
    want = on_list(lambda: A.dsv4_gqa_decode(x, n, small))
    got = on_list(lambda: A.dsv4_gqa_decode(x, n, cache))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert A.dsv4_attn_get_device_error() == 0


@pytest.mark.parametrize("size", [2.0 ** -124, 2.0 ** -118, 2.0 ** -112, 2.0 ** -101, 2.0 ** 120])
@pytest.mark.parametrize("dim,slots", [(64, 17000), (128, 9000)])
def test_smallest_and_largest_queries_on_lists(A, dim, slots, size):  # noqa: F811
    # heads of 2^-124 reach bf16's smallest values; the score's factor makes up for their size
    c = Cache4(hkv=2, dim=dim, page=128, rows=2, slots=slots, seed=9, scaled=False)
    lens, scale = [slots, 4001], 0.125 / size
    x, n, cache = c.query(2, 8).cuda(), i32(lens), c.handle(A)
    on_list(lambda: A.dsv4_gqa_decode(x, n, cache, max_len=slots))
    check_decode(A, c, lens, 8, spread=size, scale=scale, max_len=slots)
    check_decode(A, c, [60, 33], 8, spread=size, scale=scale, max_len=60)          # and on a cluster


_CAPTURE = """
import torch
from hybrid_sparse_mqa_gb300 import attn as A
from tests._launches import kernels
BF, HF, F8 = torch.bfloat16, torch.float16, torch.float8_e4m3fn
gen = torch.Generator(device="cuda").manual_seed(1)
def rand(*shape):
    return torch.randn(*shape, generator=gen, device="cuda").to({q})
def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")
pages, hkv, page, dim = 140, 2, 256, {dim}
k, v = (torch.randint(0, 256, (pages, hkv, page, dim // 2), generator=gen, device="cuda", dtype=torch.uint8) for _ in range(2))
kb, vb = ((0.2 + 0.3 * torch.rand(pages, hkv, page, dim // 16, generator=gen, device="cuda")).to(F8) for _ in range(2))
cache = A.make_gqa_cache(k, v, torch.arange(pages, device="cuda", dtype=torch.int32).view(2, 70), k_blocks=kb, v_blocks=vb)
pools = [x.view(torch.uint8) for x in (k, v, kb, vb)]
bits = lambda: [x.clone() for x in pools]
q, wide, many = rand(2, 4, dim), rand(2, 32, dim), rand(160, 4, dim)
lens, rows = ints(17500, 17000), ints(1, 0)
w = torch.rand(2, hkv, 70 * page, generator=gen, device="cuda")
new, slots = rand(2, 2 * hkv, dim), ints(17500, 17000)
crowd, short = ints(*[i % 2 for i in range(160)]), ints(*[1 + i % 100 for i in range(160)])
w_out = lambda: torch.zeros_like(w)
order = ints(0, 1)
def store():
    A.dsv4_gqa_store(new[:, :hkv], new[:, hkv:], order, slots, cache)
    return bits()
calls = dict(
    long=lambda: A.dsv4_gqa_decode(q, lens, cache),
    kept=lambda: A.dsv4_gqa_decode(q, lens, cache, weights=w, weights_out=w_out(), req_pool_indices=rows),
    wide=lambda: A.dsv4_gqa_decode(wide, lens, cache),
    wide_short=lambda: A.dsv4_gqa_decode(wide, short[:2], cache, max_len=100),
    many=lambda: A.dsv4_gqa_decode(many, short, cache, max_len=100, req_pool_indices=crowd),
    evict=lambda: [A.dsv4_gqa_evict(lens, cache, w, 1000, weights_out=w_out()), *bits()],
    load=lambda: A.dsv4_gqa_load(order, slots, cache), load_f16=lambda: A.dsv4_gqa_load(rows, slots, cache, dtype=HF),
    store=store,
)
# one short call of each function, of the forms with the fewest launches, is what was made before the captures
A.dsv4_gqa_decode(q, ints(3, 2), cache, max_len=100)
A.dsv4_gqa_store(new[:, :hkv], new[:, hkv:], ints(0, 1), slots, cache)
A.dsv4_gqa_load(ints(0, 1), slots, cache)
A.dsv4_gqa_evict(ints(3, 2), cache, w, 100, max_len=100)
A.dsv4_attn_get_device_error()
before = bits()
def restore():
    for x, y in zip(pools, before):
        x.copy_(y)
torch.cuda.synchronize()
graphs = dict()
for name, call in calls.items():
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    graphs[name] = (graph, got)
for name, call in calls.items():
    for again in range(2):
        restore()
        graphs[name][0].replay()
        torch.cuda.synchronize()
        first = [x.clone() for x in graphs[name][1] if x is not None]
        restore()
        assert all(torch.equal(x, y) for x, y in zip(first, [x for x in call() if x is not None])), name
assert A.dsv4_attn_get_device_error() == 0
assert kernels(calls["long"]) == 2 and kernels(calls["wide"]) == 2 and kernels(calls["many"]) == 1
print("captured")
"""


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("q", ["BF", "HF"])
def test_captures_after_one_call_of_each_function(A, q, dim):  # noqa: F811
    # in a process of its own: what an earlier test has launched is loaded already
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", _CAPTURE.format(q=q, dim=dim)], cwd=root, capture_output=True, text=True,
                         timeout=300)
    assert run.returncode == 0 and "captured" in run.stdout, run.stderr[-2000:]
