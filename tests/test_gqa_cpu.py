"""The grouped-query cache operators without a GPU: what the entry points
refuse before any launch (the C ABI and the Python binding), workspace sizes,
and the oracle against closed forms and small brute force."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import gqa_oracle as O
from tests._streams import Streams


@pytest.fixture(scope="module")
def A():
    from hybrid_sparse_mqa_gb300 import build
    build.build()
    from hybrid_sparse_mqa_gb300 import attn
    attn.lib()
    return attn


_ALIVE = []


def _cache(A, **kw):
    c = A.GqaCache()
    _ALIVE.append(c)          # the tests pass its address
    fields = dict(k=4096, v=8192, num_pages=8, page_stride=65536, head_stride=8192, row_stride=256, page_table=4096,
                  page_table_rows=4, page_table_stride=8, page_table_width=8, num_kv_heads=4, head_dim=128,
                  page_size=32, format=0)
    fields.update(kw)
    for name, x in fields.items():
        setattr(c, name, x)
    return c


BAD_CACHES = [
    (dict(k=None), -1), (dict(v=None), -1), (dict(page_table=None), -1), (dict(k=4104), -1), (dict(v=8), -1),
    (dict(num_pages=0), -1), (dict(page_table_rows=0), -1), (dict(page_table_width=0), -1),
    (dict(page_table_width=9), -1), (dict(num_kv_heads=0), -1), (dict(num_kv_heads=257), -2),
    (dict(page_stride=8), -1), (dict(head_stride=24), -1), (dict(row_stride=-256), -1),
    (dict(head_dim=96), -2), (dict(head_dim=512), -2), (dict(page_size=8), -2), (dict(page_size=48), -2),
    (dict(page_size=2048), -2), (dict(format=3), -2), (dict(format=-1), -2),
]


@pytest.mark.parametrize("fields,want", BAD_CACHES)
def test_bad_caches_are_refused(A, fields, want):
    lib, c = A.lib(), ctypes.addressof(_cache(A, **fields))
    assert _decode(A, c) == want and _store(A, c) == want and _evict(A, c) == want
    assert lib.dsv4_gqa_decode_workspace_size(c, 4, 16, 100, 0) == 0
    assert lib.dsv4_gqa_evict_workspace_size(c, 4, 100, 10) == 0


def _decode(A, c, q=4096, q_stride=2048, type=0, batch=4, heads=16, lens=4096, req=None, window=0, max_len=100,
            sink=None, weights=None, weights_out=None, width=0, out=4096, lse=None, ws=4096, have=1 << 40):
    return A.lib().dsv4_gqa_decode(q, q_stride, type, batch, heads, lens, req, c, window, max_len, sink, 0.1, weights,
                                   weights_out, width, 1.0, out, lse, ws, have, None)


def _store(A, c, k=4096, kt=512, kh=128, v=4096, vt=512, vh=128, type=0, n=3, req=4096, slots=4096, weights=None,
           positions=None, width=0, tokens=None):
    return A.lib().dsv4_gqa_store(k, kt, kh, v, vt, vh, type, n, req, slots, c, weights, positions, width, tokens,
                                  None)


def _evict(A, c, batch=4, lens=4096, seen=None, req=None, max_len=100, keep=10, first=0, recent=0, weights=4096,
           weights_out=4096, positions=None, positions_out=None, width=128, lens_out=4096, ws=4096, have=1 << 40):
    return A.lib().dsv4_gqa_evict(batch, lens, seen, req, c, max_len, keep, first, recent, weights, weights_out,
                                  positions, positions_out, width, lens_out, ws, have, None)


DECODE_REFUSALS = [
    (dict(q=None), -1), (dict(q=4104), -1), (dict(q_stride=2052), -1), (dict(type=2), -2), (dict(type=1), -2),
    (dict(batch=0), -1), (dict(heads=0), -1), (dict(heads=18), -1), (dict(heads=4 * 65), -2), (dict(lens=None), -1),
    (dict(window=-1), -1), (dict(max_len=0), -1), (dict(max_len=257), -1), (dict(out=None), -1), (dict(out=4100), -1),
    (dict(weights=4096), -1), (dict(weights_out=4096, width=128), -1),
    (dict(weights=4096, weights_out=4096, width=99), -1),
    (dict(weights=4096, weights_out=4096, width=128, batch=16384), -2),
    (dict(ws=None), -3), (dict(have=1000), -3), (dict(ws=4104), -1),
]


@pytest.mark.parametrize("args,want", DECODE_REFUSALS)
def test_decode_refusals(A, args, want):
    assert _decode(A, ctypes.addressof(_cache(A)), **args) == want


STORE_REFUSALS = [
    (dict(k=None), -1), (dict(v=None), -1), (dict(k=4104), -1), (dict(v=4100), -1), (dict(n=-1), -1),
    (dict(kt=516), -1), (dict(vh=4), -1), (dict(req=None), -1), (dict(slots=None), -1), (dict(type=2), -2),
    (dict(type=1), -2), (dict(positions=4096, width=64), -1), (dict(weights=4096), -1), (dict(n=0, k=None), 0),
]


@pytest.mark.parametrize("args,want", STORE_REFUSALS)
def test_store_refusals(A, args, want):
    assert _store(A, ctypes.addressof(_cache(A)), **args) == want


EVICT_REFUSALS = [
    (dict(batch=0), -1), (dict(batch=16384), -2), (dict(lens=None), -1), (dict(lens_out=None), -1),
    (dict(max_len=0), -1), (dict(max_len=257, width=300), -1), (dict(keep=0), -1), (dict(first=-1), -1),
    (dict(recent=-1), -1), (dict(first=6, recent=5), -1), (dict(first=2**31 - 1, recent=2**31 - 1), -1),
    (dict(weights=None), -1), (dict(weights_out=None), -1), (dict(positions=4096), -1), (dict(positions_out=4096), -1),
    (dict(width=99), -1), (dict(ws=None), -3), (dict(have=16), -3), (dict(ws=4104), -1),
]


OVERLAPS = [      # of arrays of 4 x 4 x 128 entries and of 4 lengths
    (dict(weights_out=4096 + 4), -1), (dict(weights=1 << 20, weights_out=(1 << 20) - 4 * 2047), -1), (dict(weights_out=4096 + 4 * 2048, ws=None), -3),
    (dict(positions=1 << 20, positions_out=(1 << 20) + 8), -1), (dict(lens_out=4096 + 4), -1), (dict(lens_out=4096 - 12), -1),
    (dict(lens_out=4096 + 16, ws=None), -3), (dict(seen=4096 * 2, lens_out=4096 * 2 + 4), -1),
    (dict(seen=4096 * 2, lens_out=4096 * 2, ws=None), -3), (dict(req=4096 * 2, lens_out=4096 * 2), -1),
    (dict(req=4096 * 2, lens_out=4096 * 2 + 16, ws=None), -3),
]


@pytest.mark.parametrize("args,want", OVERLAPS)
def test_evict_refuses_arrays_that_overlap(A, args, want):
    assert _evict(A, ctypes.addressof(_cache(A)), **args) == want


def test_decode_refuses_weights_that_overlap(A):
    c = ctypes.addressof(_cache(A))
    for shift, want in ((4, -1), (-4 * 2047, -1), (0, -3), (4 * 2048, -3)):
        assert _decode(A, c, weights=1 << 20, weights_out=(1 << 20) + shift, width=128, ws=None) == want


@pytest.mark.parametrize("args,want", EVICT_REFUSALS)
def test_evict_refusals(A, args, want):
    assert _evict(A, ctypes.addressof(_cache(A)), **args) == want


def test_workspace_sizes_grow_with_what_they_hold(A):
    lib, c = A.lib(), ctypes.addressof(_cache(A))
    plain = lib.dsv4_gqa_decode_workspace_size(c, 4, 16, 100, 0)
    # the pieces of cut requests: bounded however long the caches are
    most = lib.dsv4_gqa_decode_workspace_size(c, 4096, 16, 256, 0)
    assert 0 < plain <= most == lib.dsv4_gqa_decode_workspace_size(c, 8192, 16, 256, 0) < 64 << 20
    # with weights: 8 fp32 scores per slot of a tile, per request and KV head
    assert lib.dsv4_gqa_decode_workspace_size(c, 4, 16, 100, 1) >= plain + 4 * 4 * 112 * 8 * 4
    assert lib.dsv4_gqa_evict_workspace_size(c, 4, 100, 10) >= 4 * 4 * (4 + 2 * 10 * 4)


def test_without_a_device_the_calls_report_cuda_errors(A):
    if torch.cuda.is_available():
        pytest.skip("a device is present")
    c = ctypes.addressof(_cache(A))
    assert _decode(A, c) == -4 and _store(A, c) == -4 and _evict(A, c) == -4


def test_binding_refuses_what_is_not_a_cache(A):
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    table = torch.zeros(2, 2, dtype=torch.int32)
    bad = [
        (k[0], k[0], table), (k.float(), k.float(), table), (k, k[:2], table), (k, k.half(), table),
        (k, k.transpose(1, 2).contiguous().transpose(1, 2), table), (k.transpose(2, 3), k.transpose(2, 3), table),
        (k, k, table.long()), (k, k, table[0]), (k, k, table.t().contiguous().t()),
    ]
    for args in bad:
        with pytest.raises(A.Dsv4Error):
            A.make_gqa_cache(*args)
    with pytest.raises(A.Dsv4Error):
        A.make_gqa_cache(k, k, table, k_scale=torch.ones(2))
    k8 = k.to(torch.float8_e4m3fn)
    for scale in (torch.ones(3), torch.ones(2, dtype=torch.float64), torch.ones(4)[::2]):
        with pytest.raises(A.Dsv4Error):
            A.make_gqa_cache(k8, k8, table, v_scale=scale)
    c = A.make_gqa_cache(k8, k8, table, k_scale=torch.ones(2), v_scale=torch.ones(2))
    assert (c.num_kv_heads, c.page_size, c.head_dim, c.format, c.row_stride) == (2, 16, 64, 2, 64)


def test_binding_refuses_mismatched_arguments(A):
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    c = A.make_gqa_cache(k, k, torch.zeros(3, 2, dtype=torch.int32))
    q = torch.zeros(3, 8, 64, dtype=torch.bfloat16)
    lens = torch.zeros(3, dtype=torch.int32)
    w = torch.zeros(3, 2, 32)
    ints = torch.zeros(3, 2, 32, dtype=torch.int32)
    calls = [
        lambda: A.dsv4_gqa_decode(q.half(), lens, c), lambda: A.dsv4_gqa_decode(q[0], lens, c),
        lambda: A.dsv4_gqa_decode(q[:, :, :32], lens, c), lambda: A.dsv4_gqa_decode(q[:, ::2], lens, c),
        lambda: A.dsv4_gqa_decode(q, lens[:2], c), lambda: A.dsv4_gqa_decode(q, lens.long(), c),
        lambda: A.dsv4_gqa_decode(q, lens, c, sink=torch.zeros(4)),
        lambda: A.dsv4_gqa_decode(q, lens, c, weights=w[:2]), lambda: A.dsv4_gqa_decode(q, lens, c, weights=w.half()),
        lambda: A.dsv4_gqa_decode(q, lens, c, weights=w[:, :, :16]),
        lambda: A.dsv4_gqa_decode(q, lens, c, weights_out=w),
        lambda: A.dsv4_gqa_decode(q, lens, c, weights=w, weights_out=torch.zeros(3, 2, 48)),
        lambda: A.dsv4_gqa_decode(q, lens, c, weights=torch.zeros(3, 2, 16)),
        lambda: A.dsv4_gqa_decode(q, lens, c, out=q.half()), lambda: A.dsv4_gqa_decode(q, lens, c, lse=torch.zeros(3)),
        lambda: A.dsv4_gqa_decode(torch.zeros(4, 8, 64, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32), c),
        lambda: A.dsv4_gqa_decode(q, lens, c),                       # the pools are not on a CUDA device
        lambda: A.dsv4_gqa_store(q[:, :2], q[:, :2], lens[:2], lens, c),
        lambda: A.dsv4_gqa_store(q[:, :2], q[:, :2].half(), lens, lens, c),
        lambda: A.dsv4_gqa_store(q, q, lens, lens, c), lambda: A.dsv4_gqa_store(q[0], q[0], lens, lens, c),
        lambda: A.dsv4_gqa_store(q[:, :2], q[0], lens, lens, c),
        lambda: A.dsv4_gqa_store(q[:, :2].float(), q[:, :2].float(), lens, lens, c),
        lambda: A.dsv4_gqa_store(q[:, :2], q[:, :2], lens, lens, c, positions=ints),
        lambda: A.dsv4_gqa_store(q[:, :2], q[:, :2], lens, lens, c, token_positions=lens),
        lambda: A.dsv4_gqa_store(q[:, :2], q[:, :2], lens, lens, c, weights=w[:, :1]),
        lambda: A.dsv4_gqa_store(q[:, :2], q[:, :2], lens, lens, c),  # not on a CUDA device
        lambda: A.dsv4_gqa_evict(lens, c, w[0], 4), lambda: A.dsv4_gqa_evict(lens, c, w, 4, positions=w),
        lambda: A.dsv4_gqa_evict(lens, c, w, 4, positions_out=ints),
        lambda: A.dsv4_gqa_evict(lens, c, w, 4, positions=torch.zeros(3, 2, 16, dtype=torch.int32)),
        lambda: A.dsv4_gqa_evict(lens, c, w, 4, max_len=33), lambda: A.dsv4_gqa_evict(lens, c, w, 4, lens_out=lens[:2]),
        lambda: A.dsv4_gqa_evict(lens, c, w, 4),                      # not on a CUDA device
    ]
    for i, call in enumerate(calls):
        with pytest.raises(A.Dsv4Error):
            print("call", i)
            call()


# ---------------------------------------------------------------- the oracle
def _small(rng, rows=3, hkv=2, ps=16, width=3, dim=8):
    pages = rows * width + 2
    return {"k": rng.standard_normal((pages, hkv, ps, dim)), "v": rng.standard_normal((pages, hkv, ps, dim)),
            "table": rng.permutation(pages)[:rows * width].reshape(rows, width), "k_scale": None, "v_scale": None}


def test_oracle_decode_against_one_sum():
    rng = np.random.default_rng(3)
    c = _small(rng)
    q = rng.standard_normal((3, 4, 8))
    lens = [37, 0, 16]
    sink = rng.standard_normal(4)
    w = rng.random((3, 2, 48))
    out, lse, wo, err, _ = O.gqa_decode(q, lens, c, max_len=48, scale=0.3, sink=sink, weights=w, weights_out=w * 0 - 1,
                                        decay=0.5)
    assert err == 0
    for b, n in enumerate(lens):
        for i in range(4):
            num, den = np.zeros(8), math.exp(sink[i])
            for s in range(n):
                page = c["table"][b, s // 16]
                e = math.exp(0.3 * float(q[b, i] @ c["k"][page, i // 2, s % 16]))
                num, den = num + e * c["v"][page, i // 2, s % 16], den + e
            assert np.allclose(out[b, i], num / den, atol=1e-12) and abs(lse[b, i] - math.log(den)) < 1e-12
        assert np.all(wo[b, :, n:] == -1)
    # the weights of one request sum to the share of its heads that the sink left
    share = sum(1 - math.exp(sink[i] - lse[0, i]) for i in range(4))
    assert abs((wo[0, :, :37] - 0.5 * w[0, :, :37]).sum() - share) < 1e-10


def test_oracle_decode_of_equal_rows_and_windows():
    rng = np.random.default_rng(4)
    c = _small(rng)
    c["k"][:] = 1.0
    q = np.ones((1, 2, 8))
    out, lse, _, _, _ = O.gqa_decode(q, [40], c, max_len=48, scale=1.0, window=5)
    mean = np.mean([c["v"][c["table"][0, s // 16], 0, s % 16] for s in range(35, 40)], axis=0)
    assert np.allclose(out[0, 0], mean) and abs(lse[0, 0] - (8 + math.log(5))) < 1e-12


def test_oracle_evict_keeps_the_heaviest_and_moves_the_least():
    rng = np.random.default_rng(5)
    c = _small(rng)
    w = rng.random((3, 2, 48))
    w[0, 0, 5] = np.nan
    pos = np.stack([np.stack([rng.permutation(48) for _ in range(2)]) for _ in range(3)])
    lens = [40, 10, 30]
    n_out, k, v, wo, po, err = O.gqa_evict(lens, c, w, 20, max_len=48, first=2, recent=3, positions=pos,
                                           seq_lens=[48, 48, 48])
    assert err == 0 and n_out.tolist() == [20, 10, 20]
    for b, n in enumerate(lens):
        for h in range(2):
            rows = {s: c["k"][c["table"][b, s // 16], h, s % 16].tobytes() for s in range(n)}
            m = min(n, 20)
            left = [k[c["table"][b, s // 16], h, s % 16].tobytes() for s in range(m)]
            kept = [s for s in range(n) if rows[s] in left]
            assert len(kept) == m
            gone = [s for s in range(n) if s not in kept]
            must = [s for s in range(n) if pos[b, h, s] < 2 or pos[b, h, s] >= 45]
            assert not set(must) & set(gone)
            free = [s for s in kept if s not in must]
            if gone:
                assert np.nanmin(w[b, h, free]) >= np.nanmax(w[b, h, gone])
            # a kept row below the bound stays where it was
            assert all(left[s] == rows[s] for s in kept if s < m)
            # weights and positions went with their rows
            back = {x: s for s, x in rows.items()}
            for s in range(m):
                src = back[left[s]]
                assert po[b, h, s] == pos[b, h, src]
                assert wo[b, h, s] == w[b, h, src] or np.isnan(w[b, h, src])


def test_oracle_evict_ties_go_to_the_lower_slot():
    c = _small(np.random.default_rng(6))
    w = np.zeros((3, 2, 48))
    _, k, _, _, _, _ = O.gqa_evict([30, 0, 0], c, w, 12, max_len=48)
    assert np.array_equal(k, c["k"])            # slots 0 .. 11 are kept, nothing moves


def test_counts_whose_arithmetic_would_wrap_are_refused(A):
    # slots and tokens are ints, and tiles and runs of them end behind the last
    wide = ctypes.addressof(_cache(A, page_size=1024, page_table_width=1 << 21, page_table_stride=1 << 21))
    most = 1 << 30
    assert A.lib().dsv4_gqa_decode_workspace_size(wide, 1, 4, most, 0) > 0
    for max_len in (most + 1, 2**31 - 1):
        assert _decode(A, wide, batch=1, heads=4, max_len=max_len) == -1
        assert _evict(A, wide, batch=1, max_len=max_len, width=2**31) == -1
        assert A.lib().dsv4_gqa_decode_workspace_size(wide, 1, 4, max_len, 0) == 0
        assert A.lib().dsv4_gqa_evict_workspace_size(wide, 1, max_len, 10) == 0
        assert _store(A, wide, n=max_len) == -1


def test_what_a_call_allocates_is_its_streams_own(A, monkeypatch):
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    c = A.make_gqa_cache(k, k.clone(), torch.zeros(3, 2, dtype=torch.int32))
    q, lens, w = torch.zeros(3, 8, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32), torch.zeros(3, 2, 32)
    calls = [
        lambda s: A.dsv4_gqa_decode(q, lens, c, stream=s), lambda s: A.dsv4_gqa_decode(q, lens, c, weights=w, stream=s),
        lambda s: [A.dsv4_gqa_evict(lens, c, w, 4, stream=s)],
    ]
    for call in calls:
        with monkeypatch.context() as m:
            streams = Streams(A, m)
            streams.check(call("given"))
        with monkeypatch.context() as m:
            streams = Streams(A, m)
            call(None)
            assert all(stream == "current" for stream, _ in streams.made) and not streams.recorded
