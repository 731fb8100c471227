"""The 4-bit grouped-query cache and the reading back of rows without a GPU: the oracle's format against its definition,
what the entry points refuse before any launch, and whose memory a call allocates."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import gqa_oracle as O
from tests._gqa4 import BF, F8, HF, Cache4, pack
from tests._streams import Streams
from tests.test_gqa_cpu import A, _cache, _decode, _evict, _store  # noqa: F401


# ---------------------------------------------------------------- the format
def test_oracle_codes_and_scales_are_the_formats():
    every = torch.arange(256, dtype=torch.uint8)
    want = every.view(F8).double().numpy()
    codes = np.full((256, 8), 0x22, np.uint8)                      # 16 times 1.0
    got = O.e2m1_values(codes, every.numpy()[:, None])
    assert np.array_equal(got, np.repeat(want[:, None], 16, 1), equal_nan=True)
    for c in range(16):
        e, m = c >> 1 & 3, c & 1
        size = m * 0.5 if e == 0 else (1 + m / 2) * 2.0 ** (e - 1)
        got = O.e2m1_values(np.full((1, 8), c | (c ^ 8) << 4, np.uint8), np.array([[0x38]], np.uint8))
        assert np.array_equal(got[0, ::2], [size if c < 8 else -size] * 8)      # the low half is the even dim
        assert np.array_equal(got[0, 1::2], [-size if c < 8 else size] * 8)


def test_oracle_pack_takes_the_nearest_value():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((200, 32)) * 2.0 ** rng.integers(-8, 9, (200, 1))).astype(np.float32)
    codes, blocks = O.e2m1_pack(x, np.float32(1))
    sizes = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    scales = torch.arange(127, dtype=torch.uint8).view(F8).double().numpy()
    for i in range(200):
        for b in range(2):
            y = x[i, 16 * b: 16 * b + 16].astype(np.float64)
            want = abs(float(np.float32(abs(y).max()) / np.float32(6)) - scales)
            assert want[blocks[i, b]] == want.min()
            step = scales[blocks[i, b]]
            for d in range(16):
                byte = codes[i, 8 * b + d // 2]
                c = byte >> 4 if d % 2 else byte & 15
                if step == 0:
                    assert c == 0
                    continue
                q = float(np.float32(y[d]) / np.float32(step))
                off = [abs(abs(q) - s) for s in sizes]
                assert off[c & 7] == min(off) and (c >= 8) == (y[d] < 0)


def test_oracle_pack_ties_zeros_and_values_without_a_code():
    x = np.zeros((1, 16), np.float32)
    x[0, :9] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.0]        # block scale 1: borders go to the even code
    codes, blocks = O.e2m1_pack(x, np.float32(1))
    assert blocks[0, 0] == 0x38
    assert O.e2m1_values(codes, blocks)[0, :8].tolist() == [6, 0, 1, 1, 2, 2, 4, 4] and codes[0, 4] & 15 == 8
    x[0, 1] = np.nan
    codes, blocks = O.e2m1_pack(x, np.float32(1))
    assert blocks[0, 0] == 0x7f and not codes.any()
    x[0, 1] = -np.inf
    codes, blocks = O.e2m1_pack(x, np.float32(2))
    assert blocks[0, 0] == 0x7e and O.e2m1_values(codes, blocks)[0, :3].tolist() == [0, -6 * 448, 0]
    codes, blocks = O.e2m1_pack(np.full((1, 16), 1e-4, np.float32), np.float32(1))     # below half the smallest scale
    assert not codes.any() and not blocks.any()


def test_oracle_load_is_the_inverse_of_what_was_packed():
    c = Cache4(hkv=2, dim=64, rows=2, slots=40, seed=1)
    k, v, err = O.gqa_load([1, 0, 5, 0, 1], [3, 39, 0, 48, -1], c.oracle())
    assert err == O.ERR_LOAD_ROW and not k[2:].any() and not v[2:].any()
    page = int(c.table[1, 0])
    want = O.e2m1_values(c.k[page, :, 3].numpy(), c.kb[page, :, 3].numpy()) * c.ks.double().numpy()[:, None]
    assert np.array_equal(k[0], want)
    # rows that are values of the format already come back as they are
    x = torch.randn(9, 2, 64).clamp(-3, 3)
    x[..., ::16] = 6.0
    x = torch.from_numpy(O.e2m1_values(*(y.numpy() for y in pack(x, None)))).float()
    again = O.e2m1_values(*(y.numpy() for y in pack(x, None)))
    assert np.array_equal(again, x.double().numpy())


# ---------------------------------------------------------------- refusals
FOUR = dict(format=4, page_stride=65536, head_stride=4096, row_stride=64, k_blocks=1 << 20, v_blocks=1 << 21,
            block_page_stride=8192, block_head_stride=256, block_row_stride=8)


def _load(A, c, k=1 << 20, kt=512, kh=128, v=1 << 21, vt=512, vh=128, type=0, n=3, req=4096, slots=4096):
    return A.lib().dsv4_gqa_load(req, slots, n, c, k, kt, kh, v, vt, vh, type, None)


BAD_CACHES = [
    (dict(k_blocks=None), -1), (dict(v_blocks=None), -1), (dict(k_blocks=(1 << 20) + 8), -1), (dict(v_blocks=8), -1),
    (dict(block_page_stride=12), -1), (dict(block_head_stride=4), -1), (dict(block_row_stride=7), -1),
    (dict(block_row_stride=-8), -1), (dict(row_stride=72), -1), (dict(head_dim=96), -2), (dict(format=5), -2),
    (dict(format=3), -2), (dict(k=None), -1), (dict(page_size=8), -2),
]


@pytest.mark.parametrize("fields,want", BAD_CACHES)
def test_bad_caches_are_refused(A, fields, want):  # noqa: F811
    c = ctypes.addressof(_cache(A, **{**FOUR, **fields}))
    assert _decode(A, c) == want and _store(A, c) == want and _evict(A, c) == want and _load(A, c) == want
    assert A.lib().dsv4_gqa_decode_workspace_size(c, 4, 16, 100, 0) == 0
    assert A.lib().dsv4_gqa_evict_workspace_size(c, 4, 100, 10) == 0


LOAD_REFUSALS = [
    (dict(k=None), -1), (dict(v=None), -1), (dict(k=4104), -1), (dict(v=4100), -1), (dict(n=-1), -1),
    (dict(n=(1 << 30) + 1), -1), (dict(kt=516), -1), (dict(vh=4), -1), (dict(req=None), -1), (dict(slots=None), -1),
    (dict(type=2), -2), (dict(type=4), -2), (dict(n=0, k=None), 0),
    # rows that share memory
    (dict(kt=0), -1), (dict(kh=0), -1), (dict(vt=504), -1), (dict(vh=120), -1), (dict(kt=-512), -1), (dict(v=1 << 20), -1),
    (dict(v=(1 << 20) + 128), -1), (dict(v=(1 << 20) + 256), -1), (dict(kt=1 << 61), -1), (dict(kt=1 << 61, n=1 << 30), -1),
]


@pytest.mark.parametrize("args,want", LOAD_REFUSALS)
@pytest.mark.parametrize("format", [4, 0])
def test_load_refusals(A, args, want, format):  # noqa: F811
    c = ctypes.addressof(_cache(A, **(FOUR if format == 4 else {})))
    assert _load(A, c, **args) == want


def test_load_takes_outputs_that_lie_side_by_side(A):  # noqa: F811
    if torch.cuda.is_available():
        pytest.skip("a device is present")
    c = ctypes.addressof(_cache(A, **FOUR))
    for args in (dict(kt=1024, vt=1024, v=(1 << 20) + 1024),                       # K heads, then V heads of a token
                 dict(kt=1024, vt=1024, kh=256, vh=256, v=(1 << 20) + 256),        # a K and a V head in turn
                 dict(kt=128, vt=128, kh=384, vh=384, v=(1 << 20) + 2 * 4 * 384),  # heads outermost
                 dict(kt=0, vt=0, n=1, v=(1 << 20) + 1024), dict(type=1)):
        assert _load(A, c, **args) == -4                                           # as far as the missing device


def test_rows_of_16_bit_caches_keep_their_type(A):  # noqa: F811
    for format, type, want in ((0, 1, -2), (1, 0, -2)):
        assert _load(A, ctypes.addressof(_cache(A, format=format)), type=type) == want


def test_without_a_device_the_calls_report_cuda_errors(A):  # noqa: F811
    if torch.cuda.is_available():
        pytest.skip("a device is present")
    c = ctypes.addressof(_cache(A, **FOUR))
    assert _decode(A, c) == -4 and _store(A, c) == -4 and _evict(A, c) == -4 and _load(A, c) == -4
    assert _decode(A, c, type=1) == -4 and _store(A, c, type=1) == -4


def _pools(hkv=2, page=16, dim=64):
    return torch.zeros(4, hkv, page, dim // 2, dtype=torch.uint8), torch.zeros(4, hkv, page, dim // 16).to(F8)


def test_binding_refuses_what_is_not_a_4_bit_cache(A):  # noqa: F811
    k, b = _pools()
    table = torch.zeros(2, 2, dtype=torch.int32)
    bad = [dict(), dict(k_blocks=b), dict(v_blocks=b), dict(k_blocks=b, v_blocks=b.float()),
           dict(k_blocks=b.view(torch.uint8), v_blocks=b.view(torch.uint8)), dict(k_blocks=b[:2], v_blocks=b[:2]),
           dict(k_blocks=b[..., :2], v_blocks=b[..., :2]),
           dict(k_blocks=b, v_blocks=b.transpose(1, 2).contiguous().transpose(1, 2)),
           dict(k_blocks=b, v_blocks=b, k_scale=torch.ones(3))]
    for kw in bad:
        with pytest.raises(A.Dsv4Error):
            A.make_gqa_cache(k, k, table, **kw)
    x = torch.zeros(4, 2, 16, 64, dtype=BF)
    with pytest.raises(A.Dsv4Error):
        A.make_gqa_cache(x, x, table, k_blocks=b, v_blocks=b)
    for codes in (k, k.view(torch.float4_e2m1fn_x2)):
        c = A.make_gqa_cache(codes, codes, table, k_blocks=b, v_blocks=b, v_scale=torch.ones(2))
        assert (c.num_kv_heads, c.page_size, c.head_dim, c.format, c.row_stride) == (2, 16, 64, 4, 32)
        assert (c.block_page_stride, c.block_head_stride, c.block_row_stride) == (128, 64, 4)


def test_binding_refuses_mismatched_arguments(A):  # noqa: F811
    k, b = _pools()
    c = A.make_gqa_cache(k, k, torch.zeros(3, 2, dtype=torch.int32), k_blocks=b, v_blocks=b)
    x = torch.zeros(4, 4, 16, 64, dtype=HF)
    half = A.make_gqa_cache(x, x, torch.zeros(3, 2, dtype=torch.int32))
    n = torch.zeros(3, dtype=torch.int32)
    out = torch.zeros(3, 2, 64, dtype=BF)
    calls = [
        lambda: A.dsv4_gqa_load(n[:2], n, c), lambda: A.dsv4_gqa_load(n.long(), n, c), lambda: A.dsv4_gqa_load(n, n, c, k=out),
        lambda: A.dsv4_gqa_load(n, n, c, dtype=torch.float32), lambda: A.dsv4_gqa_load(n, n, c, dtype=F8),
        lambda: A.dsv4_gqa_load(n, n, c, dtype=torch.uint8), lambda: A.dsv4_gqa_load(n, n, half, dtype=BF),
        lambda: A.dsv4_gqa_load(n, n, c, dtype=HF, k=out, v=out.clone()),
        lambda: A.dsv4_gqa_load(n, n, c, k=out, v=out.half()), lambda: A.dsv4_gqa_load(n, n, c, k=out[:2], v=out[:2]),
        lambda: A.dsv4_gqa_load(n, n, c, k=out[..., ::2], v=out[..., ::2]),
        lambda: A.dsv4_gqa_load(n, n, c, k=out, v=out.clone()),       # not on a CUDA device
        lambda: A.dsv4_gqa_decode(out.float(), n, c), lambda: A.dsv4_gqa_decode(out[..., :32], n, c),
        lambda: A.dsv4_gqa_decode(out, n, c),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(A.Dsv4Error):
            print("call", i)
            call()


def test_what_a_load_allocates_is_its_streams_own(A, monkeypatch):  # noqa: F811
    k, b = _pools()
    c = A.make_gqa_cache(k, k.clone(), torch.zeros(3, 2, dtype=torch.int32), k_blocks=b, v_blocks=b)
    n = torch.zeros(3, dtype=torch.int32)
    for call in (lambda s: A.dsv4_gqa_load(n, n, c, stream=s), lambda s: A.dsv4_gqa_load(n, n, c, dtype=HF, stream=s)):
        with monkeypatch.context() as m:
            streams = Streams(A, m)
            streams.check(call("given"))
        with monkeypatch.context() as m:
            streams = Streams(A, m)
            call(None)
            assert all(stream == "current" for stream, _ in streams.made) and not streams.recorded
