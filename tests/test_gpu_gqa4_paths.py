"""Attention over 4-bit rows on the kernel that each test names: a call that gives every segment a cluster is one launch,
one that shares out the list of tiles is two (with weights three), and every test asserts which of them its calls take.
With 64 and 128 dims and up to 8 query heads per KV head the list is that of the block-scaled tensor cores."""
import pytest
import torch

from tests._gqa4 import BF, Cache4
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
