"""lsa_prefix_decode_attn before any sequence has a token of its own: a table [B, 0], as a caller holds it then."""
import ctypes

import pytest
import torch

import kv_chunk_selection_b200 as lsa

INVALID, NO_DEVICE, BAD_COUNT = -1, -7, 1


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from kv_chunk_selection_b200 import build
    build.build()
    lsa.lib()


def call(table, chunks):
    p = ctypes.c_void_p
    return lsa.lib().lsa_prefix_decode_attn(p(0x100000), p(0x200000), p(0x300000), 8, p(0x400000), p(0x410000), p(0x420000), 1,
                                            4, table and p(table), p(0x440000), 2, chunks, ctypes.c_float(0.1), p(0x500000),
                                            p(0x600000), 1 << 40, None)


@pytest.mark.skipif(torch.cuda.is_available(), reason="the pointers are no device memory")
def test_no_table_and_no_chunks_passes_the_checks():
    assert call(None, 0) == NO_DEVICE
    assert call(0x430000, 0) == INVALID and call(None, -1) == INVALID


@pytest.mark.gpu
@pytest.mark.parametrize("groups,B", [([(2, 100), (3, 64)], 5), ([(20, 700)], 22), ([(1, 0)], 1)])
def test_a_table_without_columns(groups, B):
    from pool_testlib import PrefixCase, i32
    lsa.read_device_status()
    c = PrefixCase(groups, [0] * B)
    good = c.call()                                  # a table of -1, one column
    c.check(good)
    c.d_table = torch.empty((B, 0), dtype=torch.int32, device="cuda")
    assert torch.equal(c.call(), good)
    c.d_table = i32([[7, 7, 7]] * B)[:, :0]
    assert torch.equal(c.call(), good)
    c.d_table = None
    assert torch.equal(c.call(max_chunks=0), good)
    assert lsa.read_device_status() == 0
    c.d_slen = i32([1] + [0] * (B - 1))              # a token, but no chunk: counts as none
    assert torch.equal(c.call(max_chunks=0), good)
    assert lsa.read_device_status() == BAD_COUNT
