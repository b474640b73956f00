"""Refusals of the pool attention calls, on any machine (no call here gets as far as a launch)."""
import ctypes

import pytest
import torch

import kv_chunk_selection_b200 as lsa

INVALID, UNSUPPORTED, WORKSPACE, MISALIGNED, NO_DEVICE = -1, -2, -3, -6, -7


@pytest.fixture(scope="module")
def L():
    from kv_chunk_selection_b200 import build
    build.build()
    return lsa.lib()


def p(x):
    return None if x is None else ctypes.c_void_p(x)


def window(L, q=0x100000, T=4, k=0x200000, v=0x300000, slots=8, table=0x400000, cu=0x410000, lens=0x420000, B=2, chunks=4,
           max_q=2, window=64, sinks=4, scale=0.1, out=0x500000, ws=0x600000, size=1 << 40):
    return L.lsa_window_attn(p(q), T, p(k), p(v), slots, p(table), p(cu), p(lens), B, chunks, max_q, window, sinks,
                             ctypes.c_float(scale), p(out), p(ws), size, None)


def prefix(L, q=0x100000, k=0x200000, v=0x300000, slots=8, ptable=0x400000, cu=0x410000, plen=0x420000, groups=1, pchunks=4,
           table=0x430000, slen=0x440000, B=2, chunks=4, scale=0.1, out=0x500000, ws=0x600000, size=1 << 40):
    return L.lsa_prefix_decode_attn(p(q), p(k), p(v), slots, p(ptable), p(cu), p(plen), groups, pchunks, p(table), p(slen),
                                    B, chunks, ctypes.c_float(scale), p(out), p(ws), size, None)


SHARED = [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(out=None), INVALID),
    (dict(slots=0), INVALID), (dict(B=0), INVALID), (dict(chunks=0), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(B=4097), UNSUPPORTED), (dict(slots=1 << 22), UNSUPPORTED), (dict(chunks=(1 << 23) + 1), UNSUPPORTED),
    (dict(q=0x100008), MISALIGNED), (dict(k=0x200008), MISALIGNED), (dict(v=0x300002), MISALIGNED),
    (dict(out=0x500008), MISALIGNED), (dict(ws=0x600008), MISALIGNED), (dict(ws=None), WORKSPACE), (dict(size=4096), WORKSPACE)]


@pytest.mark.parametrize("bad,status", SHARED + [
    (dict(cu=None), INVALID), (dict(lens=None), INVALID), (dict(T=0), INVALID), (dict(max_q=0), INVALID),
    (dict(window=0), INVALID), (dict(window=-1), INVALID), (dict(sinks=-1), INVALID), (dict(T=(1 << 30) + 1), UNSUPPORTED)])
def test_window_refuses(L, bad, status):
    assert window(L, **bad) == status


@pytest.mark.parametrize("bad,status", SHARED + [
    (dict(slen=None), INVALID), (dict(ptable=None), INVALID), (dict(cu=None), INVALID), (dict(plen=None), INVALID),
    (dict(groups=-1), INVALID), (dict(groups=3), INVALID), (dict(pchunks=0), INVALID), (dict(pchunks=(1 << 23) + 1), UNSUPPORTED)])
def test_prefix_refuses(L, bad, status):
    assert prefix(L, **bad) == status


def test_workspace_sizes(L):
    w = L.lsa_window_attn_workspace_size
    assert w(0, 1) == w(4097, 1) == w(1, 0) == 0
    # two records for each of 160 CTAs' two shares: rows of 128 floats and a log-sum-exp
    assert 0 < w(1, 1) - 4 * 160 * 8 * 129 * 4 < 1 << 16
    assert w(1, 1) < w(1, 8) < w(1, 9) == w(4096, 1 << 20)
    x = L.lsa_prefix_attn_workspace_size
    assert x(0, 0) == x(4097, 1) == x(1, 2) == x(1, -1) == 0
    assert 0 < x(4, 1) < x(5, 1) < x(64, 64)
    need = w(2, 2)
    assert window(L, size=need - 1) == WORKSPACE
    assert prefix(L, size=x(2, 1) - 1) == WORKSPACE


@pytest.mark.skipif(torch.cuda.is_available(), reason="asserts the answer on a machine without a GPU")
def test_no_device_answer(L):
    assert window(L) == NO_DEVICE and window(L, table=None) == NO_DEVICE
    assert prefix(L) == NO_DEVICE
    assert prefix(L, groups=0, ptable=None, cu=None, plen=None, pchunks=0, table=None) == NO_DEVICE
