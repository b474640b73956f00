"""Rotary frequencies against their formulas, and the refusals of the norm-and-rotation calls."""
import ctypes
import math

import pytest
import torch

import kv_chunk_selection_b200 as lsa

INVALID, UNSUPPORTED, MISALIGNED, NO_DEVICE = -1, -2, -6, -7


@pytest.fixture(scope="module")
def L():
    from kv_chunk_selection_b200 import build
    build.build()
    return lsa.lib()


@pytest.mark.parametrize("rot", [8, 64, 120, 128])
def test_unscaled_and_linear(rot):
    f, s = lsa.rope_frequencies(rot, 10000.0)
    assert f.dtype == torch.float32 and f.numel() == rot // 2 and s == 1.0
    for i in range(rot // 2):
        assert f[i].item() == pytest.approx(10000.0 ** (-2 * i / rot), rel=2 ** -23)
    g, s = lsa.rope_frequencies(rot, 10000.0, scaling="linear", factor=4.0)
    assert torch.equal(g, f / 4) and s == 1.0


def test_scaled_base_keeps_the_fastest_pair_and_stretches_the_slowest():
    f, _ = lsa.rope_frequencies(128, 10000.0)
    g, s = lsa.rope_frequencies(128, 10000.0, scaling="base", factor=8.0)
    assert g[0] == f[0] == 1 and s == 1.0
    assert (f[-1] / g[-1]).item() == pytest.approx(8.0, rel=1e-6)
    assert torch.all(g[1:] < f[1:])


def test_interpolation_by_parts():
    n, factor = 4096, 16.0
    f, _ = lsa.rope_frequencies(128, 10000.0)
    g, s = lsa.rope_frequencies(128, 10000.0, scaling="parts", factor=factor, original_context=n)
    assert s == pytest.approx(0.1 * math.log(factor) + 1)
    for i in range(64):
        fi = 10000.0 ** (-2 * i / 128)
        turns = n * fi / (2 * math.pi)
        if turns >= 32:
            assert g[i] == f[i]
        elif turns <= 1:
            assert g[i].item() == pytest.approx(fi / factor, rel=2 ** -23)
        else:
            keep = (turns - 1) / 31
            assert g[i].item() == pytest.approx(fi * keep + fi / factor * (1 - keep), rel=2 ** -23)


@pytest.mark.parametrize("bad", [dict(rot_dim=0), dict(rot_dim=12), dict(rot_dim=136), dict(rot_dim=64, scaling="other"),
                                 dict(rot_dim=64, base=0.0), dict(rot_dim=64, scaling="linear", factor=0.5),
                                 dict(rot_dim=64, scaling="parts", factor=2.0),
                                 dict(rot_dim=64, scaling="parts", factor=2.0, original_context=64, slow=4, fast=4)])
def test_frequencies_refuse(bad):
    with pytest.raises(ValueError):
        lsa.rope_frequencies(**bad)


def dense(L, qkv=0x100000, stride=10240, T=1, wq=None, wk=None, eps=1e-6, pos=0x200000, freq=0x300000, rot=128, scale=1.0,
          flags=0, q=0x400000, k=0x500000, v=0x600000):
    p = lambda x: None if x is None else ctypes.c_void_p(x)  # noqa: E731
    return L.lsa_qk_norm_rope(p(qkv), stride, T, p(wq), p(wk), ctypes.c_float(eps), p(pos), p(freq), rot,
                              ctypes.c_float(scale), flags, p(q), p(k), p(v), None)


@pytest.mark.parametrize("bad,status", [
    (dict(qkv=None), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(T=0), INVALID), (dict(T=-1), INVALID),
    (dict(stride=10232), INVALID), (dict(rot=-8), INVALID), (dict(rot=136), INVALID), (dict(pos=None), INVALID),
    (dict(freq=None), INVALID), (dict(eps=-1e-6), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(scale=float("inf")), INVALID), (dict(flags=2), INVALID),
    (dict(rot=12), UNSUPPORTED), (dict(T=1 << 31), UNSUPPORTED), (dict(qkv=0x100008), MISALIGNED),
    (dict(stride=10244), MISALIGNED), (dict(q=0x400002), MISALIGNED), (dict(v=0x600008), MISALIGNED),
    (dict(k=0x600000), INVALID), (dict(k=0x400000), INVALID), (dict(v=0x400000), INVALID), (dict(wq=0x700004), MISALIGNED), (dict(wk=0x700008), MISALIGNED)])
def test_dense_form_refuses(L, bad, status):
    assert dense(L, **bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(v=None), INVALID), (dict(seq=None), INVALID), (dict(cpos=None), INVALID), (dict(B=0), INVALID),
    (dict(max_chunks=0), INVALID), (dict(n_slots=0), INVALID), (dict(T=0), INVALID), (dict(v=0x500000), INVALID),
    (dict(v=0x600008), MISALIGNED)])
def test_pool_form_refuses(L, bad, status):
    a = dict(v=0x600000, seq=0x700000, cpos=0x200000, B=1, max_chunks=4, n_slots=4, T=1)
    a.update(bad)
    p = lambda x: None if x is None else ctypes.c_void_p(x)  # noqa: E731
    assert L.lsa_qk_norm_rope_pool(p(0x100000), 10240, a["T"], None, None, ctypes.c_float(1e-6), p(0x200000), p(0x300000),
                                   128, ctypes.c_float(1.0), 0, p(0x400000), p(0x500000), p(a["v"]), a["n_slots"], None,
                                   p(a["seq"]), p(a["cpos"]), a["B"], a["max_chunks"], None) == status


@pytest.mark.skipif(torch.cuda.is_available(), reason="asserts the answer on a machine without a GPU")
def test_no_device_answer(L):
    assert dense(L) == NO_DEVICE
    assert dense(L, rot=0, pos=None, freq=None, v=None) == NO_DEVICE


def test_binding_refuses_other_types_and_shapes():
    e = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype)  # noqa: E731
    with pytest.raises(TypeError, match="qkv"):
        lsa.lsa_qk_norm_rope(e(2, 10240), None, None, e(2, 64, 128), e(2, 8, 128))   # not on a GPU
    with pytest.raises(TypeError, match="qkv"):
        lsa.lsa_qk_norm_rope(e(2, 10240, dtype=torch.float16), None, None, e(2, 64, 128), e(2, 8, 128))
    with pytest.raises(ValueError, match="k_pool"):
        lsa._pool(torch.empty((8, 4, 64, 128), dtype=torch.bfloat16), "k_pool")
