"""What the binding of the pool operators hands to the C ABI, and what it refuses by itself, on any machine: the library
is replaced by one that records its arguments, and CPU tensors stand for the device's."""
import ctypes

import pytest
import torch

import kv_chunk_selection_b200 as lsa


class Recorder:
    """Converts the arguments as ctypes does and keeps them."""

    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        types = getattr(self.real, name).argtypes

        def call(*args):
            assert len(args) == len(types)
            values = [t.from_param(a) if t in (ctypes.c_void_p, ctypes.c_char_p) else t(a).value for t, a in zip(types, args)]
            self.calls.append((name, [a if t is ctypes.c_void_p else v for t, a, v in zip(types, args, values)]))
            return 0
        return call


@pytest.fixture
def rec(monkeypatch):
    from kv_chunk_selection_b200 import build
    build.build()
    r = Recorder(lsa.lib())
    monkeypatch.setattr(lsa, "_lib", r)
    monkeypatch.setattr(lsa, "_current_device", lambda: -1)       # Tensor.get_device() of a CPU tensor
    monkeypatch.setattr(lsa, "_stream_of", lambda stream, device: None)
    need = lsa._need
    monkeypatch.setattr(lsa, "_need", lambda t, name, dtype, cuda=True: need(t, name, dtype, cuda=False))
    return r


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def window(rec, max_chunks, window=64, sinks=4, max_q=2, table=True):
    q, pool = bf16(3, 64, 128), bf16(2, 8, 64, 128)
    lsa.lsa_window_attn(q, pool, pool, i32(2, 5) if table else None, i32(3), i32(2), max_chunks, max_q, window, sinks,
                        torch.empty_like(q), torch.zeros(16, dtype=torch.uint8))
    name, args = rec.calls[-1]
    assert name == "lsa_window_attn"
    return dict(zip(("B", "max_chunks", "max_q", "window", "n_sink"), args[8:13]))


def test_window_takes_its_chunks_from_the_table(rec):
    assert window(rec, 5)["max_chunks"] == 5
    assert window(rec, None)["max_chunks"] == 5
    assert window(rec, 7, table=False)["max_chunks"] == 7
    with pytest.raises(ValueError, match="max_chunks"):
        window(rec, None, table=False)
    with pytest.raises(ValueError, match="chunk_table"):
        window(rec, 4)


@pytest.mark.parametrize("big", [2 ** 31, 2 ** 32 + 5, 2 ** 63 - 1, 2 ** 70])
def test_numbers_past_32_bits_are_the_largest_number(rec, big):
    """Not what their low 32 bits say: a window, a count of sinks and a bound of queries that are larger than any
    sequence mean all of it; a table's width is refused by the library."""
    args = window(rec, big, window=big, sinks=big, max_q=big, table=False)
    assert args == dict(B=2, max_chunks=2 ** 31 - 1, max_q=2 ** 31 - 1, window=2 ** 31 - 1, n_sink=2 ** 31 - 1)
    args = window(rec, 5, window=-big, sinks=-big, max_q=-big)
    assert args["window"] < 0 and args["n_sink"] < 0 and args["max_q"] < 0


@pytest.mark.parametrize("big", [2 ** 32 + 5, 2 ** 70])
def test_widths_past_32_bits_in_the_other_calls(rec, big):
    q, pool, qkv = bf16(2, 64, 128), bf16(2, 8, 64, 128), bf16(2, 80 * 128)
    lsa.lsa_prefix_decode_attn(q, pool, pool, None, None, None, None, i32(2), torch.empty_like(q),
                               torch.zeros(16, dtype=torch.uint8), max_chunks=big)
    assert rec.calls[-1][1][11:13] == [2, 2 ** 31 - 1]
    lsa.lsa_qk_norm_rope_pool(qkv, None, None, q, pool, pool.clone(), None, i32(2), i32(2), big)
    assert rec.calls[-1][1][18:20] == [1, 2 ** 31 - 1]


def test_a_workspace_for_any_bound_of_queries(monkeypatch):
    sizes = []
    monkeypatch.setattr(torch, "zeros", lambda n, **kw: sizes.append(n))
    lsa.new_window_attn_workspace(2, 1 << 20)
    lsa.new_window_attn_workspace(2, 2 ** 32 + 1)
    assert sizes[0] == sizes[1]


def test_rows_of_any_other_rank_are_refused_by_name(rec, monkeypatch):
    monkeypatch.setattr(torch.Tensor, "is_cuda", True, raising=False)
    for shape in ((), (80 * 128,), (1, 1, 80 * 128)):
        with pytest.raises(ValueError, match="qkv"):
            lsa.lsa_qk_norm_rope(bf16(*shape), None, None, bf16(1, 64, 128), bf16(1, 8, 128))
