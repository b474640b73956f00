"""Window and shared-prefix attention over the paged pools against the formula in 64 bits."""
import pytest
import torch

import kv_chunk_selection_b200 as lsa
from pool_testlib import PrefixCase, WindowCase, assert_close, attend, i32

pytestmark = pytest.mark.gpu
BAD_COUNT, BAD_SLOT, CAPACITY = 1, 2, 8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from kv_chunk_selection_b200 import build
    build.build()
    lsa.lib()
    lsa.read_device_status()


def clean():
    bits = lsa.read_device_status()
    assert bits == 0, lsa.decode_status(bits)


@pytest.mark.parametrize("window,sinks", [(1, 0), (64, 0), (100, 4), (1 << 20, 0), (63, 130)])
@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 129, 700])
def test_one_token(n, window, sinks):
    c = WindowCase([(1, n)], window, sinks, seed=n)
    c.check(c.call())
    clean()


@pytest.mark.parametrize("window,sinks", [(128, 4), (1 << 20, 0), (200, 70)])
def test_decode_batch(window, sinks):
    c = WindowCase([(1, n) for n in (1, 64, 65, 500, 0, 1000, 127, 128, 3, 900)], window, sinks, spare_rows=2)
    c.check(c.call())
    clean()


@pytest.mark.parametrize("nq", [2, 15, 16, 17, 31, 32, 33, 64, 65, 150])
@pytest.mark.parametrize("window,sinks", [(1 << 20, 0), (48, 3), (130, 65)])
def test_pieces_of_a_prompt(nq, window, sinks):
    c = WindowCase([(nq, nq), (nq, nq + 77), (1, 300)], window, sinks, seed=nq, spare_rows=3)
    c.check(c.call())
    clean()


@pytest.mark.parametrize("window,sinks", [(1 << 20, 0), (256, 4), (1, 0), (1, 1)])
def test_long_prompt_is_split_over_the_chip(window, sinks):
    c = WindowCase([(700, 700)], window, sinks)
    c.check(c.call())
    clean()


def test_queries_before_the_first_token_and_empty_sequences():
    # five queries but three cached tokens: the first two see nothing
    c = WindowCase([(5, 5), (0, 100), (4, 4), (0, 0), (40, 40)], 8, 2, spare_rows=1)
    c.d_len = i32([3, 100, 4, 0, 40])
    out = c.call()
    assert bool((out[:2] == 0).all())
    k, v = c.kv[0]
    see = torch.tril(torch.ones(3, 3)).bool()
    assert_close(out[2:5], *attend(c.q[2:5], k[:3], v[:3], see))
    for b in (2, 4):
        rows = slice(c.cu[b], c.cu[b + 1])
        assert_close(out[rows], *attend(c.q[rows], *c.kv[b], c.see[b]))
    assert bool((out[-1] == 3.0).all())
    clean()


def test_large_and_small_scores():
    """Maxima that grow by steps through the list, and a scale that flattens them."""
    for scale in (1.0, 1e-3):
        c = WindowCase([(33, 400), (1, 400)], 1 << 20, 0, seed=9)
        ramp = torch.linspace(0.2, 3, 400)[:, None, None]
        for b in range(2):
            k, v = c.kv[b]
            k.copy_((k.float() * ramp).to(torch.bfloat16))
            for i in range(7):
                n = min(64, 400 - 64 * i)
                c.d_k[int(c.d_table[b, i]), :, :n] = k[64 * i: 64 * i + n].transpose(0, 1).cuda()
        out = c.call(softmax_scale=scale)
        assert bool(torch.isfinite(out).all())
        if scale < 1:
            c.check(out, scale)
        else:
            # scores up to 3 * 128: an fp32 score is off by 130 * 2^-24 * scale * |q| |k| <= 3e-3, so the
            # probabilities by as much; the bound below allows 2^-7 of A for it
            for b, (nq, n) in enumerate(c.seqs):
                rows = slice(c.cu[b], c.cu[b + 1])
                ref, mag = attend(c.q[rows], *c.kv[b], c.see[b], scale)
                err = (out[rows].cpu().double() - ref).abs()
                assert bool((err <= 2.0 ** -8 * ref.abs() + 3 * 2.0 ** -8 * mag).all())
    clean()


def test_identity_layout_and_other_scale():
    c = WindowCase([(20, 128), (1, 70), (17, 100)], 50, 3, max_chunks=2)
    t = c.d_table.clamp(min=0).long()
    c.d_k, c.d_v = (x[t].flatten(0, 1).contiguous() for x in (c.d_k, c.d_v))
    c.d_table = None
    c.check(c.call(softmax_scale=0.3), 0.3)
    clean()


def test_repeated_calls_are_bit_identical_and_captured_ones_too():
    c = WindowCase([(40, 300), (1, 800), (1, 90), (200, 500)], 150, 4)
    a = c.call()
    for _ in range(3):
        assert torch.equal(a, c.call())
    out, out2 = torch.full_like(a, 3.0), torch.full_like(a, 3.0)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        c.call(out)
    with torch.cuda.graph(g2):   # the same workspace: replays follow one another on one stream
        c.call(out2)
    for _ in range(3):
        out.fill_(3.0), out2.fill_(3.0)
        g1.replay(), g2.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, a) and torch.equal(out2, a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = c.call(stream=s)
    s.synchronize()
    assert torch.equal(a, b)
    clean()


def test_bad_offsets_compute_nothing():
    c = WindowCase([(3, 10), (2, 20)], 8, 0)
    good, cu = c.call(), c.d_cu.clone()
    for bad in ([1, 3, 5], [0, 4, 3], [0, 3, 6], [0, -1, 5]):
        c.d_cu = i32(bad)
        out = c.call()
        assert lsa.read_device_status() == CAPACITY and bool((out == 3.0).all())
    c.d_cu = cu
    c.max_q, ws = 2, lsa.new_window_attn_workspace(2, 2)   # sequence 0 has 3
    out = c.call(workspace=ws)
    assert lsa.read_device_status() == CAPACITY and bool((out == 3.0).all())
    c.max_q = 3
    assert torch.equal(c.call(), good)
    clean()


def test_bad_lengths_and_slots_are_reported():
    c = WindowCase([(3, 100), (1, 128), (20, 90)], 64, 4)
    good, lens, tab = c.call(), c.d_len.clone(), c.d_table.clone()
    for bad in (-1, 129, 1 << 30):
        c.d_len = lens.clone()
        c.d_len[1] = bad
        out = c.call()
        assert lsa.read_device_status() == BAD_COUNT
        assert bool((out[3] == 0).all())
        c.check(out, but=(1,))
    c.d_len = lens
    for bad in (-1, c.d_k.shape[0], 1 << 30):
        c.d_table = tab.clone()
        c.d_table[0, 1] = bad
        out = c.call()
        assert lsa.read_device_status() == BAD_SLOT
        assert bool(torch.isfinite(out[:3]).all()) and torch.equal(out[3:], good[3:])
    c.d_table = tab
    assert torch.equal(c.call(), good)
    clean()


@pytest.mark.parametrize("groups,suffix", [
    ([(1, 1)], [0]), ([(1, 64)], [1]), ([(4, 1000)], [1, 64, 0, 65]), ([(16, 130)], list(range(16))),
    ([(17, 130)], [5] * 17), ([(32, 65)], [70] * 32), ([(33, 300)], [3] * 33), ([(70, 513)], [(7 * i) % 90 for i in range(70)]),
    ([(3, 200), (20, 64), (1, 0), (0, 50), (5, 321)], [(11 * i) % 130 for i in range(35)]),
    ([], [1, 100, 0, 64, 700]), ([(2, 0), (2, 40)], [0, 5, 0, 9])])
def test_shared_prefixes(groups, suffix):
    c = PrefixCase(groups, suffix, seed=len(suffix))
    c.check(c.call())
    clean()


def test_prefix_equals_the_window_call_over_the_joined_tokens():
    """A whole-chunk prefix followed by own tokens is one sequence: causal attention over its joined table agrees."""
    c = PrefixCase([(6, 256)], [1, 64, 65, 100, 3, 128])
    joined = torch.cat((c.d_prefix.expand(6, -1), c.d_table), 1).contiguous()
    out = torch.empty_like(c.d_q)
    lsa.lsa_window_attn(c.d_q, c.d_k, c.d_v, joined, i32(range(7)), c.d_slen + 256, joined.shape[1], 1, 1 << 20, 0, out,
                        lsa.new_window_attn_workspace(6, 1))
    ref, mag = c.reference()
    assert_close(out, ref, mag)
    assert_close(c.call(), ref, mag)
    clean()


def test_prefix_identity_layout_repeats_and_captures():
    c = PrefixCase([(20, 200)], [(13 * i) % 64 + 1 for i in range(24)])
    a = c.call()
    assert torch.equal(a, c.call())
    t = c.d_table.clamp(min=0).long()
    n, own = c.d_k.shape[0], t.numel()
    k, v = (torch.cat((x[t].flatten(0, 1), x)).contiguous() for x in (c.d_k, c.d_v))
    c.d_k, c.d_v, c.d_table, c.d_prefix = k, v, None, (c.d_prefix + own).to(torch.int32)
    out = torch.full_like(a, 3.0)
    g = torch.cuda.CUDAGraph()
    c.call(max_chunks=1)
    with torch.cuda.graph(g):
        c.call(out, max_chunks=1)
    out.fill_(3.0)
    g.replay()
    torch.cuda.synchronize()
    assert n and torch.equal(out, a)
    clean()


def test_prefix_refuses_bad_offsets_and_reports_lengths_and_slots():
    c = PrefixCase([(2, 100), (3, 70)], [5, 6, 7, 8, 9, 10])
    ref, mag = c.reference()
    good, cu, plen, slen, tab = c.call(), c.d_cu.clone(), c.d_plen.clone(), c.d_slen.clone(), c.d_table.clone()
    for bad in ([1, 2, 5], [0, 3, 2], [0, 2, 7]):
        c.d_cu = i32(bad)
        out = c.call()
        assert lsa.read_device_status() == CAPACITY and bool((out == 3.0).all())
    c.d_cu = cu
    for bad in (-1, 129):
        c.d_plen = i32([bad, 70])
        out = c.call()
        assert lsa.read_device_status() == BAD_COUNT
        assert bool(torch.isfinite(out[:2]).all())
        assert_close(out[2:], ref[2:], mag[2:])
    c.d_plen = plen
    c.d_slen = i32([5, 6, 65, 8, 9, 10])
    out = c.call()
    assert lsa.read_device_status() == BAD_COUNT
    others = [0, 1, 3, 4, 5]
    assert_close(out[others], ref[others], mag[others])
    c.d_slen = slen
    c.d_table = tab.clone()
    c.d_table[5, 0] = -1
    out = c.call()
    assert lsa.read_device_status() == BAD_SLOT and torch.equal(out[:5], good[:5])
    assert bool((out[5] == 0).all())   # zeros for keys and values
    c.d_table = tab
    assert torch.equal(c.call(), good)
    clean()
