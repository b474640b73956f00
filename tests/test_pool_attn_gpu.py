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


@pytest.mark.parametrize("window,sinks", [(1 << 20, 0), (70, 5)])
@pytest.mark.parametrize("B,nq", [(1, 2), (1, 3), (1, 8), (2, 4), (2, 5), (2, 8), (3, 7), (4, 8)])
def test_a_few_queries_of_a_few_sequences(B, nq, window, sinks):
    """Both sides of the choice between a fold in the kernel and a second one."""
    c = WindowCase([(nq - b % 2, 1500 - 400 * b) for b in range(B)], window, sinks, seed=10 * B + nq, spare_rows=2)
    a = c.call()
    c.check(a)
    assert torch.equal(a, c.call())
    clean()


@pytest.mark.parametrize("window,sinks", [(1 << 20, 0), (256, 4), (1, 0), (1, 1)])
def test_long_prompt_is_split_over_the_chip(window, sinks):
    c = WindowCase([(700, 700)], window, sinks)
    c.check(c.call())
    clean()


@pytest.mark.parametrize("nq", [1, 3, 40])
def test_chunks_seen_in_part_after_a_call_of_nan(nq):
    """Windows and sinks that end around the 16-token parts of a chunk, right after a call whose K and V are NaN:
    what it left in the SMs' shared memory lies in the rows that are not loaded."""
    for window in (1, 15, 16, 17, 33, 48, 100):
        for sinks in (0, 1, 16, 31, 47):
            c = WindowCase([(nq, n) for n in (300, 333, 400, 64 + nq)], window, sinks, seed=window)
            nan = WindowCase([(nq, 300)] * 8, 1 << 20, 0)
            nan.d_k.fill_(float("nan")), nan.d_v.fill_(float("nan"))
            assert bool(nan.call().isnan().all())
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


def test_offsets_that_wrap_around():
    """Steps of 2^30 with max_q as large: every difference is in range and the last offset is too, but not the rows."""
    c = WindowCase([(1, 5)] * 4 + [(4, 9)], 8, 0)
    good = c.call()
    cu, c.max_q = c.d_cu, 1 << 30
    c.d_cu = i32([0, 1 << 30, -(1 << 31), -(1 << 30), 0, 8])
    ws = lsa.new_window_attn_workspace(5, 1 << 30)
    out = c.call(workspace=ws)
    assert lsa.read_device_status() == CAPACITY and bool((out == 3.0).all())
    c.d_cu = cu
    c.check(c.call(workspace=ws))   # a bound far above the batch's own is allowed
    c.max_q = 4
    assert torch.equal(c.call(), good)
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


@pytest.mark.parametrize("seed", range(4))
def test_ragged_batches_of_prompts_and_tokens(seed):
    """Wide and narrow tiles side by side in one call, at the sizes where a tile changes its kind."""
    g = torch.Generator().manual_seed(seed)
    pick = lambda v: v[int(torch.randint(len(v), (1,), generator=g))]  # noqa: E731
    seqs = []
    for _ in range(9):
        nq = pick([1, 1, 2, 7, 8, 9, 16, 31, 32, 33, 40, 41, 63, 64, 65, 73, 129])
        seqs.append((nq, nq + pick([0, 1, 63, 64, 200, 700])))
    c = WindowCase(seqs, pick([1, 17, 64, 250, 1 << 20]), pick([0, 1, 64, 100]), seed=seed, spare_rows=5)
    c.check(c.call())
    c.check(c.call())
    clean()


def test_one_token_over_a_long_window():
    c = WindowCase([(1, 20001)], 1 << 20, 0)
    c.check(c.call())
    c = WindowCase([(3, 20000), (1, 9000)], 12345, 70)
    c.check(c.call())
    clean()


def test_a_query_or_key_that_is_not_a_number_reaches_the_rows_that_see_it():
    c = WindowCase([(40, 200), (1, 150)], 1 << 20, 0)
    good = c.call()
    c.d_q[7, 3] = float("nan")                    # query 7, head 3
    out = c.call()
    assert bool(out[7, 3].isnan().all())
    out[7, 3] = good[7, 3]
    assert torch.equal(out, good)
    c.d_q.copy_(c.q)
    c.d_k[int(c.d_table[0, 2]), 5, 52] = float("nan")   # token 180 of sequence 0, KV head 5: seen from query 20 on
    out = c.call()
    assert bool(out[20:40, 40:48].isnan().all())
    assert torch.equal(out[:20], good[:20]) and torch.equal(out[40:], good[40:])
    assert torch.equal(out[:, :40], good[:, :40]) and torch.equal(out[:, 48:], good[:, 48:])
    c.d_k.copy_(c.d_k.nan_to_num(0.0))
    c.d_q[7, 3] = float("inf")                    # infinite scores of both signs
    assert bool(c.call()[7, 3].isnan().all())
    clean()


def test_two_calls_at_once_with_workspaces_of_their_own():
    a = WindowCase([(1, 700), (1, 90), (1, 4000)], 1 << 20, 0, seed=1)
    b = WindowCase([(90, 300), (1, 500)], 128, 4, seed=2)
    p = PrefixCase([(20, 600)], [(13 * i) % 200 for i in range(25)], seed=3)
    ref = [x.call() for x in (a, b, p)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for _ in range(10):
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        outs.append([x.call(stream=s) for x, s in zip((a, b, p), streams)])
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(x, y) for x, y in zip(o, ref))
    clean()


def test_one_workspace_for_calls_of_both_kinds():
    """The larger workspace serves a call with few queries too, before and after one with many."""
    many, few = WindowCase([(70, 400), (1, 300)], 1 << 20, 0), WindowCase([(1, 900), (2, 2000)], 1 << 20, 0)
    ws = many.ws
    for _ in range(3):
        many.check(many.call(workspace=ws))
        few.check(few.call(workspace=ws))
    clean()


def test_slots_past_32_bit_offsets():
    """A pool of 2^31 elements and more, its last slots in use."""
    slots = 33000                                  # 2.16e9 elements
    pool = torch.empty((slots, 8, 64, 128), dtype=torch.bfloat16, device="cuda")
    c = WindowCase([(1, 130), (20, 150)], 1 << 20, 0)
    far = torch.full_like(c.d_table, -1)
    for b in range(2):
        for i in range(3):
            s = int(c.d_table[b, i])
            far[b, i] = slots - 1 - 3 * b - i
            pool[slots - 1 - 3 * b - i] = c.d_k[s]
    want = WindowCase.call(c)
    c.d_v, c.d_k = c.d_k, c.d_k                    # keys for values: one pool does
    want = c.call()
    c.d_table, c.d_k, c.d_v = far, pool, pool
    assert torch.equal(c.call(), want)
    out = torch.empty((1, 64, 128), dtype=torch.bfloat16, device="cuda")
    ws = lsa.new_prefix_attn_workspace(1, 1)
    lsa.lsa_prefix_decode_attn(c.d_q[:1], pool, pool, far[1:, :2].contiguous(), i32([0, 1]), i32([128]), far[:1], i32([130]),
                               out, ws)
    k = torch.cat((c.kv[1][0][:128], c.kv[0][0]))
    assert_close(out, *attend(c.q[:1], k, k, torch.ones((1, 258), dtype=torch.bool)))
    qkv = torch.randn((1, 80 * 128), device="cuda").to(torch.bfloat16)
    write = lambda v: lsa.lsa_qk_norm_rope_pool(qkv, None, None, torch.empty_like(out), pool, v, far[:1], i32([0]),  # noqa: E731
                                                i32([129]), far.shape[1])
    with pytest.raises(lsa.LsaError, match="INVALID_ARG"):   # K and V of a token in one place
        write(pool)
    values = torch.empty_like(pool)
    write(values)
    assert torch.equal(pool[slots - 3, :, 1], qkv.view(80, 128)[64:72])
    assert torch.equal(values[slots - 3, :, 1], qkv.view(80, 128)[72:])
    clean()


def test_the_largest_batch():
    B = 4096
    g = torch.Generator(device="cuda").manual_seed(5)
    k, v, q = (torch.randn((B, n, m, 128), generator=g, device="cuda").to(torch.bfloat16) for n, m in ((8, 64), (8, 64), (64, 1)))
    q = q.view(B, 64, 128)
    n = torch.randint(0, 65, (B,), generator=g, device="cuda", dtype=torch.int32)
    out, out2 = torch.empty_like(q), torch.empty_like(q)
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    lsa.lsa_window_attn(q, k, v, None, cu, n, 1, 1, 1 << 20, 0, out, lsa.new_window_attn_workspace(B, 1))
    # as a prefix call: groups of 1 to 64 sequences without a prefix, own tokens only
    cut = sorted({0, B} | {int(x) for x in torch.randint(1, B, (200,), generator=torch.Generator().manual_seed(1))})
    G = len(cut) - 1
    lsa.lsa_prefix_decode_attn(q, k, v, i32([[0]] * G), i32(cut), i32([0] * G), None, n, out2,
                               lsa.new_prefix_attn_workspace(B, G), max_chunks=1)
    for b in list(range(0, B, 257)) + [B - 1]:
        m = int(n[b])
        ref = attend(q[b: b + 1].cpu(), k[b, :, :m].transpose(0, 1).cpu(), v[b, :, :m].transpose(0, 1).cpu(),
                     torch.ones((1, m), dtype=torch.bool))
        assert_close(out[b: b + 1], *ref)
        assert_close(out2[b: b + 1], *ref)
    assert bool((out[n == 0] == 0).all()) and bool((out2[n == 0] == 0).all())
    clean()


@pytest.mark.parametrize("prefix", [False, True])
def test_nothing_is_written_outside_the_buffers(prefix):
    """The output and the workspace, exactly as large as asked for, between guards."""
    c = (PrefixCase([(40, 700), (3, 90)], [(17 * i) % 150 for i in range(50)]) if prefix
         else WindowCase([(150, 400), (1, 900), (40, 100), (9, 9)], 200, 3))
    guarded = lambda n: torch.full((n + 8192,), 0xA5, dtype=torch.uint8, device="cuda")  # noqa: E731
    n, m = c.ws.numel(), c.d_q.numel() * 2
    ws, out = guarded(n), guarded(m)
    ws[4096: 4096 + n] = 0
    want = c.call()
    got = c.call(out[4096: 4096 + m].view(torch.bfloat16).view(c.d_q.shape), workspace=ws[4096: 4096 + n])
    assert torch.equal(got, want)
    for x, size in ((ws, n), (out, m)):
        assert bool((x[:4096] == 0xA5).all()) and bool((x[4096 + size:] == 0xA5).all())
    clean()
