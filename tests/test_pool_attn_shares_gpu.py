"""Shares of the pool attention's work that other tests do not reach: single tokens joined in the kernel, wide shares of
many tiles, pieces behind a long cache, sequences without a group beside grouped ones."""
import pytest
import torch

import kv_chunk_selection_b200 as lsa
from pool_testlib import PrefixCase, WindowCase, assert_close, attend

pytestmark = pytest.mark.gpu
COUNTS = 2 * 160 * 4   # bytes of the counts at the workspace's start


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from kv_chunk_selection_b200 import build
    build.build()
    lsa.lib()
    lsa.read_device_status()


@pytest.mark.parametrize("window,sinks", [(1 << 20, 0), (70, 5), (1000, 100)])
@pytest.mark.parametrize("B", [1, 2, 3, 4])
def test_single_tokens_joined_in_the_kernel_do_not_depend_on_who_is_last(B, window, sinks):
    c = WindowCase([(1, 1900 - 400 * b) for b in range(B)], window, sinks, seed=B, spare_rows=2)
    a = c.call()
    c.check(a)
    for _ in range(20):
        assert torch.equal(a, c.call())
    assert not bool(c.ws[:COUNTS].any()), "counts are left"
    out, out2 = torch.full_like(a, 3.0), torch.full_like(a, 3.0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call(out)
        c.call(out2)
    for _ in range(10):
        out.fill_(3.0), out2.fill_(3.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, a) and torch.equal(out2, a)
    assert not bool(c.ws[:COUNTS].any())
    assert lsa.read_device_status() == 0


def sample(c, out, b, picks, heads):
    """Some queries and KV heads of sequence b, over the keys that they see."""
    k, v = c.kv[b]
    for i in picks:
        row, j = c.cu[b] + i, torch.nonzero(c.see[b][i])[:, 0]
        see = torch.ones((1, len(j)), dtype=torch.bool)
        ref, mag = attend(c.q[row: row + 1], k[j], v[j], see)
        at = [8 * h + x for h in heads for x in range(8)]
        assert_close(out[row: row + 1, at], ref[:, at], mag[:, at])


@pytest.mark.parametrize("nq,n,window,sinks", [(2500, 2500, 200, 4), (2500, 2500, 64, 0), (3001, 3500, 33, 70),
                                               (2300, 6000, 1 << 20, 0)])
def test_wide_shares_of_many_tiles(nq, n, window, sinks):
    """More than 4 tiles with keys to a share (79 tiles x 8 heads on 148 CTAs): every place of the planner's ring and
    both query tiles are used again and again, and the next tile does not wait for the last one's output."""
    c = WindowCase([(nq, n), (7, 100)], window, sinks, seed=nq, spare_rows=1)
    out = c.call()
    assert torch.equal(out, c.call())
    assert bool(torch.isfinite(out).all()) and bool((out[-1] == 3.0).all())
    g = torch.Generator().manual_seed(nq)
    picks = sorted({0, 1, 31, 32, nq - 33, nq - 32, nq - 1} | set(torch.randint(nq, (60,), generator=g).tolist()))
    sample(c, out, 0, picks, [0, 3, 7])
    sample(c, out, 1, range(7), range(8))
    assert lsa.read_device_status() == 0


@pytest.mark.parametrize("nq", [1, 8, 9, 33, 200])
def test_a_piece_behind_a_long_cache(nq):
    """Causal attention over all that is cached."""
    c = WindowCase([(nq, 30000), (1, 12000)], 1 << 30, 0, seed=nq)
    out = c.call()
    sample(c, out, 0, sorted({0, nq // 2, nq - 1}), [0, 5])
    sample(c, out, 1, [0], [1, 6])
    assert lsa.read_device_status() == 0


@pytest.mark.parametrize("groups,alone,own", [([(33, 500), (2, 64)], 40, 200), ([(9, 3000)], 1, 5000), ([(1, 0), (8, 129)], 23, 65),
                                              ([(64, 2000), (12, 700), (7, 100)], 10, 0)])
def test_sequences_without_a_group_beside_grouped_ones(groups, alone, own):
    B = sum(m for m, _ in groups) + alone
    c = PrefixCase(groups, [(29 * i) % (own + 1) for i in range(B)], seed=B)
    out = c.call()
    c.check(out)
    assert torch.equal(out, c.call())
    assert lsa.read_device_status() == 0
