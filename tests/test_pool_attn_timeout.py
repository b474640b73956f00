"""Waits of the pool attention kernels that run out, without a GPU fault: one CTA is never told its share of the work, so
its bounded waits end, the call reports TIMEOUT and writes no row of which that CTA held a part."""
import pytest
import torch

import kv_chunk_selection_b200 as lsa

INVALID, TIMEOUT = -1, 16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from kv_chunk_selection_b200 import build
    build.build()
    lsa.lib()
    if torch.cuda.is_available():
        lsa.read_device_status()


@pytest.mark.parametrize("cta,limit", [(-2, 1000), (0, 0), (0, 2000001)])
def test_refusals(cta, limit):
    with pytest.raises(lsa.LsaError) as e:
        lsa.lsa_debug_withhold_share(cta, limit)
    assert e.value.status == INVALID


def test_disarmed():
    lsa.lsa_debug_withhold_share(7, 1000)
    lsa.lsa_debug_withhold_share(-1)


def gave_up(c, cta, good):
    """A call with CTA `cta` withheld: its rows are the right ones, or were left as they were."""
    lsa.lsa_debug_withhold_share(cta, 2000)
    out = c.call()
    assert lsa.read_device_status() == TIMEOUT
    rows = (out == good).flatten(1).all(1)
    heads = ((out == good) | (out == 3.0)).view(-1, 8, 8 * 128)
    assert bool(((out == good).view(heads.shape).all(-1) | (out == 3.0).view(heads.shape).all(-1)).all())
    assert not bool(rows.all()), "the CTA's rows were written"
    return out


def other_inputs(c):
    """Leaves partials of other queries in the workspace."""
    q = c.d_q.clone()
    c.d_q.copy_(-2 * q)
    c.call()
    c.d_q.copy_(q)


@pytest.mark.gpu
@pytest.mark.parametrize("seqs,window,sinks", [([(700, 700)], 1 << 20, 0), ([(1, 9000), (2, 20000), (5, 4000)], 1 << 20, 0),
                                               ([(90, 1000), (1, 3000), (33, 600)], 300, 4)])
@pytest.mark.parametrize("cta", [0, 1, 40, 147])
def test_window_call_that_gives_up(seqs, window, sinks, cta):
    from pool_testlib import WindowCase
    c = WindowCase(seqs, window, sinks)
    good = c.call()
    c.check(good)
    other_inputs(c)
    gave_up(c, cta, good)
    c.ws.zero_()
    assert torch.equal(c.call(), good)
    assert lsa.read_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("cta", [0, 70, 147])
def test_single_tokens_that_give_up(cta):
    from pool_testlib import WindowCase
    c = WindowCase([(1, 20001), (1, 700), (1, 9000)], 1 << 20, 0)
    good = c.call()
    c.check(good)
    other_inputs(c)
    gave_up(c, cta, good)
    c.ws.zero_()
    assert torch.equal(c.call(), good)
    assert lsa.read_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("cta", [0, 30, 147])
def test_prefix_call_that_gives_up(cta):
    from pool_testlib import PrefixCase
    c = PrefixCase([(20, 3000), (3, 700)], [(37 * i) % 400 for i in range(25)])
    good = c.call()
    c.check(good)
    other_inputs(c)
    gave_up(c, cta, good)
    assert torch.equal(c.call(), good)
    assert lsa.read_device_status() == 0
