"""Infinite scores in the pool attention calls: rows are numbers, NaN or zeros exactly where the formula's are.

A key of +inf or -inf in one dim makes every score with it infinite (the queries have no zero there), of the sign of
the product.  A softmax over a +inf is NaN; a -inf adds nothing, unless all scores that a row sees are -inf: 0 / 0.
"""
import pytest
import torch

import kv_chunk_selection_b200 as lsa
from pool_testlib import PrefixCase, SCALE, WindowCase, assert_close

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from kv_chunk_selection_b200 import build
    build.build()
    lsa.lib()
    lsa.read_device_status()


def formula(q, k, v, see):
    """As pool_testlib.attend, with the NaN of 0 / 0 and inf - inf kept; rows that see nothing are zeros."""
    q, k, v = q.double(), k.double().repeat_interleave(8, 1), v.double().repeat_interleave(8, 1)
    s = torch.einsum("rhd,khd->rhk", q, k) * SCALE
    s = s.masked_fill(~see[:, None], -INF)
    p = torch.softmax(s, -1).masked_fill(~see.any(-1)[:, None, None], 0.0)
    return torch.einsum("rhk,khd->rhd", p, v), torch.einsum("rhk,khd->rhd", p, v.abs())


def assert_formula(got, ref, mag):
    got, bad = got.cpu().double(), ref.isnan().any(-1)
    assert torch.equal(got.isnan().all(-1), bad), "rows that are not a number"
    assert_close(got[~bad], ref[~bad], mag[~bad])
    return int(bad.sum())


def put(c, b, token, value, dim=5, head=slice(None)):
    """The value in one dim of a cached token's keys (all KV heads), on both sides."""
    c.kv[b][0][token, head, dim] = value
    c.d_k[int(c.d_table[b, token // 64]), head, token % 64, dim] = value


def no_zero_queries(c, dim=5):
    q = c.q[..., dim]
    q[q == 0] = 1.0
    c.d_q.copy_(c.q)


def check(c):
    out, bad = c.call(), 0
    for b, (nq, n) in enumerate(c.seqs):
        rows = slice(c.cu[b], c.cu[b + 1])
        if nq:
            bad += assert_formula(out[rows], *formula(c.q[rows], *c.kv[b], c.see[b]))
    assert lsa.read_device_status() == 0
    return bad


@pytest.mark.parametrize("place", range(8))
@pytest.mark.parametrize("seqs", [[(1, 64)], [(1, 3000)], [(2, 130)], [(3, 3000)], [(40, 64)], [(40, 2500)]])
def test_one_infinite_key_wherever_it_stands_in_its_chunk(seqs, place):
    """Whole tiles and split ones, narrow and wide; the scores that are +inf lie at one place in their chunk only."""
    for sign in (1, -1):
        c = WindowCase(seqs, 1 << 20, 0, seed=place)
        no_zero_queries(c)
        nq, n = seqs[0]
        put(c, 0, (n - nq) // 128 * 64 + place, sign * INF)
        assert check(c) > 0                           # half of the rows, about


@pytest.mark.parametrize("value", [INF, -INF])
@pytest.mark.parametrize("seqs,window,sinks", [([(1, 70)], 6, 0), ([(1, 3000)], 2900, 2), ([(5, 64), (1, 0), (1, 1)], 1, 0),
                                               ([(33, 200), (40, 40)], 3, 1), ([(40, 2500)], 2000, 0)])
def test_nothing_but_infinite_scores(seqs, window, sinks, value):
    """All keys of all tokens: rows see +inf, or nothing but -inf, or (before the first token) nothing."""
    c = WindowCase(seqs, window, sinks, seed=3)
    no_zero_queries(c)
    for b, (nq, n) in enumerate(seqs):
        for t in range(n):
            if bool(c.see[b][:, t].any()):
                put(c, b, t, value)
    assert check(c) == 64 * sum(min(nq, n) for nq, n in seqs)


def test_only_minus_infinity_in_some_shares_of_a_split_row():
    """The rows whose other shares hold numbers are those numbers' average."""
    for nq in (1, 40):
        c = WindowCase([(nq, 3000)], 1 << 20, 0, seed=nq)
        c.q[..., 5] = c.q[..., 5].abs() + 1
        c.d_q.copy_(c.q)
        for t in list(range(0, 1400)) + list(range(1500, 2900)):
            put(c, 0, t, -INF)
        assert check(c) == 0
        for t in list(range(1400, 1500)) + list(range(2900, 3000)):
            put(c, 0, t, -INF)
        assert check(c) == 64 * nq


def test_an_unseen_infinite_key_changes_nothing():
    c = WindowCase([(40, 300), (1, 150)], 20, 0)
    good = c.call()
    c.d_k[int(c.d_table[1, 2]), :, 22:] = INF          # behind the last token
    c.d_k[int(c.d_table[0, 4]), :, 3, 5] = INF         # token 259, before the first query
    out = c.call()
    seen = c.see[0][:, 259]
    assert torch.equal(out[:40][~seen.cuda()], good[:40][~seen.cuda()]) and torch.equal(out[40:], good[40:])
    assert lsa.read_device_status() == 0


@pytest.mark.parametrize("place", [0, 5, 6, 7])
@pytest.mark.parametrize("groups,suffix", [([(3, 64)], [0, 1, 64, 3]), ([(20, 2000)], [5] * 22), ([], [700, 9])])
def test_prefixes_with_an_infinite_key(groups, suffix, place):
    for value in (INF, -INF):
        for prefix in ([True, False] if groups else [False]):
            c = PrefixCase(groups, suffix, seed=place)
            c.q[..., 5] = c.q[..., 5].abs() + 1
            c.q[1, ::2, 5] *= -1
            c.d_q.copy_(c.q)
            if prefix:
                c.prefix[0][1][place, :, 5] = value
                c.d_k[int(c.d_prefix[0, 0]), :, place, 5] = value
            else:
                for b, n in enumerate(suffix):
                    if n > place:
                        c.own[b][1][place, :, 5] = value
                        c.d_k[int(c.d_table[b, 0]), :, place, 5] = value
            check_prefix(c)


def test_a_prefix_of_minus_infinity():
    """With own tokens, theirs is the answer; without any, 0 / 0; no token at all stays zeros."""
    for groups, suffix in (([(2, 64), (1, 0)], [0, 3, 0]), ([(12, 1500)], [0, 9] * 6)):
        c = PrefixCase(groups, suffix, seed=1)
        c.q[..., 5] = c.q[..., 5].abs() + 1
        c.d_q.copy_(c.q)
        c.prefix[0][1][..., 5] = -INF
        c.d_k[c.d_prefix[0, : (groups[0][1] + 63) // 64].long(), ..., 5] = -INF
        assert check_prefix(c) == 64 * sum(n == 0 for n in suffix[: groups[0][0]])


def check_prefix(c):
    out, bad = c.call(), 0
    for b in range(c.B):
        n = next((n for n in range(len(c.groups)) if c.cu[n] <= b < c.cu[n + 1]), None)
        _, k, v = c.own[b]
        if n is not None:
            k, v = torch.cat((c.prefix[n][1], k)), torch.cat((c.prefix[n][2], v))
        if k.shape[0] == 0:
            assert bool((out[b] == 0).all())
            continue
        bad += assert_formula(out[b: b + 1], *formula(c.q[b: b + 1], k, v, torch.ones((1, k.shape[0]), dtype=torch.bool)))
    assert lsa.read_device_status() == 0
    return bad


def test_the_formula_of_this_file():
    """On the CPU's side: against one row worked out by hand."""
    q = torch.ones((1, 64, 128))
    k = torch.zeros((3, 8, 128))
    k[1, :, 5], k[2, :, 5] = -INF, 8.0 / SCALE
    v = torch.arange(3.0)[:, None, None].expand(3, 8, 128)
    out, _ = formula(q, k, v, torch.tensor([[True, True, True]]))
    assert torch.allclose(out, torch.full_like(out, 2 * torch.sigmoid(torch.tensor(8.0)).item()), atol=1e-6)
    assert bool(formula(q, k, v, torch.tensor([[False, True, False]]))[0].isnan().all())
    assert bool((formula(q, k, v, torch.tensor([[False, False, False]]))[0] == 0).all())
