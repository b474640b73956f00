"""Paged pools for the pool attention tests, and the attention in 64 bits.

Every pool starts as NaN: only the rows that the cached tokens occupy are
written, so a kernel that lets a page's tail, a chunk that was given back or an
unseen token into a sum shows it.

Tolerance, from the kernels' arithmetic.  With A = sum_j p_j |v_j| / sum_j p_j:
the output is rounded once to bf16 (2^-8 of it), each probability once to bf16
(2^-8 of A), and the fp32 part is at most 2^-11 of A: a score of 128 products
is off by at most 130 * 2^-24 of scale * |q| |k| / ln 2 (about 16 for N(0, 1)
values: 1.3e-4), its power of two by 2^-22, and a sum of n / 16 <= 1024 products
of the tensor cores by 1024 * 2^-23 = 1.3e-4.
"""
import numpy as np
import torch

import kv_chunk_selection_b200 as lsa

DEV = "cuda"
SCALE = 1 / np.sqrt(128)


def randn(shape, g):
    return torch.randn(shape, generator=g, dtype=torch.float32).to(torch.bfloat16)


class Pool:
    """Slots given out in shuffled order; `add` caches tokens as a row of a table."""

    def __init__(self, slots, seed):
        self.g = torch.Generator().manual_seed(seed)
        self.k = torch.full((slots, 8, 64, 128), float("nan"), dtype=torch.bfloat16)
        self.v = self.k.clone()
        self.free = torch.randperm(slots, generator=self.g).tolist()

    def add(self, n, live=None):
        """n tokens; live: a bool list of the tokens some query sees (others stay NaN, their chunks at -1)."""
        live = torch.ones(n, dtype=torch.bool) if live is None else torch.as_tensor(live, dtype=torch.bool)
        k, v = randn((n, 8, 128), self.g), randn((n, 8, 128), self.g)
        row = []
        for c in range((n + 63) // 64):
            t = slice(c * 64, min(n, c * 64 + 64))
            if not bool(live[t].any()):
                row.append(-1)
                continue
            s = self.free.pop()
            row.append(s)
            for pool, x in ((self.k, k), (self.v, v)):
                x = torch.where(live[t][:, None, None], x[t].float(), torch.tensor(float("nan"))).to(torch.bfloat16)
                pool[s, :, : x.shape[0]] = x.transpose(0, 1)
        return row, k, v

    def cuda(self):
        return self.k.to(DEV), self.v.to(DEV)


def table(rows, width):
    t = torch.full((len(rows), width), -1, dtype=torch.int32)
    for i, r in enumerate(rows):
        t[i, : len(r)] = torch.tensor(r, dtype=torch.int32)
    return t.to(DEV)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def attend(q, k, v, see, scale=SCALE):
    """q [rows, 64, 128], k and v [keys, 8, 128], see [rows, keys] -> (out, A), fp64 [rows, 64, 128]."""
    q, k, v = q.double(), k.double().repeat_interleave(8, 1), v.double().repeat_interleave(8, 1)
    s = torch.einsum("rhd,khd->rhk", q, k) * scale
    s = s.masked_fill(~see[:, None], -float("inf"))
    p = torch.exp(s - s.amax(-1, keepdim=True).clamp(min=-1e300)) if s.shape[-1] else s
    p = torch.nan_to_num(p / p.sum(-1, keepdim=True))
    return torch.einsum("rhk,khd->rhd", p, v), torch.einsum("rhk,khd->rhd", p, v.abs())


def assert_close(got, ref, mag):
    got = got.cpu().double()
    assert bool(torch.isfinite(got).all()), "not finite"
    bound = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -11) * mag
    err = (got - ref).abs()
    assert bool((err <= bound).all()), f"off by {(err / bound.clamp(min=1e-30)).max()} of the bound"


class WindowCase:
    """Sequences of (queries, cached tokens) under one window."""

    def __init__(self, seqs, window, sinks, seed=0, spare_rows=0, max_chunks=None):
        self.seqs, self.window, self.sinks = seqs, window, sinks
        width = max_chunks or max(1, max((n + 63) // 64 for _, n in seqs))
        pool = Pool(1 + sum((n + 63) // 64 for _, n in seqs), seed)
        cu, rows, kv, self.see = [0], [], [], []
        for nq, n in seqs:
            p = torch.arange(n - nq, n)[:, None]
            j = torch.arange(n)[None]
            see = (j <= p) & ((j > p - window) | (j < sinks))
            row, k, v = pool.add(n, see.any(0) if nq else torch.zeros(n, dtype=torch.bool))
            rows.append(row)
            kv.append((k, v))
            self.see.append(see)
            cu.append(cu[-1] + nq)
        self.kv, self.cu = kv, cu
        self.q = randn((cu[-1] + spare_rows, 64, 128), pool.g)
        self.max_q = max(1, max(q for q, _ in seqs))
        self.d_table, self.d_cu, self.d_len = table(rows, width), i32(cu), i32([n for _, n in seqs])
        self.d_q, (self.d_k, self.d_v) = self.q.to(DEV), pool.cuda()
        self.width = width
        self.ws = lsa.new_window_attn_workspace(len(seqs), self.max_q)

    def call(self, out=None, **kw):
        if out is None:
            out = torch.full_like(self.d_q, 3.0)
        lsa.lsa_window_attn(self.d_q, self.d_k, self.d_v, self.d_table, self.d_cu, self.d_len, self.width, self.max_q,
                            self.window, self.sinks, out, kw.pop("workspace", self.ws), **kw)
        return out

    def check(self, out, scale=SCALE, but=()):
        for b, (nq, n) in enumerate(self.seqs):
            rows = slice(self.cu[b], self.cu[b + 1])
            if nq and b not in but:
                assert_close(out[rows], *attend(self.q[rows], *self.kv[b], self.see[b], scale))
        assert bool((out[self.cu[-1]:] == 3.0).all()), "rows behind the last sequence were written"


class PrefixCase:
    """Groups of (sequences, prefix tokens), then own tokens of every sequence."""

    def __init__(self, groups, suffix, seed=0):
        self.groups, self.suffix = groups, suffix
        B = len(suffix)
        pool = Pool(1 + sum((n + 63) // 64 for n in suffix) + sum((n + 63) // 64 for _, n in groups), seed)
        self.prefix = [pool.add(n) for _, n in groups]
        self.own = [pool.add(n) for n in suffix]
        cu = [0]
        for m, _ in groups:
            cu.append(cu[-1] + m)
        assert cu[-1] <= B
        self.cu, self.B = cu, B
        self.q = randn((B, 64, 128), pool.g)
        wide = lambda v: max(1, max((n + 63) // 64 for n in v))  # noqa: E731
        self.d_prefix = table([r for r, _, _ in self.prefix], wide([n for _, n in groups])) if groups else None
        self.d_table = table([r for r, _, _ in self.own], wide(suffix))
        self.d_cu, self.d_plen = (i32(cu), i32([n for _, n in groups])) if groups else (None, None)
        self.d_slen = i32(suffix)
        self.d_q, (self.d_k, self.d_v) = self.q.to(DEV), pool.cuda()
        self.ws = lsa.new_prefix_attn_workspace(B, len(groups))

    def call(self, out=None, **kw):
        if out is None:
            out = torch.full_like(self.d_q, 3.0)
        lsa.lsa_prefix_decode_attn(self.d_q, self.d_k, self.d_v, self.d_prefix, self.d_cu, self.d_plen, self.d_table,
                                   self.d_slen, out, kw.pop("workspace", self.ws), **kw)
        return out

    def reference(self, scale=SCALE):
        refs, mags = [], []
        for b in range(self.B):
            n = next((n for n in range(len(self.groups)) if self.cu[n] <= b < self.cu[n + 1]), None)
            _, k, v = self.own[b]
            if n is not None:
                k, v = torch.cat((self.prefix[n][1], k)), torch.cat((self.prefix[n][2], v))
            r, m = attend(self.q[b: b + 1], k, v, torch.ones((1, k.shape[0]), dtype=torch.bool), scale)
            refs.append(r)
            mags.append(m)
        return torch.cat(refs), torch.cat(mags)

    def check(self, out, scale=SCALE):
        assert_close(out, *self.reference(scale))
