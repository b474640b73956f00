"""The pool operators together, as a serving step uses them: a prompt's rows are normed, rotated and written into the
pool, attended under a sliding window in pieces, then single tokens follow, and the samples of one prompt share it."""
import pytest
import torch

import kv_chunk_selection_b200 as lsa
from pool_testlib import assert_close, attend, i32

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from kv_chunk_selection_b200 import build
    build.build()
    lsa.lib()
    lsa.read_device_status()


def test_prompt_pieces_tokens_and_samples():
    window, sinks, slots = 150, 4, 40
    g = torch.Generator().manual_seed(3)
    freq, scale = lsa.rope_frequencies(64, 10000.0, scaling="parts", factor=4.0, original_context=256, device=DEV)
    qw, kw = (1 + 0.1 * torch.randn(128, generator=g)).to(DEV), (1 + 0.1 * torch.randn(128, generator=g)).to(DEV)
    kp, vp = (torch.full((slots, 8, 64, 128), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    free = torch.randperm(slots, generator=g).tolist()
    chunks = 8
    table = torch.full((2, chunks), -1, dtype=torch.int32)
    ws = lsa.new_window_attn_workspace(2, 64)
    held = [([], [], 0), ([], [], 0)]               # keys, values (as written) and length of each sequence
    # two sequences: a prompt in pieces of ragged lengths, then single tokens
    steps = [(64, 10), (33, 64), (1, 17), (40, 1)] + [(1, 1)] * 5
    for nqs in steps:
        T = sum(nqs)
        pos, seq = [], []
        for b, nq in enumerate(nqs):
            n = held[b][2]
            pos += list(range(n, n + nq))
            seq += [b] * nq
            for c in range((n + nq + 63) // 64):
                if table[b, c] < 0:
                    table[b, c] = free.pop()
        qkv = torch.randn((T, 80 * 128), generator=g).to(torch.bfloat16).to(DEV)
        q, k, v = (torch.empty((T, h, 128), dtype=torch.bfloat16, device=DEV) for h in (64, 8, 8))
        d_table = table.to(DEV)
        kwargs = dict(q_weight=qw, k_weight=kw, interleaved=True, rope_scale=scale)
        lsa.lsa_qk_norm_rope(qkv, i32(pos), freq, q, k, v, **kwargs)
        lsa.lsa_qk_norm_rope_pool(qkv, i32(pos), freq, q, kp, vp, d_table, i32(seq), i32(pos), chunks, **kwargs)
        at = 0
        for b, nq in enumerate(nqs):
            held[b] = (held[b][0] + [k[at: at + nq].cpu()], held[b][1] + [v[at: at + nq].cpu()], held[b][2] + nq)
            at += nq
        out = torch.empty_like(q)
        lens = [h[2] for h in held]
        lsa.lsa_window_attn(q, kp, vp, d_table, i32([0, nqs[0], T]), i32(lens), chunks, 64, window, sinks, out, ws)
        at = 0
        for b, nq in enumerate(nqs):
            p, j = torch.arange(lens[b] - nq, lens[b])[:, None], torch.arange(lens[b])[None]
            see = (j <= p) & ((j > p - window) | (j < sinks))
            assert_close(out[at: at + nq], *attend(q[at: at + nq].cpu(), torch.cat(held[b][0]), torch.cat(held[b][1]), see))
            at += nq
    # six samples of sequence 0 share its cache; each writes its own next tokens into a chunk of its own
    B, n = 6, held[0][2]
    own = torch.tensor([[free.pop()] for _ in range(B)], dtype=torch.int32)
    pws, out = lsa.new_prefix_attn_workspace(B, 1), torch.empty((B, 64, 128), dtype=torch.bfloat16, device=DEV)
    ks, vs = [], []
    for t in range(3):
        qkv = torch.randn((B, 80 * 128), generator=g).to(torch.bfloat16).to(DEV)
        q, k, v = (torch.empty((B, h, 128), dtype=torch.bfloat16, device=DEV) for h in (64, 8, 8))
        kwargs = dict(q_weight=qw, k_weight=kw, interleaved=True, rope_scale=scale)
        lsa.lsa_qk_norm_rope(qkv, i32([n + t] * B), freq, q, k, v, **kwargs)
        lsa.lsa_qk_norm_rope_pool(qkv, i32([n + t] * B), freq, q, kp, vp, own.to(DEV), i32(range(B)), i32([t] * B), 1, **kwargs)
        ks.append(k.cpu())
        vs.append(v.cpu())
        lsa.lsa_prefix_decode_attn(q, kp, vp, d_table[:1], i32([0, B]), i32([n]), own.to(DEV), i32([t + 1] * B), out, pws)
        for b in range(B):
            kk = torch.cat(held[0][0] + [x[b: b + 1] for x in ks])
            vv = torch.cat(held[0][1] + [x[b: b + 1] for x in vs])
            assert_close(out[b: b + 1], *attend(q[b: b + 1].cpu(), kk, vv, torch.ones((1, n + t + 1), dtype=torch.bool)))
    assert lsa.read_device_status() == 0
