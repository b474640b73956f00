"""The pool that lsa_qk_norm_rope_pool fills, read by the chunk path: scores, selection, gather and decode attention over
the kept chunks, each checked in 64 bits."""
import numpy as np
import pytest
import torch

import kv_chunk_selection_b200 as lsa
import oracle
from lsa_testlib import assert_attention_close, assert_kept_matches, assert_scores_close, f64
from pool_testlib import i32

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from kv_chunk_selection_b200 import build
    build.build()
    lsa.lib()
    lsa.read_device_status()


def bf16(shape, g):
    return torch.randn(shape, generator=g).to(torch.bfloat16).to(DEV)


class Serving:
    """Three sequences whose prompts went through the projection into the pool; what was written is kept for the oracle."""

    def __init__(self, lens=(640, 200, 1000), K=(4, 2, 6), seed=7):
        self.g = g = torch.Generator().manual_seed(seed)
        self.lens, self.B, self.chunks = list(lens), len(lens), 17
        self.table = torch.randperm(60, generator=g)[: self.B * self.chunks].view(self.B, self.chunks).to(torch.int32).to(DEV)
        self.kp, self.vp = (torch.zeros((60, 8, 64, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        self.freq, self.scale = lsa.rope_frequencies(128, 10000.0, device=DEV)
        self.qw, self.kw = (1 + 0.1 * torch.randn(128, generator=g)).to(DEV), (1 + 0.1 * torch.randn(128, generator=g)).to(DEV)
        for b, n in enumerate(lens):
            self.tokens([b] * n, list(range(n)))
        self.k_per_seq, self.w = i32(K), torch.rand(16, generator=g).to(DEV)
        self.keys = bf16((60, 128), g)

    def tokens(self, seq, pos):
        """One call over the projection's rows of these tokens; their rotated queries."""
        qkv = bf16((len(pos), 80 * 128), self.g)
        q, k, v = (torch.empty((len(pos), h, 128), dtype=torch.bfloat16, device=DEV) for h in (64, 8, 8))
        kwargs = dict(q_weight=self.qw, k_weight=self.kw, rope_scale=self.scale)
        lsa.lsa_qk_norm_rope(qkv, i32(pos), self.freq, q, k, v, **kwargs)
        lsa.lsa_qk_norm_rope_pool(qkv, i32(pos), self.freq, q, self.kp, self.vp, self.table, i32(seq), i32(pos), self.chunks,
                                  **kwargs)
        slots = self.table[torch.tensor(seq), torch.tensor(pos) // 64].long()
        assert torch.equal(self.kp[slots, :, torch.tensor(pos) % 64], k) and torch.equal(self.vp[slots, :, torch.tensor(pos) % 64], v)
        return q

    def window(self):
        from kv_chunk_selection_b200.window import LayerWindow
        n = i32([-(-x // 64) for x in self.lens])
        return LayerWindow(n, self.k_per_seq, self.table, self.chunks, DEV)


def test_the_chunk_path_over_the_filled_pool():
    s = Serving()
    for step in range(3):                            # a token of each sequence, then a window over what is cached
        q = s.tokens(range(s.B), s.lens)
        s.lens = [n + 1 for n in s.lens]
        lw, q_idx = s.window(), bf16((s.B, 16, 128), s.g)
        out = torch.empty((s.B, 64, 128), device=DEV)
        lw.select(q_idx, s.w, s.keys)
        lw.gather(s.kp, s.vp)
        lw.attend(q, out)
        torch.cuda.synchronize()
        assert lsa.read_device_status() == 0
        n = [-(-x // 64) for x in s.lens]
        scores = oracle.index_scores(f64(q_idx), f64(s.w), f64(s.keys), s.table.cpu().numpy(), np.array(n), s.chunks)
        assert_scores_close(lw.scores, scores, n)
        kept = lw.kept_lists()
        assert_kept_matches(kept, scores, n, s.k_per_seq.tolist())
        k, v, cu = oracle.gather_chunks(f64(s.kp), f64(s.vp), s.table.cpu().numpy(), kept, s.chunks)
        assert_attention_close(out, oracle.sparse_decode_attn(f64(q), k, v, cu))


def test_the_norms_between_a_gather_and_an_attention_that_reads_ahead():
    """The first step of a window: the gather, the step's norms and rotations, and an attention call whose keys the
    kernel just before it did not write."""
    s = Serving()
    lw, q_idx = s.window(), [bf16((s.B, 16, 128), s.g) for _ in range(2)]
    out, ref = (torch.empty((s.B, 64, 128), device=DEV) for _ in range(2))
    qkv = bf16((s.B, 80 * 128), s.g)
    q, k, v = (torch.empty((s.B, h, 128), dtype=torch.bfloat16, device=DEV) for h in (64, 8, 8))
    ws = lsa.new_attn_workspace(s.B)
    refs = []
    for i in range(2):
        lw.select(q_idx[i], s.w, s.keys)
        lw.gather(s.kp, s.vp)
        lsa.lsa_qk_norm_rope(qkv, i32(s.lens), s.freq, q, k, v, q_weight=s.qw, k_weight=s.kw)
        lsa.lsa_sparse_decode_attn(q, lw.k_bufs[0], lw.v_bufs[0], lw.cu_kept[0], ref, ws)
        refs.append(ref.clone())
    assert not torch.equal(refs[0], refs[1])
    pos = i32(s.lens)
    for i in range(40):
        lw.select(q_idx[i % 2], s.w, s.keys)
        lw.gather(s.kp, s.vp)
        lsa.lsa_qk_norm_rope(qkv, pos, s.freq, q, k, v, q_weight=s.qw, k_weight=s.kw)
        lsa.lsa_sparse_decode_attn(q, lw.k_bufs[0], lw.v_bufs[0], lw.cu_kept[0], out, ws, kv_unchanged=True)
        assert torch.equal(out, refs[i % 2])
    assert lsa.read_device_status() == 0
