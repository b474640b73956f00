"""Head norms with rotary positions against the formula in 64 bits.

Tolerance, from the kernel's arithmetic: the result is rounded once to bf16
(2^-8 relative), and before that a rotated value is a cos - b sin in fp32 with
a, b within 12 roundings of 2^-24 (the sum of squares halved by the root,
rsqrtf's two units, two products), cos and sin within 5, 8 more for an angle
near 2^31 (two roundings of its turns in fp64: 4.4e-7) and 3 for the products
and their sum: 28 * 2^-24 = 1.7e-6 of scale * (|a| + |b|).
"""
import numpy as np
import pytest
import torch

import kv_chunk_selection_b200 as lsa

pytestmark = pytest.mark.gpu
DEV = "cuda"
WIDTH = 80 * 128
BAD_COUNT, BAD_SLOT, BAD_CHUNK = 1, 2, 4


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from kv_chunk_selection_b200 import build
    build.build()
    lsa.lib()
    lsa.read_device_status()


def pairs(rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def reference(x, w, eps, pos, freq, scale, interleaved):
    """x [T, heads, 128] fp64 -> (result, bound on the error before and with the rounding)."""
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w if w is not None else x.copy()
    out, mag = y.copy(), np.abs(y)
    if freq is not None:
        a, b = pairs(2 * len(freq), interleaved)
        ang = pos[:, None].astype(np.float64) * freq.astype(np.float64)
        c, s = scale * np.cos(ang)[:, None], scale * np.sin(ang)[:, None]
        out[..., a], out[..., b] = y[..., a] * c - y[..., b] * s, y[..., b] * c + y[..., a] * s
        m = abs(scale) * (np.abs(y[..., a]) + np.abs(y[..., b]))
        mag[..., a], mag[..., b] = m, m
    return out, 2.0 ** -8 * np.abs(out) + 1.7e-6 * mag


def n64(t):
    return t.detach().cpu().double().numpy()


def draw(T, rot, norm, pad=0, seed=0, far=1 << 20):
    g = torch.Generator(device=DEV).manual_seed(seed)
    qkv = torch.randn((T, WIDTH + pad), generator=g, device=DEV).to(torch.bfloat16)[:, :WIDTH]
    pos = torch.randint(0, far, (T,), generator=g, device=DEV, dtype=torch.int32)
    freq = lsa.rope_frequencies(rot, 500000.0, device=DEV)[0] if rot else None
    w = [1 + 0.2 * torch.randn(128, generator=g, device=DEV) if norm else None for _ in range(2)]
    return qkv, pos, freq, w[0], w[1]


def outputs(T):
    e = lambda n: torch.full((T, n, 128), float("nan"), dtype=torch.bfloat16, device=DEV)  # noqa: E731
    return e(64), e(8), e(8)


def check(qkv, pos, freq, wq, wk, scale, inter, q, k, v, eps=1e-6):
    x = n64(qkv).reshape(-1, 80, 128)
    f, p = None if freq is None else freq.cpu().numpy(), pos.cpu().numpy()
    for got, part, w in ((q, x[:, :64], wq), (k, x[:, 64:72], wk)):
        ref, bound = reference(part, None if w is None else n64(w), eps, p, f, scale, inter)
        err = np.abs(n64(got) - ref)
        assert np.all(err <= bound), f"off by {np.max(err / bound)} of the bound"
    if v is not None:
        assert torch.equal(v.cpu(), qkv.cpu().reshape(-1, 80, 128)[:, 72:])


@pytest.mark.parametrize("T", [1, 3, 130])
@pytest.mark.parametrize("rot,inter,norm,pad,scale", [
    (128, False, True, 0, 1.0), (128, True, True, 8, 1.0), (64, False, True, 64, 1.25), (64, True, False, 0, 1.0),
    (24, False, True, 0, 1.0), (8, False, False, 0, 0.5), (8, True, True, 0, 1.0), (120, False, True, 0, 1.0),
    (0, False, True, 0, 1.0), (0, True, False, 0, 1.0)])
def test_dense_form(T, rot, inter, norm, pad, scale):
    qkv, pos, freq, wq, wk = draw(T, rot, norm, pad, seed=rot + T)
    q, k, v = outputs(T)
    lsa.lsa_qk_norm_rope(qkv, pos, freq, q, k, v, q_weight=wq, k_weight=wk, interleaved=inter, rope_scale=scale)
    check(qkv, pos, freq, wq, wk, scale, inter, q, k, v)
    assert lsa.read_device_status() == 0


def test_far_and_first_positions_keep_their_phase():
    qkv, _, freq, wq, wk = draw(6, 128, True, seed=5)
    pos = torch.tensor([0, 1, 1 << 20, (1 << 24) + 1, (1 << 31) - 1, 12345677], dtype=torch.int32, device=DEV)
    q, k, v = outputs(6)
    lsa.lsa_qk_norm_rope(qkv, pos, freq, q, k, v, q_weight=wq, k_weight=wk)
    check(qkv, pos, freq, wq, wk, 1.0, False, q, k, v)


def test_one_norm_only_and_no_value_heads():
    qkv, pos, freq, wq, _ = draw(7, 64, True, seed=6)
    q, k, v = outputs(7)
    lsa.lsa_qk_norm_rope(qkv, pos, freq, q, k, None, q_weight=wq, eps=1e-2)
    check(qkv, pos, freq, wq, None, 1.0, False, q, k, None, eps=1e-2)
    q2, k2, v2 = outputs(7)
    lsa.lsa_qk_norm_rope(qkv, pos, freq, q2, k2, v2, k_weight=wq)
    check(qkv, pos, freq, None, wq, 1.0, False, q2, k2, v2)


def test_zero_rows_and_wide_values():
    qkv, pos, freq, wq, wk = draw(4, 128, True, seed=7)
    qkv[0] = 0
    qkv[1] *= 1e15
    qkv[2] *= 1e-15
    q, k, v = outputs(4)
    lsa.lsa_qk_norm_rope(qkv, pos, freq, q, k, v, q_weight=wq, k_weight=wk)
    check(qkv, pos, freq, wq, wk, 1.0, False, q, k, v)
    assert torch.all(q[0] == 0) and torch.all(k[0] == 0)


def pool_case(T, B, max_chunks, seed):
    g = torch.Generator().manual_seed(seed)
    n_slots = B * max_chunks + 3
    table = torch.randperm(n_slots, generator=g)[: B * max_chunks].view(B, max_chunks).to(torch.int32)
    rows = torch.randperm(B * max_chunks * 64, generator=g)[:T]
    seq, cpos = (rows // (max_chunks * 64)).to(torch.int32), (rows % (max_chunks * 64)).to(torch.int32)
    return n_slots, table, seq, cpos


@pytest.mark.parametrize("T,inter,identity", [(1, False, False), (33, True, False), (200, False, True)])
def test_pool_form_writes_its_rows_and_no_others(T, inter, identity):
    qkv, pos, freq, wq, wk = draw(T, 64, True, seed=T)
    n_slots, table, seq, cpos = pool_case(T, 5, 3, T)
    if identity:
        table, n_slots = torch.arange(15, dtype=torch.int32).view(5, 3), 15
    cpos[T // 2] = -1 if T > 1 else cpos[0]   # padding
    kp, vp = (torch.full((n_slots, 8, 64, 128), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    q, k, v = outputs(T)
    lsa.lsa_qk_norm_rope(qkv, pos, freq, q, k, v, q_weight=wq, k_weight=wk, interleaved=inter)
    q2 = torch.empty_like(q)
    lsa.lsa_qk_norm_rope_pool(qkv, pos, freq, q2, kp, vp, None if identity else table.to(DEV), seq.to(DEV),
                              cpos.to(DEV), 3, q_weight=wq, k_weight=wk, interleaved=inter)
    assert lsa.read_device_status() == 0
    check(qkv, pos, freq, wq, wk, 1.0, inter, q, k, v)
    assert torch.equal(q, q2)
    want_k, want_v = (torch.full((n_slots, 8, 64, 128), 7.0, dtype=torch.bfloat16) for _ in range(2))
    for t in range(T):
        if cpos[t] >= 0:
            s, r = int(table[seq[t], cpos[t] // 64]), int(cpos[t] % 64)
            want_k[s, :, r], want_v[s, :, r] = k[t].cpu(), v[t].cpu()
    assert torch.equal(kp.cpu(), want_k) and torch.equal(vp.cpu(), want_v)


@pytest.mark.parametrize("what,bit", [("seq_low", BAD_COUNT), ("seq_high", BAD_COUNT), ("chunk", BAD_CHUNK),
                                      ("slot", BAD_SLOT), ("slot_high", BAD_SLOT)])
def test_bad_places_are_reported_and_not_written(what, bit):
    T = 4
    qkv, pos, freq, wq, wk = draw(T, 128, True, seed=1)
    n_slots, table, seq, cpos = pool_case(T, 2, 2, 3)
    seq[:], cpos[:] = torch.tensor([0, 0, 1, 1], dtype=torch.int32), torch.tensor([0, 64, 0, 64], dtype=torch.int32)
    if what == "seq_low":
        seq[1] = -1
    elif what == "seq_high":
        seq[1] = 2
    elif what == "chunk":
        cpos[1] = 128
    else:
        table[0, 1] = -1 if what == "slot" else n_slots
    kp, vp = (torch.zeros((n_slots, 8, 64, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    q, k, v = outputs(T)
    lsa.lsa_qk_norm_rope_pool(qkv, pos, freq, q, kp, vp, table.to(DEV), seq.to(DEV), cpos.to(DEV), 2, q_weight=wq,
                              k_weight=wk)
    assert lsa.read_device_status() == bit
    lsa.lsa_qk_norm_rope(qkv, pos, freq, torch.empty_like(q), k, v, q_weight=wq, k_weight=wk)
    check(qkv, pos, freq, wq, wk, 1.0, False, q, k, v)
    assert int((vp != 0).any(-1).sum()) == 3 * 8    # three tokens' rows, none of the fourth's
    for t in (0, 2, 3):
        s = int(table[seq[t], cpos[t] // 64])
        assert torch.equal(kp[s, :, int(cpos[t] % 64)], k[t]) and torch.equal(vp[s, :, int(cpos[t] % 64)], v[t])


def test_captured_and_on_another_stream():
    qkv, pos, freq, wq, wk = draw(9, 128, True, seed=11)
    q, k, v = outputs(9)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    lsa.lsa_qk_norm_rope(qkv, pos, freq, q, k, v, q_weight=wq, k_weight=wk, stream=s)
    s.synchronize()
    check(qkv, pos, freq, wq, wk, 1.0, False, q, k, v)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lsa.lsa_qk_norm_rope(qkv, pos, freq, q, k, v, q_weight=wq, k_weight=wk)
    qkv.copy_(torch.randn_like(qkv, dtype=torch.float32).to(torch.bfloat16))
    g.replay()
    torch.cuda.synchronize()
    check(qkv, pos, freq, wq, wk, 1.0, False, q, k, v)


def test_the_rows_feed_the_fused_append():
    """k_out and v_out of one step are the fused append's k_new and v_new."""
    B = 3
    qkv, pos, freq, wq, wk = draw(B, 128, True, seed=13)
    q, k, v = outputs(B)
    kl, vl = (torch.zeros((B, 8, 64, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    n0, n1 = (torch.zeros(B, dtype=torch.int32, device=DEV) for _ in range(2))
    buf = torch.zeros((8, 1, 64, 128), dtype=torch.bfloat16, device=DEV)
    cu = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    out = torch.empty((B, 64, 128), device=DEV)
    lsa.lsa_qk_norm_rope(qkv, pos, freq, q, k, v, q_weight=wq, k_weight=wk)
    lsa.lsa_sparse_decode_attn_append(q, buf, buf, cu, k, v, kl, vl, n0, n1, out, lsa.new_attn_workspace(B))
    torch.cuda.synchronize()
    assert n1.tolist() == [1] * B and torch.equal(kl[:, :, 0], k)
    # one token: its value head is the answer of each of its 8 query heads
    assert torch.allclose(out.view(B, 8, 8, 128), v.float()[:, :, None].expand(B, 8, 8, 128), rtol=2 ** -15, atol=0)
