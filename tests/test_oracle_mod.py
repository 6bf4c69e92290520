"""Pins of the oracle's score modifications and compaction (no GPU): a scalar textbook loop, the
plain oracle where nothing is modified, library attention with an additive mask, and moves
written out by hand."""
import math

import numpy as np
import pytest
import torch

import workloads as wl
from oracle import rcp_oracle as orc

TINY = wl.SHAPES["tiny"]


def test_visible_tokens_by_hand():
    see = orc.visible_tokens
    assert list(np.nonzero(see(5, 8))[0]) == [0, 1, 2, 3, 4, 5]
    assert list(np.nonzero(see(5, 8, window=2))[0]) == [4, 5]
    assert list(np.nonzero(see(5, 8, window=2, prefix=1))[0]) == [0, 4, 5]
    assert list(np.nonzero(see(1, 8, prefix=4))[0]) == [0, 1, 2, 3]       # later ones of the prefix
    assert list(np.nonzero(see(5, 8, begin=3))[0]) == [3, 4, 5]
    assert list(np.nonzero(see(5, 8, begin=3, window=5))[0]) == [3, 4, 5]
    assert not see(5, 8, begin=6).any()
    assert see(5, 8, prefix=99).all()


def test_nothing_modified_is_the_plain_oracle():
    inp = wl.make_prefill_inputs(TINY, [37, 0], [21, 16], seed=5)
    c = inp.cache
    kp, vp = orc.append_kv(c.k_pages, c.v_pages, inp.U_k, inp.W_v, inp.k, inp.v, inp.slot_mapping)
    args = (inp.q, inp.cu_chunk_lens, kp, vp, inp.U_k, inp.W_v, c.block_table, inp.seq_lens_after)
    np.testing.assert_allclose(orc.prefill_attn_mod(*args), orc.prefill_attn(*args), rtol=0,
                               atol=1e-13)


def test_scalar_loop():
    """One head and row at a time, in python floats."""
    inp = wl.make_decode_inputs(TINY, [41, 30], seed=6)
    c = inp.cache
    slopes = [0.5, 0.25, 0.0, 0.01]
    mod = dict(softcap=0.7, alibi_slopes=slopes, window=9, prefix_lens=[3, 40], row_begin=[35, 25])
    got = orc.decode_attn_mod(inp.q, c.k_pages, c.v_pages, inp.U_k, inp.W_v, c.block_table,
                              c.seq_lens, **mod)
    H, d, rk, R = (TINY[k] for k in ("num_heads", "head_dim", "rank_k", "rank_v"))
    for b, L in enumerate([41, 30]):
        pos = L - 1
        ts = [t for t in range(L) if t < mod["prefix_lens"][b]
              or (mod["row_begin"][b] <= t <= pos and t > pos - 9)]
        for h in range(H):
            K = inp.cache.ck[b][:, h].astype(float) @ inp.U_k[h].astype(float)   # explicit keys
            V = inp.cache.cv[b].astype(float) @ inp.W_v.astype(float)[:, h * d:(h + 1) * d]
            s = {}
            for t in ts:
                x = sum(float(a) * float(k) for a, k in zip(inp.q[b, h], K[t])) / math.sqrt(d)
                s[t] = 0.7 * math.tanh(x / 0.7) - slopes[h] * abs(pos - t)
            den = sum(math.exp(x) for x in s.values())
            want = sum(math.exp(x) / den * V[t] for t, x in s.items())
            np.testing.assert_allclose(got[b, h], want, rtol=0, atol=1e-9)


def test_library_attention_with_an_additive_mask():
    inp = wl.make_prefill_inputs(TINY, [20], [30], seed=7)
    c = inp.cache
    kp, vp = orc.append_kv(c.k_pages, c.v_pages, inp.U_k, inp.W_v, inp.k, inp.v, inp.slot_mapping)
    H, d = TINY["num_heads"], TINY["head_dim"]
    begin = np.where(np.arange(30) < 12, 15, 32).astype(np.int32)
    mod = dict(alibi_slopes=[0.1, 0.2, 0.3, 0.4], window=25, prefix_lens=[4], row_begin=begin)
    got = orc.prefill_attn_mod(inp.q, inp.cu_chunk_lens, kp, vp, inp.U_k, inp.W_v, c.block_table,
                               [50], **mod)
    ck, cv = orc.gather_request(kp, vp, c.block_table[0], 50, 16)
    K = np.einsum("thk,hkd->htd", ck, inp.U_k.astype(float))
    V = (cv @ inp.W_v.astype(float)).reshape(50, H, d).transpose(1, 0, 2)
    mask = np.full((H, 30, 50), -np.inf)
    for i in range(30):
        for t in range(50):
            if t < 4 or (begin[i] <= t <= 20 + i and t > 20 + i - 25):
                mask[:, i, t] = [-0.1 * (h + 1) * abs(20 + i - t) for h in range(H)]
    want = torch.nn.functional.scaled_dot_product_attention(
        torch.tensor(inp.q.astype(float)).transpose(0, 1), torch.tensor(K), torch.tensor(V),
        attn_mask=torch.tensor(mask)).transpose(0, 1).numpy()
    np.testing.assert_allclose(got, want, rtol=0, atol=1e-11)


def test_rows_that_see_nothing_are_zero_and_hidden_tokens_take_no_part():
    inp = wl.make_decode_inputs(TINY, [40, 40], seed=8)
    c = inp.cache
    mod = dict(window=8, row_begin=[0, 40])
    a = orc.decode_attn_mod(inp.q, c.k_pages, c.v_pages, inp.U_k, inp.W_v, c.block_table,
                            c.seq_lens, **mod)
    assert np.all(a[1] == 0) and np.any(a[0] != 0)
    kp, vp = c.k_pages.copy(), c.v_pages.copy()
    for t in range(32):                                   # hidden by the window
        kp[c.block_table[0, t // 16], :, t % 16] = np.nan
        vp[c.block_table[0, t // 16], t % 16] = np.nan
    with np.errstate(invalid="ignore"):
        b = orc.decode_attn_mod(inp.q, kp, vp, inp.U_k, inp.W_v, c.block_table, c.seq_lens, **mod)
    assert np.array_equal(a, b)


@pytest.mark.parametrize("pages", ["fp16", "int4"])
def test_compaction_by_hand(pages):
    inp = wl.make_decode_inputs(TINY, [20], seed=9)
    c = inp.cache
    kp, vp = c.k_pages, c.v_pages
    if pages == "int4":
        kp, vp = orc.int4_pack_pages(*orc.int4_pages(kp, vp))
    keep = np.zeros((1, 32), np.uint8)
    keep[0, [0, 3, 17, 19, 25]] = 1                       # 25 is past the end
    k, v, lens = orc.compact_tokens(kp, vp, pages, TINY, c.block_table, c.seq_lens, keep)
    assert list(lens) == [4]

    def token(kk, vv, t):
        if pages == "int4":
            kk, vv = orc.int4_page_coefficients(kk, vv, 4, 16, 64)
        ck, cv = orc.gather_request(kk, vv, c.block_table[0], 20, 16)
        return np.concatenate([ck[t].ravel(), cv[t]])
    for j, t in enumerate([0, 3, 17, 19]):
        assert np.array_equal(token(k, v, j), token(kp, vp, t))
    for t in range(4, 20):
        assert np.array_equal(token(k, v, t), token(kp, vp, t))


@pytest.mark.parametrize("slope", [-2.0 ** 60, -2.0 ** 53])
def test_scores_decide_between_tokens_at_the_same_distance(slope):
    """A row in the middle of a prefix whose bias leaves its two farthest tokens alone: their
    weights are those of their scores, whatever the bias is."""
    inp = wl.make_decode_inputs(TINY, [7], seed=10)
    c = inp.cache
    ck, cv = orc.gather_request(c.k_pages, c.v_pages, c.block_table[0], 7, 16)
    see = orc.visible_tokens(3, 7, prefix=7)[None]
    H = inp.q.shape[1]
    _, p = orc.attend_mod(inp.q, ck, cv, inp.U_k, inp.W_v, inp.q.shape[2], [3], see, 0.0, [slope] * H)
    for h in range(H):
        qt = inp.q[0, h].astype(np.float64) @ np.asarray(inp.U_k[h], np.float64).T
        s = [float(qt @ np.asarray(ck[t, h], np.float64)) / math.sqrt(inp.q.shape[2]) for t in (0, 6)]
        first = 1 / (1 + math.exp(s[1] - s[0]))
        np.testing.assert_allclose(p[0, h], [first, 0, 0, 0, 0, 0, 1 - first], rtol=0, atol=1e-12)
        assert abs(first - 0.5) > 1e-3
