"""Score-modified decode and chunked prefill vs the fp64 oracle, through the C ABI (needs a
GB300): capped scores, distance bias, windows, prefixes and document masks on every page
format and both shapes."""
import numpy as np
import pytest

import workloads as wl
from oracle import rcp_oracle as orc
from tests.mod_util import assert_within, cache_of, encode, score_mod, values
from tests.gpu_util import t

pytestmark = pytest.mark.gpu

SHAPES = {"tiny": wl.SHAPES["tiny"], "main": wl.SHAPES["mha32"]}
FORMATS = ["fp16", "fp8_e4m3", "int4"]
LENS = [0, 1, 15, 16, 17, 33, 200, 256, 385, 500]


def slopes_of(shape):
    H = shape["num_heads"]
    return [2.0 ** (-8 * (h + 1) / H) for h in range(H)]


def decode_mods(shape, lens):
    L = np.asarray(lens)
    return {
        "cap": dict(softcap=5.0),
        "bias": dict(alibi_slopes=slopes_of(shape)),
        "window": dict(window=23),
        "window1": dict(window=1),
        "sinks": dict(window=40, prefix_lens=np.minimum(L, 5)),
        "prefix": dict(prefix_lens=np.full(len(L), 35), row_begin=L),     # the prefix alone
        "hole": dict(prefix_lens=np.full(len(L), 3), row_begin=np.full(len(L), 9)),
        "docs": dict(row_begin=L * 2 // 3, softcap=20.0),
        "empty": dict(row_begin=L + 1),
        "odd": dict(prefix_lens=np.array([-4, 2 ** 31 - 1] * (len(L) // 2)),
                    row_begin=np.array([2 ** 31 - 1, -7] * (len(L) // 2))),
        "all": dict(softcap=3.0, alibi_slopes=slopes_of(shape), window=100,
                    prefix_lens=np.full(len(L), 18), row_begin=L // 2),
    }


_decode_cache = {}


def decode_inputs(shape_name, pages, lens=LENS, seed=301, scale=4.0):
    key = (shape_name, pages, tuple(lens), seed)
    if key not in _decode_cache:
        shape = SHAPES[shape_name]
        inp = wl.make_decode_inputs(shape, lens, seed=seed, fill=np.nan if pages == "fp16" else 0.0)
        inp.q = wl.fp16(inp.q.astype(np.float64) * scale)
        inp.k, inp.v = encode(pages, inp.cache.k_pages, inp.cache.v_pages)
        _decode_cache[key] = inp
    return _decode_cache[key]


def oracle_decode(inp, pages, mod, k=None, v=None):
    kk, vv = values(pages, inp.shape, inp.k if k is None else k, inp.v if v is None else v, False)
    ref = orc.decode_attn_mod(inp.q, kk, vv, inp.U_k, inp.W_v, inp.cache.block_table,
                              inp.cache.seq_lens, magnitudes=True, **mod)
    return (*ref, int(max(inp.cache.seq_lens)))


@pytest.mark.parametrize("name", sorted(decode_mods(SHAPES["tiny"], LENS)))
@pytest.mark.parametrize("pages", FORMATS)
@pytest.mark.parametrize("shape_name", ["tiny", "main"])
def test_decode_matches_oracle(shape_name, pages, name):
    import torch
    inp = decode_inputs(shape_name, pages)
    mod = decode_mods(inp.shape, LENS)[name]
    cache = cache_of(pages, inp.shape, inp.U_k, inp.W_v, inp.k, inp.v)
    out = cache.decode_attn(t(inp.q), t(inp.cache.block_table), t(inp.cache.seq_lens),
                            mod=score_mod(mod))
    torch.cuda.synchronize()
    assert cache.read_device_error() == 0
    assert_within(out.cpu().numpy(), oracle_decode(inp, pages, mod), f"{shape_name} {pages} {name}")


@pytest.mark.parametrize("pages", FORMATS)
@pytest.mark.parametrize("shape_name", ["tiny", "main"])
def test_decode_without_effective_modifications_is_the_plain_decode(shape_name, pages):
    """No modification is the plain call, bit for bit.  Masks that hide nothing and a zero bias
    give the same attention with its weights rounded in another scale (pages are met in the
    other order, so the running maximum is another one): within the bound of the exact
    result, like the plain call."""
    inp = decode_inputs(shape_name, pages)
    cache = cache_of(pages, inp.shape, inp.U_k, inp.W_v, inp.k, inp.v)
    args = t(inp.q), t(inp.cache.block_table), t(inp.cache.seq_lens)
    plain = cache.decode_attn(*args).cpu().numpy()
    got = cache.decode_attn(*args, mod=score_mod({})).cpu().numpy()
    assert np.array_equal(plain.view(np.uint16), got.view(np.uint16))
    ref = oracle_decode(inp, pages, {})
    assert_within(plain, ref, "plain")
    B, H = len(LENS), inp.shape["num_heads"]
    for mod in (dict(window=500), dict(row_begin=np.zeros(B)), dict(alibi_slopes=np.zeros(H)),
                dict(prefix_lens=np.full(B, 600))):
        got = cache.decode_attn(*args, mod=score_mod(mod)).cpu().numpy()
        assert_within(got, ref, str(mod))


@pytest.mark.parametrize("pages", FORMATS)
@pytest.mark.parametrize("mod", [dict(window=4100, prefix_lens=[70]),
                                 dict(row_begin=[3000], softcap=30.0),
                                 dict(softcap=50.0)])
def test_decode_of_one_long_request(pages, mod):
    """One request over many partitions: partial records of the visible pages only."""
    import torch
    inp = decode_inputs("main", pages, lens=[7003], seed=302)
    cache = cache_of(pages, inp.shape, inp.U_k, inp.W_v, inp.k, inp.v)
    out = cache.decode_attn(t(inp.q), t(inp.cache.block_table), t(inp.cache.seq_lens),
                            mod=score_mod(mod))
    torch.cuda.synchronize()
    assert cache.read_device_error() == 0
    assert_within(out.cpu().numpy(), oracle_decode(inp, pages, mod), f"long {pages} {mod}")


def hide(inp, pages, k, v, b, tokens):
    """Fills the slots of tokens with the worst bytes the format has: NaN (fp16, E4M3), NaN
    scales and codes of -8 (4-bit)."""
    H, rk, R = (inp.shape[x] for x in ("num_heads", "rank_k", "rank_v"))
    for tok in tokens:
        blk, off = inp.cache.block_table[b, tok // 16], tok % 16
        if pages == "int4":
            kc, vc = H * 16 * rk // 2, 16 * R // 2
            for h in range(H):
                row = h * 16 + off
                k[blk, row * rk // 2:(row + 1) * rk // 2] = 0x88
                k[blk, kc + 2 * row:kc + 2 * row + 2] = (0x00, 0x7E)
            v[blk, off * R // 2:(off + 1) * R // 2] = 0x88
            n = R // 64 * 2
            v[blk, vc + off * n:vc + (off + 1) * n] = np.tile(np.uint8([0x00, 0x7E]), R // 64)
        else:
            k[blk, :, off] = np.nan if pages == "fp16" else 0x7F
            v[blk, off] = np.nan if pages == "fp16" else 0x7F


@pytest.mark.parametrize("pages", FORMATS)
@pytest.mark.parametrize("shape_name", ["tiny", "main"])
def test_decode_hidden_tokens_may_hold_anything_and_their_pages_may_be_gone(shape_name, pages):
    import torch
    lens = [300, 301, 90]
    inp = decode_inputs(shape_name, pages, lens=lens, seed=303)
    mod = dict(window=50, prefix_lens=[21, 0, 21], row_begin=[0, 280, 60], softcap=9.0)
    seen = [orc.visible_tokens(L - 1, L, mod["prefix_lens"][b], mod["row_begin"][b], 50)
            for b, L in enumerate(lens)]
    k, v = inp.k.copy(), inp.v.copy()
    table = inp.cache.block_table.copy()
    for b, L in enumerate(lens):
        hide(inp, pages, k, v, b, np.nonzero(~seen[b])[0])
        for j in range((L + 15) // 16):
            if not seen[b][16 * j:16 * j + 16].any():
                table[b, j] = (-5, 1 << 30)[j % 2]         # freed: the entry is not looked at
    cache = cache_of(pages, inp.shape, inp.U_k, inp.W_v, k, v)
    out = cache.decode_attn(t(inp.q), t(table), t(inp.cache.seq_lens), mod=score_mod(mod))
    torch.cuda.synchronize()
    assert cache.read_device_error() == 0
    assert_within(out.cpu().numpy(), oracle_decode(inp, pages, mod), f"hidden {pages}")


def test_decode_bad_block_among_the_visible_pages_is_reported_and_left_out():
    import torch
    from rank_compressed_paged_gb300 import _lib
    inp = decode_inputs("main", "fp16", lens=[200, 200], seed=304)
    mod = dict(window=100, softcap=9.0)
    table = inp.cache.block_table.copy()
    table[1, 9] = inp.k.shape[0] + 3
    cache = cache_of("fp16", inp.shape, inp.U_k, inp.W_v, inp.k, inp.v)
    out = cache.decode_attn(t(inp.q), t(table), t(inp.cache.seq_lens), mod=score_mod(mod))
    torch.cuda.synchronize()
    assert cache.read_device_error() == _lib.RCP_DEVERR_BAD_BLOCK
    see = orc.visible_tokens(199, 200, window=100)
    see[144:160] = False
    ck, cv = orc.gather_request(inp.k, inp.v, inp.cache.block_table[1], 200, 16)
    want, _ = orc.attend_mod(inp.q[1:2], ck, cv, inp.U_k, inp.W_v, 128, [199], see[None], 9.0)
    ref = oracle_decode(inp, "fp16", mod)
    got = out.cpu().numpy()
    assert_within(got[:1], (ref[0][:1], ref[1][:1], ref[2][:1], 200), "unaffected request")
    np.testing.assert_allclose(got[1], want[0], rtol=0, atol=2e-3)


def test_decode_bad_lengths_give_zeros():
    import torch
    from rank_compressed_paged_gb300 import _lib
    inp = decode_inputs("tiny", "fp16", lens=[40, 40, 40], seed=305)
    cache = cache_of("fp16", inp.shape, inp.U_k, inp.W_v, inp.k, inp.v)
    lens = np.array([-3, 40, 49], np.int32)          # 3 table columns: 48 tokens
    out = cache.decode_attn(t(inp.q), t(inp.cache.block_table), t(lens),
                            mod=score_mod(dict(window=7, prefix_lens=[9, 9, 9])))
    torch.cuda.synchronize()
    assert cache.read_device_error() == _lib.RCP_DEVERR_BAD_LEN
    o = out.cpu().numpy()
    assert np.all(o[0] == 0) and np.all(o[2] == 0) and np.any(o[1] != 0)


@pytest.mark.parametrize("pages", FORMATS)
def test_decode_step_appends_first(pages):
    """The step's own token is the newest visible one; in a graph, with the masks rewritten
    between replays."""
    import torch
    lens = [100, 17, 16, 1]
    shape = SHAPES["main"]
    inp = wl.make_decode_inputs(shape, lens, seed=306, append=True)
    k0, v0 = encode(pages, inp.cache.k_pages, inp.cache.v_pages)
    cache = cache_of(pages, shape, inp.U_k, inp.W_v, k0, v0)
    mods = [dict(softcap=7.0, window=20, row_begin=[0, 0, 3, 0], prefix_lens=[4, 0, 0, 1]),
            dict(softcap=7.0, window=20, row_begin=[90, 17, 0, 0], prefix_lens=[0, 2, 5, 0])]
    dev = score_mod(mods[0])
    k, v, sl, q = t(inp.new_k), t(inp.new_v), t(inp.slot_mapping), t(inp.q)
    table, sq = t(inp.cache.block_table), t(inp.cache.seq_lens)
    ws = cache.workspace(len(lens))
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cache.decode_step(k, v, sl, q, table, sq, out=out, workspace=ws, mod=dev)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.decode_step(k, v, sl, q, table, sq, out=out, workspace=ws, mod=dev)
    for mod in mods:
        dev.row_begin.copy_(t(np.asarray(mod["row_begin"], np.int32)))
        dev.prefix_lens.copy_(t(np.asarray(mod["prefix_lens"], np.int32)))
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert cache.read_device_error() == 0
        kk, vv = values(pages, shape, cache.k_pages.cpu().numpy(), cache.v_pages.cpu().numpy(), False)
        ref = orc.decode_attn_mod(inp.q, kk, vv, inp.U_k, inp.W_v, inp.cache.block_table,
                                  inp.cache.seq_lens, magnitudes=True, **mod)
        assert_within(out.cpu().numpy(), (*ref, 100), f"step {pages}")
    # the append wrote the same pages as the plain step's
    other = cache_of(pages, shape, inp.U_k, inp.W_v, k0, v0)
    other.append_kv(k, v, sl)
    assert torch.equal(cache.k_pages.view(torch.uint8), other.k_pages.view(torch.uint8))
    assert torch.equal(cache.v_pages.view(torch.uint8), other.v_pages.view(torch.uint8))


# ------------------------------------------------------------------------------- prefill
PRIOR, CHUNK = [0, 37, 300, 5, 130, 17], [40, 21, 150, 0, 1, 290]


def doc_begin(rows, prior, chunk, size):
    """Start of the document (every ``size`` tokens) that each chunk row belongs to."""
    return np.concatenate([(p + np.arange(c)) // size * size for p, c in zip(prior, chunk)])


def prefill_mods(shape):
    rows = sum(CHUNK)
    B = len(PRIOR)
    rng = np.random.default_rng(1)
    pos = np.concatenate([p + np.arange(c) for p, c in zip(PRIOR, CHUNK)])
    pad = np.where(rng.random(rows) < 0.3, 2 ** 31 - 1, 0)
    return {
        "cap": dict(softcap=5.0),
        "bias": dict(alibi_slopes=slopes_of(shape)),
        "window": dict(window=60),
        "window1": dict(window=1),
        "sinks": dict(window=33, prefix_lens=np.full(B, 4)),
        "prefix_lm": dict(prefix_lens=np.array([25, 50, 400, 0, 2 ** 31 - 1, 150])),
        "prefix_bias": dict(prefix_lens=np.full(B, 140), alibi_slopes=slopes_of(shape), window=3),
        "prefix_only": dict(prefix_lens=np.full(B, 10), row_begin=pos + 1,
                            alibi_slopes=slopes_of(shape)),
        "docs": dict(row_begin=doc_begin(rows, PRIOR, CHUNK, 29)),
        "docs_long": dict(row_begin=doc_begin(rows, PRIOR, CHUNK, 171), softcap=20.0),
        "empty_rows": dict(row_begin=pad),
        "empty": dict(row_begin=pos + 1),
        "self_only": dict(row_begin=pos),
        "all": dict(softcap=3.0, alibi_slopes=slopes_of(shape), window=100,
                    prefix_lens=np.full(B, 18), row_begin=doc_begin(rows, PRIOR, CHUNK, 171)),
    }


_prefill_cache = {}


def prefill_inputs(shape_name, pages):
    key = (shape_name, pages)
    if key not in _prefill_cache:
        shape = SHAPES[shape_name]
        inp = wl.make_prefill_inputs(shape, PRIOR, CHUNK, seed=311,
                                     fill=np.nan if pages == "fp16" else 0.0)
        inp.q = wl.fp16(inp.q.astype(np.float64) * 4)
        # every token's coefficients as given (the append has tests of its own)
        rng = np.random.default_rng(312)
        c = inp.cache
        kp, vp = c.k_pages.copy(), c.v_pages.copy()
        for b, L in enumerate(inp.seq_lens_after):
            for j in range((int(L) + 15) // 16):
                n = min(16, int(L) - 16 * j)
                blk = c.block_table[b, j]
                kp[blk, :, :n] = wl.fp16(rng.standard_normal(kp[blk, :, :n].shape))
                vp[blk, :n] = wl.fp16(rng.standard_normal(vp[blk, :n].shape))
        inp.kp, inp.vp = encode(pages, kp, vp)
        _prefill_cache[key] = inp
    return _prefill_cache[key]


_ref_cache = {}


def oracle_prefill(inp, shape_name, pages, name, mod):
    key = (shape_name, pages, name)
    if key not in _ref_cache:
        kk, vv = values(pages, inp.shape, inp.kp, inp.vp, True)
        ref = orc.prefill_attn_mod(inp.q, inp.cu_chunk_lens, kk, vv, inp.U_k, inp.W_v,
                                   inp.cache.block_table, inp.seq_lens_after, magnitudes=True, **mod)
        _ref_cache[key] = (*ref, int(max(inp.seq_lens_after)))
    return _ref_cache[key]


CASES = [("main", "fp16", m) for m in sorted(prefill_mods(SHAPES["main"]))] + \
        [("tiny", p, m) for p in FORMATS for m in sorted(prefill_mods(SHAPES["tiny"]))] + \
        [("main", p, m) for p in ("fp8_e4m3", "int4") for m in ("all", "docs", "prefix_bias")]


@pytest.mark.parametrize("variant", ["rank", "reconstruct"])
@pytest.mark.parametrize("shape_name,pages,name", CASES)
def test_prefill_matches_oracle(shape_name, pages, name, variant):
    import torch
    inp = prefill_inputs(shape_name, pages)
    mod = prefill_mods(inp.shape)[name]
    cache = cache_of(pages, inp.shape, inp.U_k, inp.W_v, inp.kp, inp.vp)
    out = torch.full(inp.q.shape, float("nan"), dtype=torch.float16, device="cuda")
    cache.prefill_attn(t(inp.q), t(inp.cu_chunk_lens), t(inp.cache.block_table),
                       t(inp.seq_lens_after), out=out, variant=variant, mod=score_mod(mod))
    torch.cuda.synchronize()
    assert cache.read_device_error() == 0
    assert_within(out.cpu().numpy(), oracle_prefill(inp, shape_name, pages, name, mod),
                  f"{shape_name} {pages} {name} {variant}")


@pytest.mark.parametrize("variant", ["rank", "reconstruct"])
@pytest.mark.parametrize("shape_name,pages", [("main", "fp16"), ("tiny", "fp8_e4m3"), ("tiny", "int4")])
def test_prefill_without_effective_modifications_is_the_plain_prefill(shape_name, pages, variant):
    """No modification is the plain call, bit for bit.  Masks that hide nothing and a zero bias
    give the same attention with its weights rounded in another scale (key tiles are met in
    the other order, so a row's running maximum is another one): within the bound of the
    exact result, like the plain call."""
    inp = prefill_inputs(shape_name, pages)
    cache = cache_of(pages, inp.shape, inp.U_k, inp.W_v, inp.kp, inp.vp)
    args = (t(inp.q), t(inp.cu_chunk_lens), t(inp.cache.block_table), t(inp.seq_lens_after))
    plain = cache.prefill_attn(*args, variant=variant).cpu().numpy()
    got = cache.prefill_attn(*args, variant=variant, mod=score_mod({})).cpu().numpy()
    assert np.array_equal(plain.view(np.uint16), got.view(np.uint16))
    ref = oracle_prefill(inp, shape_name, pages, "plain", {})
    assert_within(plain, ref, "plain")
    rows, H = sum(CHUNK), inp.shape["num_heads"]
    for mod in (dict(window=1000), dict(row_begin=np.zeros(rows)), dict(alibi_slopes=np.zeros(H)),
                dict(prefix_lens=np.zeros(len(PRIOR)))):
        got = cache.prefill_attn(*args, variant=variant, mod=score_mod(mod)).cpu().numpy()
        assert_within(got, ref, str(mod))


@pytest.mark.parametrize("variant", ["rank", "reconstruct"])
@pytest.mark.parametrize("shape_name,pages", [("main", "fp16"), ("main", "fp8_e4m3"),
                                              ("tiny", "fp16"), ("tiny", "int4")])
def test_prefill_hidden_tokens_may_hold_anything_and_their_pages_may_be_gone(shape_name, pages,
                                                                             variant):
    """Tokens no row sees (before every window, and padding rows in the middle of the chunk)
    hold NaN; pages before every row's first token and behind the prefix are gone."""
    import torch
    inp = prefill_inputs(shape_name, pages)
    B, rows = len(PRIOR), sum(CHUNK)
    begin = np.zeros(rows, np.int64)
    at = 0
    for p, c in zip(PRIOR, CHUNK):          # document, padding, document
        for i in range(c):
            if c // 3 <= i < c // 2:
                begin[at + i] = 2 ** 31 - 1
            elif i >= c // 2:
                begin[at + i] = p + c // 2
        at += c
    mod = dict(window=45, prefix_lens=np.full(B, 19), row_begin=begin, softcap=9.0)
    k, v = inp.kp.copy(), inp.vp.copy()
    table = inp.cache.block_table.copy()
    hidden = 0
    for b in range(B):
        L, c0, c1 = int(inp.seq_lens_after[b]), inp.cu_chunk_lens[b], inp.cu_chunk_lens[b + 1]
        if c1 == c0:
            continue
        see = np.stack([orc.visible_tokens(L - (c1 - c0) + i, L, 19, begin[c0 + i], 45)
                        for i in range(c1 - c0)]).any(axis=0)
        hide(inp, pages, k, v, b, np.nonzero(~see)[0])
        hidden += int((~see).sum())
        first = np.nonzero(see[19:])[0][0] + 19 if see[19:].any() else L
        for j in range(2, first // 16):
            table[b, j] = (-5, 1 << 30)[j % 2]
    assert hidden > 100
    cache = cache_of(pages, inp.shape, inp.U_k, inp.W_v, k, v)
    out = cache.prefill_attn(t(inp.q), t(inp.cu_chunk_lens), t(table), t(inp.seq_lens_after),
                             variant=variant, mod=score_mod(mod))
    torch.cuda.synchronize()
    assert cache.read_device_error() == 0
    assert_within(out.cpu().numpy(), oracle_prefill(inp, shape_name, pages, "hidden", mod),
                  f"hidden {shape_name} {pages} {variant}")


@pytest.mark.parametrize("variant", ["rank", "reconstruct"])
def test_prefill_bad_block_is_reported_and_left_out(variant):
    import torch
    from rank_compressed_paged_gb300 import _lib
    inp = prefill_inputs("main", "fp16")
    mod = dict(window=200, softcap=9.0)
    table = inp.cache.block_table.copy()
    table[2, 20] = -1                                    # request 2: tokens 320 .. 335
    cache = cache_of("fp16", inp.shape, inp.U_k, inp.W_v, inp.kp, inp.vp)
    out = cache.prefill_attn(t(inp.q), t(inp.cu_chunk_lens), t(table), t(inp.seq_lens_after),
                             variant=variant, mod=score_mod(mod))
    torch.cuda.synchronize()
    assert cache.read_device_error() == _lib.RCP_DEVERR_BAD_BLOCK
    got = out.cpu().numpy()
    ref = oracle_prefill(inp, "main", "fp16", "bad", mod)
    c0, c1 = inp.cu_chunk_lens[2], inp.cu_chunk_lens[3]
    rest = np.r_[0:c0, c1:sum(CHUNK)]
    assert_within(got[rest], (ref[0][rest], ref[1][rest], ref[2][rest], ref[3]), "other requests")
    L, n = 450, 150
    see = np.stack([orc.visible_tokens(300 + i, L, window=200) for i in range(n)])
    see[:, 320:336] = False
    ck, cv = orc.gather_request(inp.kp, inp.vp, inp.cache.block_table[2], L, 16)
    want, _ = orc.attend_mod(inp.q[c0:c1], ck, cv, inp.U_k, inp.W_v, 128, 300 + np.arange(n), see, 9.0)
    np.testing.assert_allclose(got[c0:c1], want, rtol=0, atol=4e-3)


@pytest.mark.parametrize("variant", ["rank", "reconstruct"])
def test_prefill_step_appends_first_and_replays_on_a_side_stream(variant):
    import torch
    shape = SHAPES["main"]
    inp = wl.make_prefill_inputs(shape, [100, 3], [140, 20], seed=313)
    c = inp.cache
    cache = cache_of("fp16", shape, inp.U_k, inp.W_v, c.k_pages, c.v_pages)
    mod = dict(window=130, prefix_lens=[10, 23], softcap=6.0, alibi_slopes=slopes_of(shape))
    dev = score_mod(mod)
    args = (t(inp.k), t(inp.v), t(inp.slot_mapping), t(inp.q), t(inp.cu_chunk_lens),
            t(c.block_table), t(inp.seq_lens_after))
    ws = torch.empty(cache.reconstruct_workspace_bytes(160, 2, c.block_table.shape[1]),
                     dtype=torch.uint8, device="cuda")
    out = torch.empty_like(args[3])
    kp, vp = orc.append_kv(c.k_pages, c.v_pages, inp.U_k, inp.W_v, inp.k, inp.v, inp.slot_mapping)
    ref = (*orc.prefill_attn_mod(inp.q, inp.cu_chunk_lens, kp, vp, inp.U_k, inp.W_v, c.block_table,
                                 inp.seq_lens_after, magnitudes=True, **mod), 240)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cache.prefill_step(*args, out=out, workspace=ws, variant=variant, mod=dev)
    side.synchronize()
    # one fp16 ulp of an appended coefficient moves a value by 2^-11 of it and a score likewise
    np.testing.assert_allclose(out.cpu().numpy(), ref[0], rtol=0, atol=4e-3)
    eager = out.clone()
    out.fill_(float("nan"))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        cache.prefill_step(*args, out=out, workspace=ws, variant=variant, mod=dev)
    g.replay()
    torch.cuda.synchronize()
    assert cache.read_device_error() == 0
    assert torch.equal(eager, out)


@pytest.mark.parametrize("variant", ["rank", "reconstruct"])
@pytest.mark.parametrize("shape_name,pages,B", [("tiny", "fp16", 90), ("tiny", "int4", 90),
                                                ("main", "fp16", 14), ("main", "fp8_e4m3", 14)])
def test_prefill_of_many_query_tiles_some_without_keys(shape_name, pages, B, variant):
    """More (query tile, head) items than SMs; runs of requests whose rows see nothing, and
    tiles of a request that see something behind tiles that do not."""
    import torch
    shape = SHAPES[shape_name]
    rng = np.random.default_rng(341)
    prior = rng.integers(0, 300, B).tolist()
    chunk = np.where(rng.random(B) < 0.2, rng.integers(129, 400, B), rng.integers(0, 60, B)).tolist()
    inp = wl.make_prefill_inputs(shape, prior, chunk, seed=342)
    c = inp.cache
    kp = wl.fp16(rng.standard_normal(c.k_pages.shape))
    vp = wl.fp16(rng.standard_normal(c.v_pages.shape))
    inp.kp, inp.vp = encode(pages, kp, vp)
    begin = [np.full(n, 2 ** 31 - 1) if (b // 4) % 3 else (np.arange(n) + p) // 90 * 90
             for b, (p, n) in enumerate(zip(prior, chunk))]
    for b in range(0, B, 12):
        begin[b][:128] = 2 ** 31 - 1
    mod = dict(softcap=8.0, row_begin=np.concatenate(begin))
    kk, vv = values(pages, shape, inp.kp, inp.vp, True)
    ref = (*orc.prefill_attn_mod(inp.q, inp.cu_chunk_lens, kk, vv, inp.U_k, inp.W_v, c.block_table,
                                 inp.seq_lens_after, magnitudes=True, **mod),
           int(max(inp.seq_lens_after)))
    cache = cache_of(pages, shape, inp.U_k, inp.W_v, inp.kp, inp.vp)
    args = (t(inp.q), t(inp.cu_chunk_lens), t(c.block_table), t(inp.seq_lens_after))
    dev = score_mod(mod)
    out = torch.full(inp.q.shape, float("nan"), dtype=torch.float16, device="cuda")
    first = None
    for _ in range(3):                  # which CTA takes an item does not show in the result
        cache.prefill_attn(*args, out=out, variant=variant, mod=dev)
        torch.cuda.synchronize()
        assert cache.read_device_error() == 0
        first = out.clone() if first is None else first
        assert torch.equal(out, first)
    assert_within(out.cpu().numpy(), ref, f"{shape_name} {pages} {variant}")


@pytest.mark.parametrize("variant", ["rank", "reconstruct"])
def test_prefill_bad_chunk_offsets_write_nothing(variant):
    import torch
    from rank_compressed_paged_gb300 import _lib
    inp = prefill_inputs("main", "fp16")
    cache = cache_of("fp16", inp.shape, inp.U_k, inp.W_v, inp.kp, inp.vp)
    cu = np.asarray(inp.cu_chunk_lens).copy()
    cu[3] = cu[2] - 1
    out = torch.full(inp.q.shape, 7.0, dtype=torch.float16, device="cuda")
    cache.prefill_attn(t(inp.q), t(cu), t(inp.cache.block_table), t(inp.seq_lens_after), out=out,
                       variant=variant, mod=score_mod(dict(window=50)))
    torch.cuda.synchronize()
    assert cache.read_device_error() & _lib.RCP_DEVERR_BAD_LEN
    assert bool((out == 7.0).all())


# ------------------------------------------------------------- biases, padding, streams, graphs
def odd_slopes(shape):
    """Biases that grow with the distance, steep ones and none.  A prefill tile's terms reach
    128 * 4 log2(e) < 2^10, of which fp32 keeps 2^-14 / 2: within the bound's 2^-15 of a unit
    (times log 2)."""
    return [(-0.05, 4.0, 0.0, -0.4, 0.3)[h % 5] for h in range(shape["num_heads"])]


@pytest.mark.parametrize("extra", [dict(), dict(window=90, prefix_lens=7, softcap=11.0)])
@pytest.mark.parametrize("shape_name,pages", [("main", "fp16"), ("main", "fp8_e4m3"), ("tiny", "int4")])
def test_biases_of_either_sign(shape_name, pages, extra):
    import torch
    for chunked in (False, True):
        inp = prefill_inputs(shape_name, pages) if chunked else decode_inputs(shape_name, pages)
        mod = dict(alibi_slopes=odd_slopes(inp.shape), **extra)
        if "prefix_lens" in mod:
            mod["prefix_lens"] = np.full(len(PRIOR if chunked else LENS), mod["prefix_lens"])
        if chunked:
            ref = oracle_prefill(inp, shape_name, pages, f"odd{len(extra)}", mod)
            for variant in ("rank", "reconstruct"):
                cache = cache_of(pages, inp.shape, inp.U_k, inp.W_v, inp.kp, inp.vp)
                out = cache.prefill_attn(t(inp.q), t(inp.cu_chunk_lens), t(inp.cache.block_table),
                                         t(inp.seq_lens_after), variant=variant, mod=score_mod(mod))
                assert_within(out.cpu().numpy(), ref, f"prefill {variant}")
        else:
            cache = cache_of(pages, inp.shape, inp.U_k, inp.W_v, inp.k, inp.v)
            out = cache.decode_attn(t(inp.q), t(inp.cache.block_table), t(inp.cache.seq_lens),
                                    mod=score_mod(mod))
            assert_within(out.cpu().numpy(), oracle_decode(inp, pages, mod), "decode")
        torch.cuda.synchronize()
        assert cache.read_device_error() == 0


@pytest.mark.parametrize("variant", ["rank", "reconstruct"])
@pytest.mark.parametrize("shape_name,pages", [("main", "fp16"), ("tiny", "fp8_e4m3")])
def test_prefill_rows_outside_the_chunks_are_left_as_they_were(shape_name, pages, variant):
    """Query rows ahead of the first chunk and behind the last one (a padded batch), whose
    row_begin holds anything."""
    import torch
    inp = prefill_inputs(shape_name, pages)
    rows, ahead, behind = sum(CHUNK), 3, 140
    begin = doc_begin(rows, PRIOR, CHUNK, 50)
    mod = dict(softcap=6.0, row_begin=begin)
    cache = cache_of(pages, inp.shape, inp.U_k, inp.W_v, inp.kp, inp.vp)
    args = (t(inp.cache.block_table), t(inp.seq_lens_after))
    pad = [(ahead, behind), (0, 0), (0, 0)]
    q = np.pad(inp.q, pad, constant_values=np.nan)
    cu = (np.asarray(inp.cu_chunk_lens) + ahead).astype(np.int32)
    wide = np.concatenate([[-5, 2 ** 31 - 1, -2 ** 31], begin, np.full(behind, -2 ** 31)])
    out = torch.full(q.shape, 7.0, dtype=torch.float16, device="cuda")
    cache.prefill_attn(t(q), t(cu), *args, out=out, variant=variant,
                       mod=score_mod(dict(mod, row_begin=wide)))
    torch.cuda.synchronize()
    assert cache.read_device_error() == 0
    assert bool((out[:ahead] == 7.0).all()) and bool((out[ahead + rows:] == 7.0).all())
    assert_within(out[ahead:ahead + rows].cpu().numpy(),
                  oracle_prefill(inp, shape_name, pages, "padded", mod), f"{shape_name} {variant}")


def stream_jobs(cache, shape, n):
    """Decodes and prefills of several masks over one cache: (call(stream, out), output)."""
    import torch
    rng = np.random.default_rng(331)
    jobs = []
    for i in range(n):
        B = 3 + 5 * i
        lens = rng.integers(1, 700, B).astype(np.int32)
        table = rng.integers(0, cache.num_blocks, (B, 44)).astype(np.int32)
        table, lens = t(table), t(lens)
        H, d = shape["num_heads"], shape["head_dim"]
        if i % 2 == 0:
            q = t(wl.fp16(rng.standard_normal((B, H, d)) * 3))
            mod = score_mod(dict(softcap=4.0 + i, window=200, prefix_lens=np.full(B, 20)))

            def call(stream, out, a=(q, table, lens), mod=mod):
                cache.decode_attn(*a, out=out, stream=stream, mod=mod)
        else:
            chunk = np.minimum(lens.cpu().numpy(), 1 + 40 * i)
            cu = t(np.concatenate([[0], np.cumsum(chunk)]).astype(np.int32))
            q = t(wl.fp16(rng.standard_normal((int(chunk.sum()), H, d)) * 3))
            mod = score_mod(dict(softcap=9.0, alibi_slopes=slopes_of(shape), window=150 + i))

            def call(stream, out, a=(q, cu, table, lens), mod=mod):
                cache.prefill_attn(*a, out=out, stream=stream, mod=mod)
        jobs.append((call, torch.empty_like(q)))
    return jobs


def stream_cache(shape_name, pages):
    shape = SHAPES[shape_name]
    rng = np.random.default_rng(332)
    H, d, rk, R = (shape[k] for k in ("num_heads", "head_dim", "rank_k", "rank_v"))
    k = wl.fp16(rng.standard_normal((300, H, 16, rk)))
    v = wl.fp16(rng.standard_normal((300, 16, R)))
    U = wl.fp16(rng.standard_normal((H, rk, d)) / np.sqrt(rk))
    W = wl.fp16(rng.standard_normal((R, H * d)) / np.sqrt(R))
    return shape, cache_of(pages, shape, U, W, *encode(pages, k, v))


@pytest.mark.parametrize("shape_name,pages", [("main", "fp16"), ("main", "fp8_e4m3"), ("tiny", "int4")])
def test_calls_on_several_streams_at_once(shape_name, pages):
    """Calls that overlap, each on a stream of its own with the cache's own workspaces."""
    import torch
    shape, cache = stream_cache(shape_name, pages)
    jobs = stream_jobs(cache, shape, 4)
    want = []
    for call, out in jobs:
        call(None, out)
        torch.cuda.synchronize()
        want.append(out.clone())
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(10):
        for _, out in jobs:
            out.fill_(float("nan"))
        torch.cuda.synchronize()
        for _ in range(4):
            for s, (call, out) in zip(streams, jobs):
                call(s, out)
        torch.cuda.synchronize()
        for (_, out), w in zip(jobs, want):
            assert torch.equal(out, w)
    assert cache.read_device_error() == 0


@pytest.mark.parametrize("shape_name,pages", [("main", "fp16"), ("tiny", "int4")])
def test_captured_calls_keep_their_workspaces(shape_name, pages):
    """Graphs captured without a workspace of the caller's: replayed after larger eager calls
    have replaced the cache's, and both at once."""
    import torch
    shape, cache = stream_cache(shape_name, pages)
    jobs = stream_jobs(cache, shape, 4)
    want = []
    for call, out in jobs[:2]:
        call(None, out)
        torch.cuda.synchronize()
        want.append(out.clone())
    graphs = []
    for call, out in jobs[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(None, out)
        graphs.append(g)
    for call, out in jobs[2:]:                           # larger workspaces
        call(None, out)
    torch.cuda.synchronize()
    junk = [torch.full((1 << 22,), 255, dtype=torch.uint8, device="cuda") for _ in range(64)]
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(10):
        for _, out in jobs[:2]:
            out.fill_(float("nan"))
        torch.cuda.synchronize()
        for _ in range(4):
            for s, g in zip(streams, graphs):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for (_, out), w in zip(jobs, want):
            assert torch.equal(out, w)
    assert cache.read_device_error() == 0
    assert all(bool((x == 255).all()) for x in junk)     # nothing wrote to memory handed on


@pytest.mark.parametrize("shape_name,pages", [("main", "fp16"), ("tiny", "int4")])
def test_calls_without_requests_or_rows(shape_name, pages):
    import torch
    shape, cache = stream_cache(shape_name, pages)
    H, d = shape["num_heads"], shape["head_dim"]
    q = torch.empty((0, H, d), dtype=torch.float16, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    table = torch.zeros((1, 4), dtype=torch.int32, device="cuda")
    mod = score_mod(dict(window=3, softcap=2.0, prefix_lens=[], row_begin=[]))
    assert cache.decode_attn(q, table, none, mod=mod).shape == q.shape
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    for variant in ("rank", "reconstruct", "auto"):
        assert cache.prefill_attn(q, cu, table, none, variant=variant, mod=mod).shape == q.shape
    # a request without chunk rows among none at all
    cu = torch.zeros(2, dtype=torch.int32, device="cuda")
    lens = torch.full((1,), 20, dtype=torch.int32, device="cuda")
    mod = score_mod(dict(window=3, softcap=2.0, prefix_lens=[7], row_begin=[]))
    assert cache.prefill_attn(q, cu, table, lens, mod=mod).shape == q.shape
    torch.cuda.synchronize()
    assert cache.read_device_error() == 0


def steep_slopes(shape):
    """Biases that leave one token of a row any weight: its nearest, or (negative) its farthest."""
    return [(1.0, -1.0)[h % 2] * 2.0 ** (9, 14, 20, 27, 34, 60)[h // 2 % 6]
            for h in range(shape["num_heads"])]


@pytest.mark.parametrize("extra", [dict(), dict(window=77), dict(window=50, prefix_lens=7, softcap=11.0)])
@pytest.mark.parametrize("shape_name,pages", [("main", "fp16"), ("main", "int4"), ("tiny", "fp8_e4m3")])
def test_steep_biases(shape_name, pages, extra):
    """Up to the largest magnitude allowed: the row is the value of one token, exactly weighted."""
    import torch
    for chunked in (False, True):
        inp = prefill_inputs(shape_name, pages) if chunked else decode_inputs(shape_name, pages)
        mod = dict(alibi_slopes=steep_slopes(inp.shape), **extra)
        if "prefix_lens" in mod:
            mod["prefix_lens"] = np.full(len(PRIOR if chunked else LENS), mod["prefix_lens"])
        if chunked:
            ref = oracle_prefill(inp, shape_name, pages, f"steep{len(extra)}", mod)
            for variant in ("rank", "reconstruct"):
                cache = cache_of(pages, inp.shape, inp.U_k, inp.W_v, inp.kp, inp.vp)
                out = cache.prefill_attn(t(inp.q), t(inp.cu_chunk_lens), t(inp.cache.block_table),
                                         t(inp.seq_lens_after), variant=variant, mod=score_mod(mod))
                assert_within(out.cpu().numpy(), ref, f"prefill {variant}")
        else:
            cache = cache_of(pages, inp.shape, inp.U_k, inp.W_v, inp.k, inp.v)
            out = cache.decode_attn(t(inp.q), t(inp.cache.block_table), t(inp.cache.seq_lens),
                                    mod=score_mod(mod))
            assert_within(out.cpu().numpy(), oracle_decode(inp, pages, mod), "decode")
        torch.cuda.synchronize()
        assert cache.read_device_error() == 0


@pytest.mark.parametrize("prior,chunk", [([500], [100]), ([90, 300, 40, 7], [8, 3, 5, 9])])
def test_auto_variant_without_effective_modifications_is_the_plain_call(prior, chunk):
    """Bit for bit, at sizes where the plain rule and the one under modifications differ."""
    import torch
    shape = SHAPES["main"]
    inp = wl.make_prefill_inputs(shape, prior, chunk, seed=351, fill=0.5)
    c = inp.cache
    cache = cache_of("fp16", shape, inp.U_k, inp.W_v, c.k_pages, c.v_pages)
    args = (t(inp.q), t(inp.cu_chunk_lens), t(c.block_table), t(inp.seq_lens_after))
    plain, got = cache.prefill_attn(*args), cache.prefill_attn(*args, mod=score_mod({}))
    torch.cuda.synchronize()
    assert torch.equal(plain.view(torch.int16), got.view(torch.int16))


def test_calls_keep_no_workspace():
    """Calls without a workspace of the caller's, plain and modified, on several streams: the
    allocator has all of their scratch back."""
    import torch
    shape, cache = stream_cache("main", "fp8_e4m3")
    jobs = stream_jobs(cache, shape, 4)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for s in [None] + [torch.cuda.Stream() for _ in range(3)]:
        for call, out in jobs:
            call(s, out)
    q = torch.zeros((2, shape["num_heads"], shape["head_dim"]), dtype=torch.float16, device="cuda")
    table, lens = t(np.zeros((2, 3), np.int32)), t(np.full(2, 40, np.int32))
    cache.decode_attn(q, table, lens)
    del q, table, lens
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() == before
    assert cache.read_device_error() == 0


def test_results_on_another_stream_take_that_streams_memory():
    """Memory freed on the current stream may still be in use there when a call on another
    stream writes its result."""
    import torch
    shape, cache = stream_cache("main", "fp16")
    H, d = shape["num_heads"], shape["head_dim"]
    B, n, mb = 24, 96, 7
    q = torch.zeros((n, H, d), dtype=torch.float16, device="cuda")
    table, lens = t(np.zeros((B, mb), np.int32)), t(np.full(B, 100, np.int32))
    cu, keep = t(np.arange(B + 1, dtype=np.int32) * 4), t(np.ones((B, mb * 16), np.uint8))
    mod = score_mod(dict(window=9))
    slots = t(np.full(B, -1, np.int64))
    kv = torch.zeros((B, H, d), dtype=torch.float16, device="cuda")
    side = torch.cuda.Stream()
    calls = {
        "decode": (q[:B], lambda: cache.decode_attn(q[:B], table, lens, stream=side)),
        "modified decode": (q[:B], lambda: cache.decode_attn(q[:B], table, lens, stream=side, mod=mod)),
        "sparse": (q[:B], lambda: cache.decode_attn_sparse(q[:B], table, lens, 2 ** -8, stream=side)),
        "step": (q[:B], lambda: cache.decode_step(kv, kv, slots, q[:B], table, lens, stream=side)),
        "prefill": (q, lambda: cache.prefill_attn(q, cu, table, lens, stream=side, mod=mod)),
        "prefill step": (q, lambda: cache.prefill_step(kv, kv, slots, q, cu, table, lens, stream=side)),
        "compaction": (lens, lambda: cache.compact_tokens(table, lens, keep, stream=side)),
    }
    torch.cuda.synchronize()
    for name, (like, call) in calls.items():
        freed = torch.empty_like(like)
        at, size = freed.data_ptr(), freed.numel() * freed.element_size()
        del freed
        out = call()
        assert not at - size < out.data_ptr() < at + size, name
        del out
    torch.cuda.synchronize()
    assert cache.read_device_error() == 0


@pytest.mark.parametrize("variant", ["rank", "reconstruct"])
@pytest.mark.parametrize("name", sorted(set(prefill_mods(SHAPES["main"])) - {"all", "docs", "prefix_bias"}))
def test_prefill_on_4_bit_pages_at_the_main_shape(name, variant):
    """The masks that the list above leaves to the small shape."""
    test_prefill_matches_oracle("main", "int4", name, variant)


_long = {}


def long_prefill(pages):
    """Two chunks behind thousands of tokens, coefficients as given."""
    if pages not in _long:
        shape = SHAPES["main"]
        inp = wl.make_prefill_inputs(shape, [5003, 2100], [139, 9], seed=361)
        rng = np.random.default_rng(362)
        c = inp.cache
        kp, vp = (wl.fp16(rng.standard_normal(x.shape)) for x in (c.k_pages, c.v_pages))
        inp.q = wl.fp16(inp.q.astype(np.float64) * 4)
        inp.kp, inp.vp = encode(pages, kp, vp)
        _long[pages] = inp
    return _long[pages]


@pytest.mark.parametrize("variant", ["rank", "reconstruct"])
@pytest.mark.parametrize("extra", [dict(), dict(window=2500, prefix_lens=[300, 40], softcap=20.0)])
@pytest.mark.parametrize("pages", ["fp16", "int4"])
def test_prefill_bias_behind_thousands_of_tokens(pages, extra, variant):
    """Gentle and ordinary biases of either sign: a tile's terms stay below 2^8 where weights are
    not zero, of which fp32 keeps 2^-16."""
    import torch
    inp = long_prefill(pages)
    H = inp.shape["num_heads"]
    slopes = [(2.0 ** (-8 * (h + 1) / H), 2.0 ** -10, -2.0 ** -10, -2.0 ** -8)[h % 4] for h in range(H)]
    mod = dict(alibi_slopes=slopes, **extra)
    key = ("long", pages, len(extra))
    if key not in _ref_cache:
        kk, vv = values(pages, inp.shape, inp.kp, inp.vp, True)
        _ref_cache[key] = (*orc.prefill_attn_mod(
            inp.q, inp.cu_chunk_lens, kk, vv, inp.U_k, inp.W_v, inp.cache.block_table,
            inp.seq_lens_after, magnitudes=True, **mod), int(max(inp.seq_lens_after)))
    cache = cache_of(pages, inp.shape, inp.U_k, inp.W_v, inp.kp, inp.vp)
    out = cache.prefill_attn(t(inp.q), t(inp.cu_chunk_lens), t(inp.cache.block_table),
                             t(inp.seq_lens_after), variant=variant, mod=score_mod(mod))
    torch.cuda.synchronize()
    assert cache.read_device_error() == 0
    assert_within(out.cpu().numpy(), _ref_cache[key], f"long {pages} {variant}")
