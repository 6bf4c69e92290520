"""Page copies, forks and compaction vs the oracle, byte for byte (needs a GB300)."""
import numpy as np
import pytest

import workloads as wl
from oracle import rcp_oracle as orc
from tests.mod_util import assert_within, cache_of, encode, score_mod, values
from tests.gpu_util import t

pytestmark = pytest.mark.gpu

SHAPES = {"tiny": wl.SHAPES["tiny"], "main": wl.SHAPES["mha32"]}
FORMATS = ["fp16", "fp8_e4m3", "int4"]


def random_pages(shape, pages, num_blocks, seed):
    """Every byte random (the moves do not look at what it means)."""
    rng = np.random.default_rng(seed)
    H, rk, R = (shape[x] for x in ("num_heads", "rank_k", "rank_v"))
    if pages == "int4":
        kb, vb = orc.int4_page_bytes(H, rk, R)
        return (rng.integers(0, 256, (num_blocks, kb), np.uint8),
                rng.integers(0, 256, (num_blocks, vb), np.uint8))
    n = 2 if pages == "fp16" else 1
    k = rng.integers(0, 256, (num_blocks, H, 16, rk * n), np.uint8)
    v = rng.integers(0, 256, (num_blocks, 16, R * n), np.uint8)
    return (k.view(np.float16), v.view(np.float16)) if n == 2 else (k, v)


def new_cache(shape, pages, k, v):
    U, W = wl.make_factors(np.random.default_rng(0), *(shape[x] for x in (
        "num_heads", "head_dim", "rank_k", "rank_v")))
    return cache_of(pages, shape, U, W, k, v)


def raw(x):
    x = x if isinstance(x, np.ndarray) else x.cpu().numpy()
    return x.view(np.uint8)


# ---------------------------------------------------------------------------------- copies
@pytest.mark.parametrize("pages", FORMATS)
@pytest.mark.parametrize("shape_name", ["tiny", "main"])
@pytest.mark.parametrize("n", [1, 2, 7, 90])
def test_copy_blocks(shape_name, pages, n):
    import torch
    shape = SHAPES[shape_name]
    k, v = random_pages(shape, pages, 200, seed=n)
    cache = new_cache(shape, pages, k, v)
    rng = np.random.default_rng(n)
    dst = rng.permutation(200)[:n]
    src = rng.choice(np.setdiff1d(np.arange(200), dst), n)      # a source may serve many
    pairs = np.stack([src, dst], 1).astype(np.int32)
    cache.copy_blocks(t(pairs))
    torch.cuda.synchronize()
    assert cache.read_device_error() == 0
    k, v = raw(k).copy(), raw(v).copy()
    k[dst], v[dst] = k[src], v[src]
    assert np.array_equal(raw(cache.k_pages), k) and np.array_equal(raw(cache.v_pages), v)


def test_copy_blocks_padding_bad_ids_and_replay():
    """-1 skips; a bad id is reported and copies nothing; a graph replays with new pairs."""
    import torch
    from rank_compressed_paged_gb300 import _lib
    shape = SHAPES["main"]
    k, v = random_pages(shape, "fp16", 12, seed=3)
    cache = new_cache(shape, "fp16", k, v)
    pairs = t(np.array([[0, 5], [-1, 6], [7, -1], [1, 1]], np.int32))
    cache.copy_blocks(pairs)
    torch.cuda.synchronize()
    assert cache.read_device_error() == 0
    want = raw(k).copy()
    want[5] = want[0]
    assert np.array_equal(raw(cache.k_pages), want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.copy_blocks(pairs)
    pairs.copy_(t(np.array([[12, 6], [2, -7], [3, 8], [4, 9]], np.int32)))
    g.replay()
    torch.cuda.synchronize()
    assert cache.read_device_error() == _lib.RCP_DEVERR_BAD_BLOCK
    want[8], want[9] = want[3], want[4]
    assert np.array_equal(raw(cache.k_pages), want)


@pytest.mark.parametrize("pages", FORMATS)
@pytest.mark.parametrize("children", [1, 3, 1000])
def test_fork_sequence_copies_the_partial_page(pages, children):
    import torch
    shape = SHAPES["tiny"]
    k, v = random_pages(shape, pages, 1100, seed=5)
    cache = new_cache(shape, pages, k, v)
    ids = cache.alloc_blocks(6)
    kids = cache.fork_sequence(ids, 16 * 4 + 3, children)
    torch.cuda.synchronize()
    assert len(kids) == children and all(x[:4] == ids[:4] for x in kids)
    own = [x[4] for x in kids]
    assert len(set(own)) == children and not set(own) & set(ids)
    assert cache.block_refs(ids) == [1 + children] * 4 + [1, 1]
    assert cache.block_refs(own) == [1] * children
    assert cache.num_free_blocks() == 1100 - 6 - children
    wk, wv = raw(k).copy(), raw(v).copy()
    wk[own], wv[own] = wk[ids[4]], wv[ids[4]]
    assert np.array_equal(raw(cache.k_pages), wk) and np.array_equal(raw(cache.v_pages), wv)
    for x in kids:
        cache.free_blocks(x)
    assert cache.block_refs(ids) == [1] * 6 and cache.num_free_blocks() == 1094


# ------------------------------------------------------------------------------ compaction
def keep_patterns(lens, T, seed):
    rng = np.random.default_rng(seed)
    B = len(lens)
    none, every = np.zeros((B, T), np.uint8), np.full((B, T), 255, np.uint8)
    first, last, pages = every.copy(), none.copy(), none.copy()
    first[:, 0] = 0                                     # everything moves by one
    for b, L in enumerate(lens):
        if L > 0:
            last[b, L - 1] = 1
    pages[:, (np.arange(T) // 16) % 3 == 1] = 7         # whole pages
    return {"none": none, "all": every, "first_dropped": first, "last_kept": last, "pages": pages,
            "half": (rng.random((B, T)) < 0.5).astype(np.uint8),
            "few": (rng.random((B, T)) < 0.03).astype(np.uint8),
            "most": (rng.random((B, T)) < 0.97).astype(np.uint8) * 128,
            "tail": (np.arange(T)[None] > np.asarray(lens)[:, None] // 2).astype(np.uint8)
            * (rng.random((B, T)) < 0.8)}


PATTERNS = ["none", "all", "first_dropped", "last_kept", "pages", "half", "few", "most", "tail"]


def compaction(shape, pages, lens, keep_of, seed):
    import torch
    nblk = [(L + 15) // 16 for L in lens]
    mb = max(nblk) + 1
    total = sum(nblk) + 5
    k, v = random_pages(shape, pages, total, seed)
    perm = np.random.default_rng(seed).permutation(total).astype(np.int32)
    table = np.full((len(lens), mb), 1 << 29, np.int32)          # never looked at past the end
    at = 0
    for b, n in enumerate(nblk):
        table[b, :n] = perm[at:at + n]
        at += n
    keep = np.ascontiguousarray(keep_of(mb * 16).astype(np.uint8))
    cache = new_cache(shape, pages, k, v)
    new = cache.compact_tokens(t(table), t(np.asarray(lens, np.int32)), t(keep))
    torch.cuda.synchronize()
    assert cache.read_device_error() == 0
    wk, wv, wl_ = orc.compact_tokens(k, v, pages, shape, table, lens, keep)
    assert np.array_equal(new.cpu().numpy(), wl_)
    assert np.array_equal(raw(cache.k_pages), raw(wk)), "keys"
    assert np.array_equal(raw(cache.v_pages), raw(wv)), "values"


@pytest.mark.parametrize("pattern", PATTERNS)
@pytest.mark.parametrize("pages", FORMATS)
@pytest.mark.parametrize("shape_name", ["tiny", "main"])
def test_compact_tokens(shape_name, pages, pattern):
    lens = [0, 1, 15, 16, 17, 40, 333, 512]
    compaction(SHAPES[shape_name], pages, lens,
               lambda T: keep_patterns(lens, T, 7)[pattern], seed=8)


@pytest.mark.parametrize("pattern", ["half", "few", "most", "tail", "first_dropped"])
@pytest.mark.parametrize("pages", FORMATS)
def test_compact_tokens_long_requests(pages, pattern):
    """Lengths around and far past the span of mask bytes scanned at a time."""
    lens = [2048, 2047, 2049, 9000, 4097, 6]
    compaction(SHAPES["tiny"], pages, lens, lambda T: keep_patterns(lens, T, 9)[pattern], seed=10)
    if pattern == "half":
        compaction(SHAPES["main"], pages, [5003], lambda T: keep_patterns([5003], T, 9)[pattern],
                   seed=11)


def test_compact_tokens_many_requests():
    lens = [int(x) for x in np.random.default_rng(1).integers(0, 70, 400)]
    compaction(SHAPES["tiny"], "fp16", lens, lambda T: keep_patterns(lens, T, 2)["half"], seed=12)


def test_compact_tokens_leaves_shared_pages_that_stay():
    """Two requests share a page of which every token stays; both drop tokens behind it."""
    import torch
    shape = SHAPES["main"]
    k, v = random_pages(shape, "fp16", 10, seed=13)
    table = np.array([[0, 1, 2, 3], [0, 4, 5, 6]], np.int32)
    keep = np.ones((2, 64), np.uint8)
    keep[0, 20:30] = 0
    keep[1, 16:60:2] = 0
    cache = new_cache(shape, "fp16", k, v)
    lens = np.array([60, 64], np.int32)
    new = cache.compact_tokens(t(table), t(lens), t(keep))
    torch.cuda.synchronize()
    wk, wv, wlens = orc.compact_tokens(k, v, "fp16", shape, table, lens, keep)
    assert np.array_equal(new.cpu().numpy(), wlens)
    assert np.array_equal(raw(cache.k_pages), raw(wk)) and np.array_equal(raw(cache.v_pages), raw(wv))


def test_compact_tokens_bad_lengths_and_blocks():
    import torch
    from rank_compressed_paged_gb300 import _lib
    shape = SHAPES["tiny"]
    k, v = random_pages(shape, "fp16", 20, seed=14)
    table = np.arange(16, dtype=np.int32).reshape(4, 4)
    table[2, 1] = 20                                    # tokens 16 .. 31 of request 2
    lens = np.array([-1, 65, 64, 64], np.int32)
    keep = np.ones((4, 64), np.uint8)
    keep[:, 40] = 0
    keep[2, 3] = 0
    cache = new_cache(shape, "fp16", k, v)
    new = cache.compact_tokens(t(table), t(lens), t(keep))
    torch.cuda.synchronize()
    assert cache.read_device_error() == _lib.RCP_DEVERR_BAD_LEN | _lib.RCP_DEVERR_BAD_BLOCK
    assert list(new.cpu().numpy()) == [0, 0, 62, 63]
    wk, wv = k.copy(), v.copy()
    for b in (2, 3):
        src, dst = orc.compact_moves(table[b], 64, keep[b])
        ok = (src // 16 < 20) & (dst // 16 < 20)
        src, dst = src[ok], dst[ok]
        wk[dst // 16, :, dst % 16] = k[src // 16, :, src % 16]
        wv[dst // 16, dst % 16] = v[src // 16, src % 16]
    assert np.array_equal(raw(cache.k_pages), raw(wk)) and np.array_equal(raw(cache.v_pages), raw(wv))


def test_compact_tokens_replays_from_a_graph():
    import torch
    shape = SHAPES["main"]
    k, v = random_pages(shape, "int4", 30, seed=15)
    cache = new_cache(shape, "int4", k, v)
    table = t(np.arange(24, dtype=np.int32).reshape(2, 12))
    lens, keep = t(np.array([190, 150], np.int32)), t(np.ones((2, 192), np.uint8))
    new = torch.zeros(2, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.compact_tokens(table, lens, keep, new_lens=new)
    wk, wv, wlens = k, v, [190, 150]
    for seed in (1, 2):
        kp = (np.random.default_rng(seed).random((2, 192)) < 0.7).astype(np.uint8)
        keep.copy_(t(kp))
        lens.copy_(t(np.asarray(wlens, np.int32)))
        g.replay()
        torch.cuda.synchronize()
        wk, wv, wlens = orc.compact_tokens(wk, wv, "int4", shape, table.cpu().numpy(), wlens, kp)
        assert np.array_equal(new.cpu().numpy(), wlens)
        assert np.array_equal(raw(cache.k_pages), wk) and np.array_equal(raw(cache.v_pages), wv)


# --------------------------------------------------------------------------------- together
@pytest.mark.parametrize("pages", FORMATS)
def test_fork_step_copy_on_write_compact_and_attend(pages):
    """A conversation as a server runs it: a prompt is forked, each branch appends tokens of
    its own and attends with a window behind the shared prompt, a shared page is copied
    before it is written, a branch drops tokens and frees the pages behind them, and both
    attend again."""
    import torch
    shape = SHAPES["main"]
    H, d = shape["num_heads"], shape["head_dim"]
    rng = np.random.default_rng(20)
    U, W = wl.make_factors(rng, H, d, shape["rank_k"], shape["rank_v"])
    kp = wl.fp16(rng.standard_normal((64, H, 16, shape["rank_k"])))
    vp = wl.fp16(rng.standard_normal((64, 16, shape["rank_v"])))
    cache = cache_of(pages, shape, U, W, *encode(pages, kp, vp))
    ids = cache.alloc_blocks(7)
    length = 100
    child, = cache.fork_sequence(ids, length)
    tables = [ids, child]
    mod = dict(softcap=20.0, window=40, prefix_lens=np.array([30, 30]),
               alibi_slopes=[2.0 ** (-8 * (h + 1) / H) for h in range(H)])

    def table():
        out = np.full((2, 8), -1, np.int32)
        for b, x in enumerate(tables):
            out[b, :len(x)] = x
        return out

    def check(q, out, lens, what):
        torch.cuda.synchronize()
        assert cache.read_device_error() == 0
        kk, vv = values(pages, shape, cache.k_pages.cpu().numpy(), cache.v_pages.cpu().numpy(), False)
        ref = orc.decode_attn_mod(q, kk, vv, U, W, table(), lens, magnitudes=True, **mod)
        assert_within(out.cpu().numpy(), (*ref, max(lens)), what)

    lens = np.array([length, length], np.int32)
    before = cache.k_pages[ids[6]].clone()
    for step in range(3):
        lens = lens + 1
        tab = table()
        slots = np.array([wl.slot_for(tab, b, int(L) - 1) for b, L in enumerate(lens)], np.int64)
        k, v = (wl.fp16(rng.standard_normal((2, H, d))) for _ in range(2))
        q = wl.fp16(4 * rng.standard_normal((2, H, d)))
        out = cache.decode_step(t(k), t(v), t(slots), t(q), t(tab), t(lens), mod=score_mod(mod))
        check(q, out, lens, f"step {step}")
    assert child[6] != ids[6] and not torch.equal(cache.k_pages[ids[6]], cache.k_pages[child[6]])
    assert not torch.equal(before, cache.k_pages[ids[6]])

    # the child drops tokens from position 20 on: its copy of every page from there must be its own
    own = cache.alloc_blocks(5)
    cache.copy_blocks(t(np.stack([child[1:6], own], 1).astype(np.int32)))
    cache.free_blocks(child[1:6])
    tables[1] = child[:1] + own + child[6:]
    assert cache.block_refs(ids) == [2, 1, 1, 1, 1, 1, 1]
    parent = cache.k_pages[torch.tensor(ids, device="cuda")].clone()
    keep = np.ones((2, 128), np.uint8)
    keep[1, 20:90] = rng.random(70) < 0.4
    new = cache.compact_tokens(t(table()), t(lens), t(keep)).cpu().numpy()
    assert new[0] == lens[0] and new[1] == keep[1, :lens[1]].sum()
    assert torch.equal(parent, cache.k_pages[torch.tensor(ids, device="cuda")])
    used = (int(new[1]) + 15) // 16
    free0 = cache.num_free_blocks()
    cache.free_blocks(tables[1][used:])
    assert cache.num_free_blocks() == free0 + 7 - used
    tables[1] = tables[1][:used]
    q = wl.fp16(4 * rng.standard_normal((2, H, d)))
    out = cache.decode_attn(t(q), t(table()), t(new.astype(np.int32)), mod=score_mod(mod))
    check(q, out, new, "after compaction")
    # a chunk of queries over both branches
    cu = np.array([0, 3, 10], np.int32)
    q = wl.fp16(4 * rng.standard_normal((10, H, d)))
    for variant in ("rank", "reconstruct"):
        out = cache.prefill_attn(t(q), t(cu), t(table()), t(new.astype(np.int32)), variant=variant,
                                 mod=score_mod(mod))
        torch.cuda.synchronize()
        kk, vv = values(pages, shape, cache.k_pages.cpu().numpy(), cache.v_pages.cpu().numpy(), True)
        ref = orc.prefill_attn_mod(q, cu, kk, vv, U, W, table(), new, magnitudes=True, **mod)
        assert_within(out.cpu().numpy(), (*ref, max(new)), variant)


def test_calls_on_nothing():
    import torch
    k, v = random_pages(SHAPES["tiny"], "fp16", 6, 1)
    cache = new_cache(SHAPES["tiny"], "fp16", k, v)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    cache.copy_blocks(none.view(0, 2))
    keep = torch.empty((0, 64), dtype=torch.uint8, device="cuda")
    assert cache.compact_tokens(none.view(0, 4), none, keep).shape == (0,)
    ids = cache.alloc_blocks(2)
    assert cache.fork_sequence(ids, 0, children=3) == [[], [], []]
    assert cache.fork_sequence(ids, 20, children=0) == []
    assert cache.block_refs(ids) == [1, 1] and cache.num_free_blocks() == 4
    for bad in (dict(ids=ids, length=33), dict(ids=ids, length=-1), dict(ids=ids, length=2 ** 32),
                dict(ids=ids, length=20, children=-1), dict(ids=[2 ** 32], length=3)):
        with pytest.raises(ValueError):
            cache.fork_sequence(**bad)
    assert cache.block_refs(ids) == [1, 1] and cache.num_free_blocks() == 4
    torch.cuda.synchronize()
    assert np.array_equal(raw(cache.k_pages), raw(k)) and np.array_equal(raw(cache.v_pages), raw(v))
    assert cache.read_device_error() == 0


# ------------------------------------------------- requests of several spans of 32768 tokens
def span_masks(lens, T, name):
    """none of the first span moves; a destination inside a page is carried over to the second;
    whole spans are dropped; every third token goes."""
    rng = np.random.default_rng(21)
    B, pos = len(lens), np.arange(T)[None]
    if name == "second_moves":
        keep = np.broadcast_to(pos != 32768 + 5, (B, T))
    elif name == "carried":
        keep = np.broadcast_to(~np.isin(pos, [3, 32000, 32766]) & (pos % 7 != 5), (B, T))
    elif name == "late_carried":                       # the first move is the span's last token
        keep = np.broadcast_to((pos != 32766) & ((pos < 33000) | (rng.random((B, T)) < 0.4)), (B, T))
    elif name == "span_dropped":
        keep = np.broadcast_to(((pos < 11) | (pos >= 32768)) & (pos != 65536), (B, T))
    else:
        keep = rng.random((B, T)) < 0.6
    return keep.astype(np.uint8)


@pytest.mark.parametrize("name", ["second_moves", "carried", "late_carried", "span_dropped", "random"])
@pytest.mark.parametrize("pages", FORMATS)
@pytest.mark.parametrize("beside", [0, 120])
def test_compact_tokens_over_several_spans(pages, name, beside):
    """Few requests (a cluster of CTAs per slice), and many short ones beside the long ones (one
    CTA per slice)."""
    if beside:
        lens = [70001, 32769] + [int(x) for x in np.random.default_rng(4).integers(0, 40, beside)]
    else:
        lens = [32767, 32768, 32769, 70001]
    compaction(SHAPES["tiny"], pages, lens, lambda T: span_masks(lens, T, name), seed=22)


@pytest.mark.parametrize("pages", FORMATS)
def test_compact_tokens_over_several_spans_main_shape(pages):
    lens = [33007]
    compaction(SHAPES["main"], pages, lens, lambda T: span_masks(lens, T, "late_carried"), seed=23)


@pytest.mark.parametrize("pages", FORMATS)
@pytest.mark.parametrize("masked", [True, False])
def test_a_step_without_visible_tokens_ends_with_its_append(pages, masked):
    """A step of which no row sees a token (masked: by its row_begin; else by its length) still
    appends; the page copy queued behind it takes the appended pages."""
    import torch
    shape = SHAPES["main"]
    H, d = shape["num_heads"], shape["head_dim"]
    n, B, tokens = 400, 3, 2048
    k, v = random_pages(shape, pages, n, seed=24)
    cache, other = new_cache(shape, pages, k, v), new_cache(shape, pages, k, v)
    rng = np.random.default_rng(25)
    new_k, new_v = (t(wl.fp16(rng.standard_normal((tokens, H, d)))) for _ in range(2))
    slots = t(rng.permutation(tokens).astype(np.int64))          # blocks 0 .. 127
    q = t(wl.fp16(rng.standard_normal((B, H, d))))
    table = t(np.arange(3 * 9, dtype=np.int32).reshape(B, 9) + 150)
    lens = t(np.full(B, 120 if masked else 0, np.int32))
    mod = score_mod(dict(row_begin=np.full(B, 120))) if masked else None
    pairs = t(np.stack([np.arange(128), 200 + np.arange(128)], 1).astype(np.int32))
    other.append_kv(new_k, new_v, slots)
    torch.cuda.synchronize()
    want = [x[:128].clone() for x in (other.k_pages.view(torch.uint8), other.v_pages.view(torch.uint8))]
    old = [t(raw(x)) for x in (k, v)]
    got = [x.view(torch.uint8) for x in (cache.k_pages, cache.v_pages)]
    for _ in range(5):
        for x, o in zip(got, old):
            x.copy_(o)
        cache.decode_step(new_k, new_v, slots, q, table, lens, mod=mod)
        cache.copy_blocks(pairs)
        torch.cuda.synchronize()
        assert cache.read_device_error() == 0
        for x, w in zip(got, want):
            assert torch.equal(x[:128], w) and torch.equal(x[200:328], w)
