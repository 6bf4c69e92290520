"""Pool references, host checks and binding checks of the score-modified attention, page copy,
fork and compaction calls (no GPU: every call returns before any CUDA call)."""
import ctypes

import pytest
import torch

import rank_compressed_paged_gb300 as rcp
from rank_compressed_paged_gb300 import ScoreMod, _lib

CPU = torch.device("cpu")
INF = float("inf")


@pytest.fixture(scope="module")
def lib():
    from rank_compressed_paged_gb300 import build
    build.build()
    return _lib.load()


@pytest.fixture
def handle(lib):
    cfg = _lib.CacheConfig(32, 128, 64, 1024, 16, 12, 0)
    h = ctypes.c_void_p()
    assert lib.rcp_create_cache(ctypes.byref(cfg), 0x10000, 0x20000, 0x30000, 0x40000, 0x50000,
                                ctypes.byref(h)) == _lib.RCP_OK
    yield h
    lib.rcp_destroy_cache(h)


def ids(*x):
    return (ctypes.c_int32 * max(len(x), 1))(*x)


def refs(lib, h, *x):
    out = (ctypes.c_int32 * len(x))()
    assert lib.rcp_block_refs(h, len(x), ids(*x), out) == _lib.RCP_OK
    return list(out)


def num_free(lib, h):
    n = ctypes.c_int64()
    lib.rcp_num_free_blocks(h, ctypes.byref(n))
    return n.value


def test_references_hold_blocks_until_the_last_is_freed(lib, handle):
    got = (ctypes.c_int32 * 4)()
    assert lib.rcp_alloc_blocks(handle, 4, got) == _lib.RCP_OK
    a, b, c, d = got
    assert refs(lib, handle, a, b, c, d, 11) == [1, 1, 1, 1, 0]
    assert lib.rcp_fork_blocks(handle, 3, ids(a, b, a)) == _lib.RCP_OK     # a twice
    assert refs(lib, handle, a, b, c) == [3, 2, 1]
    assert lib.rcp_free_blocks(handle, 3, ids(a, b, c)) == _lib.RCP_OK
    assert refs(lib, handle, a, b, c) == [2, 1, 0] and num_free(lib, handle) == 9
    assert lib.rcp_free_blocks(handle, 2, ids(a, a)) == _lib.RCP_ERR_CAPACITY   # repeated, as before
    assert lib.rcp_free_blocks(handle, 1, ids(c)) == _lib.RCP_ERR_CAPACITY
    assert refs(lib, handle, a, b, c) == [2, 1, 0]
    for _ in range(2):
        assert lib.rcp_free_blocks(handle, 1, ids(a)) == _lib.RCP_OK
    assert refs(lib, handle, a) == [0] and num_free(lib, handle) == 10
    again = (ctypes.c_int32 * 1)()
    assert lib.rcp_alloc_blocks(handle, 1, again) == _lib.RCP_OK and again[0] == a
    assert refs(lib, handle, a) == [1]


def test_fork_refuses_free_and_unknown_blocks(lib, handle):
    got = (ctypes.c_int32 * 2)()
    assert lib.rcp_alloc_blocks(handle, 2, got) == _lib.RCP_OK
    for bad in (5, 12, -1):
        assert lib.rcp_fork_blocks(handle, 2, ids(got[0], bad)) == _lib.RCP_ERR_CAPACITY
    assert refs(lib, handle, *got) == [1, 1]
    assert lib.rcp_fork_blocks(handle, -1, got) == _lib.RCP_ERR_INVALID_ARG
    assert lib.rcp_fork_blocks(handle, 1, None) == _lib.RCP_ERR_INVALID_ARG
    assert lib.rcp_fork_blocks(None, 0, None) == _lib.RCP_ERR_INVALID_ARG
    assert lib.rcp_fork_blocks(handle, 0, None) == _lib.RCP_OK
    out = (ctypes.c_int32 * 1)()
    assert lib.rcp_block_refs(handle, 1, ids(12), out) == _lib.RCP_ERR_CAPACITY
    assert lib.rcp_block_refs(handle, 1, ids(0), None) == _lib.RCP_ERR_INVALID_ARG


def test_fork_sequence_of_full_pages_shares_them(lib, handle):
    """No partial page: nothing is copied, so no CUDA call is made."""
    got = (ctypes.c_int32 * 3)()
    assert lib.rcp_alloc_blocks(handle, 3, got) == _lib.RCP_OK
    child = (ctypes.c_int32 * 4)()
    assert lib.rcp_fork_sequence(handle, got, 3, 32, 2, child, None) == _lib.RCP_OK
    assert list(child) == [got[0], got[1]] * 2
    assert refs(lib, handle, *got) == [3, 3, 1] and num_free(lib, handle) == 9
    assert lib.rcp_fork_sequence(handle, got, 3, 0, 2, child, None) == _lib.RCP_OK
    assert lib.rcp_fork_sequence(handle, got, 3, 32, 0, None, None) == _lib.RCP_OK
    assert refs(lib, handle, *got) == [3, 3, 1]


def test_fork_sequence_checks_change_nothing(lib, handle):
    got = (ctypes.c_int32 * 10)()
    assert lib.rcp_alloc_blocks(handle, 10, got) == _lib.RCP_OK
    child = (ctypes.c_int32 * 30)()
    fork = lib.rcp_fork_sequence
    assert fork(handle, got, 2, 33, 1, child, None) == _lib.RCP_ERR_INVALID_ARG   # needs 3 blocks
    assert fork(handle, got, 3, -1, 1, child, None) == _lib.RCP_ERR_INVALID_ARG
    assert fork(handle, got, 3, 40, -1, child, None) == _lib.RCP_ERR_INVALID_ARG
    assert fork(handle, None, 3, 40, 1, child, None) == _lib.RCP_ERR_INVALID_ARG
    assert fork(handle, got, 3, 40, 1, None, None) == _lib.RCP_ERR_INVALID_ARG
    assert fork(handle, got, 3, 40, 3, child, None) == _lib.RCP_ERR_CAPACITY      # two are free
    assert fork(handle, ids(got[0], 11, got[1]), 3, 40, 1, child, None) == _lib.RCP_ERR_CAPACITY
    assert refs(lib, handle, *got) == [1] * 10 and num_free(lib, handle) == 2


def test_copy_and_compact_host_checks(lib, handle):
    INV = _lib.RCP_ERR_INVALID_ARG
    assert lib.rcp_copy_blocks(handle, 0x1000, -1, None) == INV
    assert lib.rcp_copy_blocks(handle, None, 2, None) == INV
    assert lib.rcp_copy_blocks(handle, 0x1002, 2, None) == INV
    assert lib.rcp_copy_blocks(handle, None, 0, None) == _lib.RCP_OK

    def compact(table=0x1000, mb=4, lens=0x2000, keep=0x3000, batch=8, new=0x4000):
        return lib.rcp_compact_tokens(handle, table, mb, lens, keep, batch, new, None)
    for bad in (dict(table=None), dict(lens=None), dict(keep=None), dict(new=None), dict(mb=0),
                dict(mb=(1 << 26) + 1), dict(batch=-1), dict(keep=0x3008), dict(new=0x4002),
                dict(new=0x2000), dict(new=0x2000 + 28), dict(new=0x2000 - 28)):
        assert compact(**bad) == INV, bad
    assert compact(batch=(1 << 20) + 1, new=0x80000000) == _lib.RCP_ERR_UNSUPPORTED
    assert compact(batch=0, table=None) == _lib.RCP_OK


def test_score_mod_host_checks(lib, handle):
    """Every member is checked before any CUDA call, for decode and prefill alike."""
    INV = _lib.RCP_ERR_INVALID_ARG
    b = ctypes.c_size_t()
    assert lib.rcp_prefill_reconstruct_workspace_size(handle, 8, 8, 64, ctypes.byref(b)) == 0

    def both(mod, mb=64, ws=None, recon=1, T=0):
        ws = b.value if ws is None else ws
        p = ctypes.byref(mod) if mod is not None else None
        d = lib.rcp_decode_step_mod(handle, 0x1000, 0x2000, 0x3000, T, 0x4000, 0x5000, mb, 0x6000, 8,
                                    p, 0x7000, 0x100000, ws, None)
        f = lib.rcp_prefill_step_mod(handle, 0x1000, 0x2000, 0x3000, T, 0x4000, 0x8000, 8, 0x5000, mb,
                                     0x6000, 8, recon, p, 0x7000, 0x100000, ws, None)
        return d, f
    A = _lib.ScoreModArgs
    for cap in (-1.0, float("nan"), INF, 2.0 ** -11, 2.0 ** 10 * 1.01):
        assert both(A(softcap=cap)) == (INV, INV), cap
    assert both(A(window=-1)) == (INV, INV)
    assert both(A(alibi_slopes=0x1002)) == (INV, INV)
    assert both(A(prefix_lens=0x1001)) == (INV, INV)
    assert both(A(row_begin=0x1003)) == (INV, INV)
    assert both(A(softcap=1.0), mb=(1 << 26) + 1) == (INV, INV)
    # what is in range goes on to the checks of the plain calls
    for mod in (None, A(), A(softcap=2.0 ** -10, window=2 ** 31 - 1), A(softcap=2.0 ** 10)):
        assert both(mod, ws=1024) == (_lib.RCP_ERR_WORKSPACE,) * 2
    assert both(A(softcap=1.0), T=-1) == (INV, INV)
    assert both(A(softcap=1.0), recon=2)[1] == INV


# ------------------------------------------------------------------------ python arguments
def test_score_mod_tensors_are_checked():
    ok = ScoreMod(alibi_slopes=torch.zeros(4), prefix_lens=torch.zeros(3, dtype=torch.int32),
                  row_begin=torch.zeros(7, dtype=torch.int32))
    rcp._validate_mod(CPU, 4, 3, 7, ok)
    rcp._validate_mod(CPU, 4, 3, 7, ScoreMod())
    for kw, match in ((dict(alibi_slopes=torch.zeros(5)), "alibi_slopes must have shape"),
                      (dict(alibi_slopes=torch.zeros(4, dtype=torch.float16)), "float32"),
                      (dict(alibi_slopes=[0.5] * 4), "torch.Tensor"),
                      (dict(alibi_slopes=torch.zeros(8)[::2]), "contiguous"),
                      (dict(prefix_lens=torch.zeros(3, dtype=torch.int64)), "int32"),
                      (dict(prefix_lens=torch.zeros(2, dtype=torch.int32)), "prefix_lens must have"),
                      (dict(row_begin=torch.zeros(3, dtype=torch.int32)), "row_begin must have")):
        with pytest.raises(ValueError, match=match):
            rcp._validate_mod(CPU, 4, 3, 7, ScoreMod(**kw))
    with pytest.raises(ValueError, match="ScoreMod"):
        rcp._validate_mod(CPU, 4, 3, 7, dict(softcap=1.0))
    with pytest.raises(ValueError, match="must be on cuda:0"):
        rcp._validate_mod(torch.device("cuda", 0), 4, 3, 7, ok)
    with pytest.raises(ValueError, match="32 bits"):
        ScoreMod(window=2 ** 31)


def test_compact_tensors_are_checked():
    def args(**kw):
        a = dict(block_table=torch.zeros((3, 5), dtype=torch.int32),
                 seq_lens=torch.zeros(3, dtype=torch.int32),
                 keep=torch.zeros((3, 80), dtype=torch.uint8),
                 new_lens=torch.zeros(3, dtype=torch.int32))
        a.update(kw)
        return a
    assert rcp._validate_compact(CPU, **args()) == 3
    for kw, match in ((dict(keep=torch.zeros((3, 79), dtype=torch.uint8)), "keep must have shape"),
                      (dict(keep=torch.zeros((3, 80), dtype=torch.bool)), "uint8"),
                      (dict(keep=torch.zeros((80, 3), dtype=torch.uint8).t()), "contiguous"),
                      (dict(new_lens=torch.zeros(2, dtype=torch.int32)), "new_lens must have shape"),
                      (dict(block_table=torch.zeros((2, 5), dtype=torch.int32)), "rows"),
                      (dict(seq_lens=torch.zeros(3, dtype=torch.int64)), "int32")):
        with pytest.raises(ValueError, match=match):
            rcp._validate_compact(CPU, **args(**kw))


def test_a_mod_that_modifies_nothing_leaves_the_variant_to_the_plain_rule():
    for mod, modifies in ((ScoreMod(), False), (ScoreMod(softcap=2.0), True), (ScoreMod(window=1), True),
                          (ScoreMod(alibi_slopes=torch.zeros(4)), True),
                          (ScoreMod(prefix_lens=torch.zeros(1, dtype=torch.int32)), True),
                          (ScoreMod(row_begin=torch.zeros(1, dtype=torch.int32)), True),
                          # refused by the call itself: not the plain one
                          (ScoreMod(softcap=float("nan")), True), (ScoreMod(window=-1), True)):
        assert mod.modifies() is modifies
    cache = object.__new__(rcp.PagedCoeffCache)
    for pages in ("fp16", "int4"):
        cache.page_format = pages
        for rows, B in ((1, 1), (8, 1), (128, 1), (129, 1), (8, 4), (64, 4), (500, 4), (0, 0)):
            plain = cache._prefill_variant("auto", rows, B)
            assert cache._prefill_variant("auto", rows, B, ScoreMod()) == plain, (pages, rows, B)
            for v in ("rank", "reconstruct"):
                assert cache._prefill_variant(v, rows, B, ScoreMod(window=3)) == v
    cache.page_format = "fp16"
    assert cache._prefill_variant("auto", 128, 1, ScoreMod(window=3)) == "rank"
    assert cache._prefill_variant("auto", 8, 2, ScoreMod(window=3)) == "reconstruct"


def test_a_window_that_does_not_fit_is_refused_whenever_it_was_set():
    for bad in (2 ** 31, -2 ** 31 - 1, 2 ** 32 + 5, 2.5, float("nan")):
        with pytest.raises(ValueError):
            ScoreMod(window=bad)
        mod = ScoreMod(window=7)
        mod.window = bad
        with pytest.raises(ValueError):
            mod._args()
    mod = ScoreMod(window=7)
    mod.window = 2 ** 31 - 1
    assert mod._args().window == 2 ** 31 - 1 and ScoreMod(window=4096.0)._args().window == 4096
