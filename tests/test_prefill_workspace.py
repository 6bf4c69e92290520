"""Workspace of a prefill: what only differential heads take is asked for by their calls alone."""
import ctypes

import numpy as np
import pytest
import torch

import rank_compressed_paged_gb300 as rcp
import workloads as wl
from rank_compressed_paged_gb300 import _lib

FORMATS = {"fp16": _lib.RCP_PAGES_FP16, "fp8_e4m3": _lib.RCP_PAGES_FP8_E4M3, "int4": _lib.RCP_PAGES_INT4}


class Handle(rcp.PagedCoeffCache):
    """A cache over addresses that nothing reads, whose scratch is a number of bytes."""

    def __init__(self, pages):
        from rank_compressed_paged_gb300 import build
        build.build()
        self.page_format, self._lib, self._ws_bytes, self._h = pages, _lib.load(), {}, ctypes.c_void_p()
        cfg = _lib.CacheConfig(32, 128, 64, 1024, 16, 100, FORMATS[pages])
        assert self._lib.rcp_create_cache(ctypes.byref(cfg), 0x10000, 0x20000, 0x30000, 0x40000, 0x50000,
                                          ctypes.byref(self._h)) == _lib.RCP_OK

    def workspace(self, rows, need=None, stream=None):
        return self.workspace_bytes(rows) if need is None else need


def test_a_plain_prefill_takes_no_room_for_a_difference():
    """V^, and fp16 copies of quantized pages, by their sizes; on 4-bit pages a difference takes the
    keys' scales (fp32) and the values' second parts besides."""
    rows, B, mb = 70, 3, 400
    pages = B * mb
    diff = rcp.DiffHeads(torch.zeros(16))
    caches = {f: Handle(f) for f in FORMATS}
    size = {f: c._prefill_scratch(None, "reconstruct", rows, B, mb, None) for f, c in caches.items()}
    with_diff = {f: c._prefill_scratch(None, "reconstruct", rows, B, mb, None, diff)
                 for f, c in caches.items()}
    wide = 2 * pages * 16 * (32 * 64 + 1024) + (4 * pages + 255) // 256 * 256
    assert size["int4"] == size["fp8_e4m3"] == size["fp16"] + wide
    assert with_diff["fp16"] == size["fp16"] and with_diff["fp8_e4m3"] == size["fp8_e4m3"]
    assert with_diff["int4"] - size["int4"] == pages * 16 * (4 * 32 + 2 * 1024)
    for f, c in caches.items():      # what the size without options tells stays enough for every call
        assert c.reconstruct_workspace_bytes(rows, B, mb) == with_diff[f]
        assert c.reconstruct_workspace_bytes(rows, B, mb, diff=False) == size[f]


def test_sizes_by_options():
    c = Handle("int4")
    n = ctypes.c_size_t()

    def need(options, rows=70, batch=3, mb=400, out=ctypes.byref(n)):
        return c._lib.rcp_prefill_step_workspace_size(c._h, rows, batch, mb, options, out), n.value
    plain = need(None)
    diff = _lib.StepOptions(None, None, ctypes.pointer(_lib.DiffHeadsArgs(0x1000, None, 0.0, 1.0)))
    rot = _lib.StepOptions(None, ctypes.pointer(_lib.RotaryArgs(0x1000, 10, 32, 0, 0x2000, 0x3000)), None)
    assert plain[0] == _lib.RCP_OK and need(ctypes.byref(rot)) == plain
    assert need(ctypes.byref(diff)) == (_lib.RCP_OK, c.reconstruct_workspace_bytes(70, 3, 400)) != plain
    for bad in (dict(rows=-1), dict(batch=-1), dict(mb=-1), dict(out=None)):
        assert need(None, **bad)[0] == _lib.RCP_ERR_INVALID_ARG
    assert c._lib.rcp_prefill_step_workspace_size(None, 1, 1, 1, None, ctypes.byref(n)) \
        == _lib.RCP_ERR_INVALID_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("pages", sorted(FORMATS))
@pytest.mark.parametrize("variant", ["rank", "reconstruct"])
def test_a_plain_prefill_runs_in_its_own_workspace(pages, variant):
    from tests.gpu_util import t
    from tests.mod_util import cache_of, encode
    shape = wl.SHAPES["tiny"]
    inp = wl.make_prefill_inputs(shape, [40, 0, 300], [3, 33, 250], seed=701, fill=0.0)
    c = inp.cache
    cache = cache_of(pages, shape, inp.U_k, inp.W_v, *encode(pages, c.k_pages, c.v_pages))
    table = np.full((3, 1000), -1, np.int32)     # wide enough for the pages to set the size
    table[:, :c.block_table.shape[1]] = c.block_table
    args = t(inp.q), t(inp.cu_chunk_lens), t(table), t(inp.seq_lens_after)
    want = cache.prefill_attn(*args, variant=variant)
    need = cache.reconstruct_workspace_bytes(inp.q.shape[0], 3, 1000, diff=False)
    guard = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    got = cache.prefill_attn(*args, variant=variant, workspace=guard[:need])
    assert torch.equal(got, want) and torch.all(guard[need:] == 0xA5)
    diff = rcp.DiffHeads(t(np.zeros(shape["num_heads"] // 2, np.float32)))
    if pages == "int4" and variant == "reconstruct":
        with pytest.raises(rcp.RcpError):
            cache.prefill_attn(*args, workspace=guard[:need], diff=diff)
