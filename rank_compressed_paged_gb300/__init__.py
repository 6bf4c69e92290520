"""Rank-compressed paged attention on GB300 (sm_103a).

A thin Python layer over the C ABI of ``librcp.so`` (``include/rcp.h``): it passes torch
device pointers and the current CUDA stream through ctypes and does nothing else; every
step of the path runs in the library's CUDA kernels.

    cache = PagedCoeffCache(num_heads=32, head_dim=128, rank_k=64, rank_v=1024,
                            num_blocks=..., U_k=U, W_v=W)       # U, W: fp16 CUDA tensors
    cache.append_kv(k, v, slot_mapping)                          # project + scatter
    out = cache.decode_attn(q, block_table, seq_lens)            # [B][H][d] fp16
    out = cache.prefill_attn(q, cu_chunk_lens, block_table, seq_lens)
    out = cache.decode_attn(q, block_table, seq_lens, mod=ScoreMod(softcap=30.0, window=4096))
    child, = cache.fork_sequence(ids, length)                    # shares pages, copies the last
    new_lens = cache.compact_tokens(block_table, seq_lens, keep) # drops tokens in place
"""
from __future__ import annotations

import ctypes

from . import _lib
from ._lib import RcpError  # noqa: F401

BLOCK_SIZE = 16
RECONSTRUCT_MIN_CHUNK = 16   # mean chunk rows from which prefill_attn(variant="auto") rebuilds V


def _ptr(t) -> int:
    return t.data_ptr()


def _fits(shape, want) -> bool:
    if len(shape) != len(want):
        return False
    for have, e in zip(shape, want):
        if e is not None and have != e:
            return False
    return True


def _need(name: str, x, dtype, shape=None, device=None) -> None:
    """Check one tensor argument before its pointer crosses the C ABI, which cannot see
    dtypes, strides or devices: raise ValueError unless ``x`` is a contiguous tensor of
    ``dtype`` on ``device`` whose shape matches ``shape`` (None entries match any size)."""
    import torch
    if not isinstance(x, torch.Tensor):
        raise ValueError(f"{name} must be a torch.Tensor, got {type(x).__name__}")
    if x.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {x.dtype}")
    if shape is not None and not _fits(x.shape, shape):
        want = "[" + ", ".join("*" if e is None else str(e) for e in shape) + "]"
        raise ValueError(f"{name} must have shape {want}, got {list(x.shape)}")
    if not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and x.device != device:
        raise ValueError(f"{name} must be on {device}, got {x.device}")


def _validate_append(device, H: int, d: int, k, v, slot_mapping) -> int:
    """k, v: [T][H][d] fp16; slot_mapping: [T] int64.  Returns T."""
    import torch
    _need("slot_mapping", slot_mapping, torch.int64, (None,), device)
    T = int(slot_mapping.shape[0])
    _need("k", k, torch.float16, (T, H, d), device)
    _need("v", v, torch.float16, (T, H, d), device)
    return T


def _validate_decode(device, H: int, d: int, q, block_table, seq_lens, out) -> int:
    """q, out: [B][H][d] fp16; block_table: [>= B][max_blocks] int32; seq_lens: [B] int32.
    Returns B."""
    import torch
    _need("q", q, torch.float16, (None, H, d), device)
    B = int(q.shape[0])
    _need("seq_lens", seq_lens, torch.int32, (B,), device)
    _need("block_table", block_table, torch.int32, (None, None), device)
    if block_table.shape[0] < B or block_table.shape[1] < 1:
        raise ValueError(f"block_table needs at least {B} rows and one column, "
                         f"got {list(block_table.shape)}")
    _need("out", out, torch.float16, (B, H, d), device)
    return B


def _validate_prefill(device, H: int, d: int, q, cu_chunk_lens, block_table, seq_lens,
                      out) -> tuple[int, int]:
    """q, out: [rows][H][d] fp16; seq_lens: [B] int32; cu_chunk_lens: [B+1] int32;
    block_table: [>= B][max_blocks] int32.  Returns (rows, B)."""
    import torch
    _need("q", q, torch.float16, (None, H, d), device)
    rows = int(q.shape[0])
    _need("seq_lens", seq_lens, torch.int32, (None,), device)
    B = int(seq_lens.shape[0])
    _need("cu_chunk_lens", cu_chunk_lens, torch.int32, (B + 1,), device)
    _need("block_table", block_table, torch.int32, (None, None), device)
    if block_table.shape[0] < B or block_table.shape[1] < 1:
        raise ValueError(f"block_table needs at least {B} rows and one column, "
                         f"got {list(block_table.shape)}")
    _need("out", out, torch.float16, (rows, H, d), device)
    return rows, B


def _validate_workspace(device, ws) -> None:
    import torch
    _need("workspace", ws, torch.uint8, (None,), device)


def _validate_mod(device, H: int, B: int, rows: int, mod) -> None:
    """The tensors of a ScoreMod for B requests with ``rows`` query rows."""
    import torch
    if not isinstance(mod, ScoreMod):
        raise ValueError(f"mod must be a ScoreMod, got {type(mod).__name__}")
    if mod.alibi_slopes is not None:
        _need("alibi_slopes", mod.alibi_slopes, torch.float32, (H,), device)
    if mod.prefix_lens is not None:
        _need("prefix_lens", mod.prefix_lens, torch.int32, (B,), device)
    if mod.row_begin is not None:
        _need("row_begin", mod.row_begin, torch.int32, (rows,), device)


def _validate_compact(device, block_table, seq_lens, keep, new_lens) -> int:
    """block_table: [>= B][max_blocks] int32; seq_lens, new_lens: [B] int32; keep:
    [B][max_blocks * 16] uint8.  Returns B."""
    import torch
    _need("seq_lens", seq_lens, torch.int32, (None,), device)
    B = int(seq_lens.shape[0])
    _need("block_table", block_table, torch.int32, (None, None), device)
    if block_table.shape[0] < B or block_table.shape[1] < 1:
        raise ValueError(f"block_table needs at least {B} rows and one column, "
                         f"got {list(block_table.shape)}")
    _need("keep", keep, torch.uint8, (B, int(block_table.shape[1]) * BLOCK_SIZE), device)
    _need("new_lens", new_lens, torch.int32, (B,), device)
    return B


def _on_current(device) -> None:
    """The library launches on the current device, which has to be the cache's."""
    import torch
    if torch.cuda.current_device() != device.index:
        raise ValueError(f"the cache is on {device}, the current device is "
                         f"cuda:{torch.cuda.current_device()}")


def _ids(ids):
    if any(not -2**31 <= i < 2**31 for i in ids):   # ctypes would keep the low 32 bits
        raise ValueError("block ids must fit 32 bits")
    return (ctypes.c_int32 * max(len(ids), 1))(*ids)


def _stream(stream=None) -> int:
    import torch
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _empty_like(x, stream):
    """A result of a call on ``stream``: its memory is that stream's, because other streams' may
    still be read or written by what was queued there before it was freed."""
    import torch
    if stream is None:
        return torch.empty_like(x)
    with torch.cuda.stream(stream):
        return torch.empty_like(x)


def int4_page_bytes(num_heads: int, rank_k: int, rank_v: int):
    """Bytes of one 4-bit K page and one V page: the codes (two per byte), then the fp16
    scales (one per key row of a head, one per 64 value coefficients of a token)."""
    k = num_heads * BLOCK_SIZE * rank_k // 2 + num_heads * BLOCK_SIZE * 2
    v = BLOCK_SIZE * rank_v // 2 + BLOCK_SIZE * (rank_v // 64) * 2
    return k, v


class ScoreMod:
    """Score modifications of an attention call (include/rcp.h, rcp_score_mod): the row at
    position pos sees tokens t < prefix_lens[b], and tokens row_begin[row] <= t <= pos with
    t > pos - window, with scores softcap * tanh(s / softcap) - alibi_slopes[h] * |pos - t|.
    What is left at 0 / None takes no part.

    softcap: 0, or between 2**-10 and 2**10; window: tokens, the row's own included;
    alibi_slopes: [H] float32; prefix_lens: [B] int32; row_begin: [query rows] int32 (decode: [B],
    a document mask's start of the row's document).  The tensors are read by the kernels, on
    the call's stream.
    """

    __slots__ = ("softcap", "alibi_slopes", "window", "prefix_lens", "row_begin")

    def __init__(self, softcap: float = 0.0, alibi_slopes=None, window: int = 0,
                 prefix_lens=None, row_begin=None):
        self.softcap = float(softcap)
        self.alibi_slopes = alibi_slopes
        self.window = window
        self.prefix_lens = prefix_lens
        self.row_begin = row_begin
        self._window()

    def modifies(self) -> bool:
        """Whether a call with it differs from the plain one."""
        return (self.softcap != 0 or self.window != 0 or self.alibi_slopes is not None
                or self.prefix_lens is not None or self.row_begin is not None)

    def _window(self) -> int:
        w = int(self.window)
        if w != self.window or not -2**31 <= w < 2**31:   # ctypes would keep the low 32 bits
            raise ValueError(f"window must be a whole number of 32 bits, got {self.window}")
        return w

    def _args(self):
        def at(x):
            return None if x is None else _ptr(x)
        return _lib.ScoreModArgs(self.softcap, self._window(), at(self.alibi_slopes),
                                 at(self.prefix_lens), at(self.row_begin))


class PagedCoeffCache:
    """Paged low-rank coefficient cache on one GPU.

    Owns (as torch tensors) the K pages [num_blocks][H][16][r_k], V pages
    [num_blocks][16][R], the factors and a device error word; the
    library handle borrows their pointers.  page_format "fp16" stores fp16 coefficients,
    "fp8_e4m3" stores E4M3 codes (uint8 tensors), "int4" stores 4-bit codes with fp16
    scales as raw bytes (K pages [num_blocks][int4_page_bytes()[0]], V pages
    [num_blocks][int4_page_bytes()[1]], uint8).  A prefill on quantized pages first widens
    the pages it reads to fp16 in the workspace (the "auto" variant reconstructs).
    """

    def __init__(self, num_heads: int, head_dim: int, rank_k: int, rank_v: int,
                 num_blocks: int, U_k, W_v, k_pages=None, v_pages=None, device=None,
                 page_format: str = "fp16"):
        import torch
        lib = _lib.load()
        dev = U_k.device if device is None else torch.device(device)
        if dev.type != "cuda":
            raise ValueError(f"the cache lives on a CUDA device, got {dev}")
        if dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        formats = {"fp16": _lib.RCP_PAGES_FP16, "fp8_e4m3": _lib.RCP_PAGES_FP8_E4M3,
                   "int4": _lib.RCP_PAGES_INT4}
        if page_format not in formats:
            raise ValueError(f"unknown page_format {page_format!r}")
        fmt = formats[page_format]
        page_dtype = torch.float16 if fmt == _lib.RCP_PAGES_FP16 else torch.uint8
        self.page_format = page_format
        self.shape = dict(num_heads=num_heads, head_dim=head_dim, rank_k=rank_k, rank_v=rank_v)
        self.num_blocks = int(num_blocks)
        self.device = dev
        _need("U_k", U_k, torch.float16, (num_heads, rank_k, head_dim), dev)
        _need("W_v", W_v, torch.float16, (rank_v, num_heads * head_dim), dev)
        self.U_k = U_k
        self.W_v = W_v
        if fmt == _lib.RCP_PAGES_INT4:
            kb, vb = int4_page_bytes(num_heads, rank_k, rank_v)
            k_shape, v_shape = (num_blocks, kb), (num_blocks, vb)
        else:
            k_shape = (num_blocks, num_heads, BLOCK_SIZE, rank_k)
            v_shape = (num_blocks, BLOCK_SIZE, rank_v)
        if k_pages is None:
            k_pages = torch.zeros(k_shape, dtype=page_dtype, device=dev)
        if v_pages is None:
            v_pages = torch.zeros(v_shape, dtype=page_dtype, device=dev)
        _need("k_pages", k_pages, page_dtype, k_shape, dev)
        _need("v_pages", v_pages, page_dtype, v_shape, dev)
        self.k_pages = k_pages
        self.v_pages = v_pages
        self.dev_error = torch.zeros(1, dtype=torch.int32, device=dev)
        self._ws_bytes = {}
        self._cfg = _lib.CacheConfig(num_heads, head_dim, rank_k, rank_v, BLOCK_SIZE,
                                     self.num_blocks, fmt)
        h = ctypes.c_void_p()
        _lib.check("rcp_create_cache", lib.rcp_create_cache(
            ctypes.byref(self._cfg), _ptr(self.k_pages), _ptr(self.v_pages), _ptr(self.U_k),
            _ptr(self.W_v), _ptr(self.dev_error), ctypes.byref(h)))
        self._h = h
        self._lib = lib

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value:
            self._lib.rcp_destroy_cache(h)
            self._h = None

    # ------------------------------------------------------------------ block pool
    def alloc_blocks(self, n: int):
        ids = (ctypes.c_int32 * max(n, 1))()
        _lib.check("rcp_alloc_blocks", self._lib.rcp_alloc_blocks(self._h, n, ids))
        return [ids[i] for i in range(n)]

    def free_blocks(self, ids) -> None:
        """Takes one reference from each block, and returns it to the pool with its last.  A block
        listed twice is refused, whatever references it has: sequences that share pages are
        freed in a call each."""
        _lib.check("rcp_free_blocks", self._lib.rcp_free_blocks(self._h, len(ids), _ids(ids)))

    def num_free_blocks(self) -> int:
        n = ctypes.c_int64()
        _lib.check("rcp_num_free_blocks", self._lib.rcp_num_free_blocks(self._h, ctypes.byref(n)))
        return n.value

    def fork_blocks(self, ids) -> None:
        """One more reference to each block (free_blocks takes one away, and returns a block to
        the pool with its last)."""
        _lib.check("rcp_fork_blocks", self._lib.rcp_fork_blocks(self._h, len(ids), _ids(ids)))

    def block_refs(self, ids):
        """References to each block (0: free)."""
        refs = (ctypes.c_int32 * max(len(ids), 1))()
        _lib.check("rcp_block_refs",
                   self._lib.rcp_block_refs(self._h, len(ids), _ids(ids), refs))
        return [refs[i] for i in range(len(ids))]

    def fork_sequence(self, ids, length: int, children: int = 1, stream=None):
        """Forks the sequence of ``length`` tokens in blocks ``ids``: returns ``children`` lists
        of block ids, each sharing the full pages and holding a copy of the last, partly
        filled one (queued on the stream)."""
        _on_current(self.device)
        if not 0 <= length <= len(ids) * BLOCK_SIZE or not 0 <= children < 2**31:
            raise ValueError(f"{len(ids)} blocks hold no {length} tokens for {children} children")
        n = -(-int(length) // BLOCK_SIZE)
        out = (ctypes.c_int32 * max(n * int(children), 1))()
        _lib.check("rcp_fork_sequence", self._lib.rcp_fork_sequence(
            self._h, _ids(ids), len(ids), int(length), int(children), out, _stream(stream)))
        return [[out[c * n + j] for j in range(n)] for c in range(int(children))]

    def copy_blocks(self, pairs, stream=None) -> None:
        """Copies K and V pages: pairs [n][2] int32 on the cache's device, (source, destination)
        block ids; a pair with -1 in it is skipped."""
        import torch
        _need("pairs", pairs, torch.int32, (None, 2), self.device)
        _on_current(self.device)
        _lib.check("rcp_copy_blocks", self._lib.rcp_copy_blocks(
            self._h, _ptr(pairs), int(pairs.shape[0]), _stream(stream)))

    def compact_tokens(self, block_table, seq_lens, keep, new_lens=None, stream=None):
        """Drops tokens in place: token t of request b stays if keep[b][t] != 0, the kept ones
        move to the front of the request's pages.  keep: [B][max_blocks * 16] uint8.  Returns
        the new lengths [B] int32 (``new_lens``, which must not be ``seq_lens``); the pages past
        them may then be freed."""
        if new_lens is None:
            new_lens = _empty_like(seq_lens, stream)
        B = _validate_compact(self.device, block_table, seq_lens, keep, new_lens)
        _on_current(self.device)
        _lib.check("rcp_compact_tokens", self._lib.rcp_compact_tokens(
            self._h, _ptr(block_table), int(block_table.shape[1]), _ptr(seq_lens), _ptr(keep), B,
            _ptr(new_lens), _stream(stream)))
        return new_lens

    # ------------------------------------------------------------------ workspace
    def workspace_bytes(self, rows: int) -> int:
        need = self._ws_bytes.get(rows)   # a function of the cache's shape alone
        if need is None:
            n = ctypes.c_size_t()
            _lib.check("rcp_workspace_size",
                       self._lib.rcp_workspace_size(self._h, rows, ctypes.byref(n)))
            need = n.value
            if len(self._ws_bytes) < 4096:
                self._ws_bytes[rows] = need
        return need

    def workspace(self, rows: int, need: int | None = None, stream=None):
        """Scratch for a call of ``rows`` query rows (or of ``need`` bytes) on ``stream``, from
        torch's allocator: a call that is given none takes one and gives it back, which hands its
        memory to nothing but later work of that stream (of the graph, where it is captured).
        Calls on two streams may overlap and have one each; none is kept between calls."""
        import torch
        if stream is not None and stream != torch.cuda.current_stream():
            with torch.cuda.stream(stream):
                return self.workspace(rows, need)
        need = self.workspace_bytes(rows) if need is None else need
        return torch.empty(need, dtype=torch.uint8, device=self.device)

    def _scratch(self, workspace, rows: int, stream):
        """The caller's workspace, checked, or one for this call."""
        if workspace is None:
            return self.workspace(rows, stream=stream)
        _validate_workspace(self.device, workspace)
        return workspace

    def reconstruct_workspace_bytes(self, rows: int, batch: int, max_blocks_per_seq: int) -> int:
        n = ctypes.c_size_t()
        _lib.check("rcp_prefill_reconstruct_workspace_size",
                   self._lib.rcp_prefill_reconstruct_workspace_size(
                       self._h, rows, batch, max_blocks_per_seq, ctypes.byref(n)))
        return n.value

    def prefill_crossover_rows(self) -> int:
        n = ctypes.c_int32()
        _lib.check("rcp_prefill_crossover_rows",
                   self._lib.rcp_prefill_crossover_rows(self._h, ctypes.byref(n)))
        return n.value

    def read_device_error(self) -> int:
        return int(self.dev_error.item())

    def clear_device_error(self) -> None:
        self.dev_error.zero_()

    def set_profile_events(self, start=None, stop=None) -> None:
        """Record torch.cuda.Event pair around the split-K attention kernel (None: off)."""
        def handle(ev):
            if ev is None:
                return None
            if not ev.cuda_event:
                ev.record()            # torch creates the CUDA event lazily
            return ev.cuda_event
        _lib.check("rcp_set_profile_events",
                   self._lib.rcp_set_profile_events(self._h, handle(start), handle(stop)))

    # ------------------------------------------------------------------ hot path
    def append_kv(self, k, v, slot_mapping, stream=None) -> None:
        """k, v: [T][H][d] fp16; slot_mapping: [T] int64 (all on the cache's device)."""
        H, d = self.shape["num_heads"], self.shape["head_dim"]
        T = _validate_append(self.device, H, d, k, v, slot_mapping)
        _lib.check("rcp_append_kv", self._lib.rcp_append_kv(
            self._h, _ptr(k), _ptr(v), _ptr(slot_mapping), T, _stream(stream)))

    def _decode_mod(self, mod, app, q, block_table, seq_lens, out, ws, stream):
        """rcp_decode_step_mod; app: (k, v, slot_mapping), or None for the attention alone."""
        H, B = self.shape["num_heads"], int(seq_lens.shape[0])
        _validate_mod(self.device, H, B, B, mod)
        _on_current(self.device)
        k, v, slots, T = (None, None, None, 0) if app is None else (
            _ptr(app[0]), _ptr(app[1]), _ptr(app[2]), int(app[2].shape[0]))
        _lib.check("rcp_decode_step_mod", self._lib.rcp_decode_step_mod(
            self._h, k, v, slots, T, _ptr(q), _ptr(block_table), int(block_table.shape[1]),
            _ptr(seq_lens), B, ctypes.byref(mod._args()), _ptr(out), _ptr(ws),
            ws.numel() * ws.element_size(), _stream(stream)))

    def decode_attn(self, q, block_table, seq_lens, out=None, workspace=None, stream=None,
                    mod=None):
        """q: [B][H][d] fp16; block_table: [B][max_blocks] int32; seq_lens: [B] int32; mod: None
        or a ScoreMod."""
        if out is None:
            out = _empty_like(q, stream)
        H, d = self.shape["num_heads"], self.shape["head_dim"]
        B = _validate_decode(self.device, H, d, q, block_table, seq_lens, out)
        ws = self._scratch(workspace, B, stream)
        if mod is not None:
            self._decode_mod(mod, None, q, block_table, seq_lens, out, ws, stream)
            return out
        _lib.check("rcp_decode_attn", self._lib.rcp_decode_attn(
            self._h, _ptr(q), _ptr(block_table), int(block_table.shape[1]), _ptr(seq_lens), B,
            _ptr(out), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))
        return out

    def decode_attn_sparse(self, q, block_table, seq_lens, skip_threshold: float,
                           page_kept=None, out=None, workspace=None, stream=None):
        """Block-sparse decode: as decode_attn, but a page is left out (its values unread,
        its tokens out of the softmax) when every head's largest weight in it is below
        ``skip_threshold`` times that head's running maximum weight.  ``page_kept``: None
        or a [B][max_blocks] uint8 tensor that receives 1 / 0 per page read / left out."""
        import torch
        if out is None:
            out = _empty_like(q, stream)
        H, d = self.shape["num_heads"], self.shape["head_dim"]
        B = _validate_decode(self.device, H, d, q, block_table, seq_lens, out)
        if page_kept is not None:
            _need("page_kept", page_kept, torch.uint8, tuple(block_table.shape), self.device)
        ws = self._scratch(workspace, B, stream)
        _lib.check("rcp_decode_attn_sparse", self._lib.rcp_decode_attn_sparse(
            self._h, _ptr(q), _ptr(block_table), int(block_table.shape[1]), _ptr(seq_lens), B,
            float(skip_threshold), _ptr(page_kept) if page_kept is not None else None,
            _ptr(out), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))
        return out

    def decode_step(self, k, v, slot_mapping, q, block_table, seq_lens, out=None, workspace=None,
                    stream=None, mod=None):
        """append_kv(k, v, slot_mapping) then decode_attn(q, ..., mod=mod), queued as one step."""
        if out is None:
            out = _empty_like(q, stream)
        H, d = self.shape["num_heads"], self.shape["head_dim"]
        _validate_append(self.device, H, d, k, v, slot_mapping)
        B = _validate_decode(self.device, H, d, q, block_table, seq_lens, out)
        ws = self._scratch(workspace, B, stream)
        if mod is not None:
            self._decode_mod(mod, (k, v, slot_mapping), q, block_table, seq_lens, out, ws, stream)
            return out
        _lib.check("rcp_decode_step", self._lib.rcp_decode_step(
            self._h, _ptr(k), _ptr(v), _ptr(slot_mapping), int(slot_mapping.shape[0]), _ptr(q),
            _ptr(block_table), int(block_table.shape[1]), _ptr(seq_lens), B, _ptr(out), _ptr(ws),
            ws.numel() * ws.element_size(), _stream(stream)))
        return out

    def _prefill_variant(self, variant: str, rows: int, B: int, mod=None) -> str:
        if variant == "auto" and isinstance(mod, ScoreMod) and mod.modifies():
            # one 128-row tile is 128 rank-space CTAs, one wave of the SMs; measured, rank space
            # against reconstruction in us, 1 to 128 rows of one request: capped behind 777 tokens
            # 36-39 / 39-41, behind 4096 85-96 / 100-111, behind 32768 512-594 / 628-722, a window
            # of 1024 35-37 / 43-44; two requests 64-66 / 46-47, 178-182 / 137-140, 1136-1175 /
            # 877-907 and 62-64 / 44-46 (the small shape: within 8 us of each other, or 8 %)
            variant = "rank" if self.page_format == "fp16" and B == 1 and rows <= 128 else "reconstruct"
        if variant == "auto":
            variant = "reconstruct" if (self.page_format != "fp16" or
                                        (B > 0 and rows >= B * RECONSTRUCT_MIN_CHUNK)) else "rank"
        if variant not in ("rank", "reconstruct"):
            raise ValueError(f"unknown prefill variant {variant!r}")
        return variant

    def _prefill_scratch(self, workspace, variant: str, rows: int, B: int, mb: int, stream):
        # quantized pages are widened into the workspace first (both variants)
        if workspace is not None or (variant == "rank" and self.page_format == "fp16"):
            return self._scratch(workspace, rows, stream)
        return self.workspace(rows, self.reconstruct_workspace_bytes(rows, B, mb), stream)

    def _prefill_mod(self, mod, app, q, cu_chunk_lens, block_table, seq_lens, out, ws, stream,
                     variant: str):
        """rcp_prefill_step_mod; app: (k, v, slot_mapping), or None for the attention alone."""
        H, B, rows = self.shape["num_heads"], int(seq_lens.shape[0]), int(q.shape[0])
        _validate_mod(self.device, H, B, rows, mod)
        _on_current(self.device)
        k, v, slots, T = (None, None, None, 0) if app is None else (
            _ptr(app[0]), _ptr(app[1]), _ptr(app[2]), int(app[2].shape[0]))
        _lib.check("rcp_prefill_step_mod", self._lib.rcp_prefill_step_mod(
            self._h, k, v, slots, T, _ptr(q), _ptr(cu_chunk_lens), rows, _ptr(block_table),
            int(block_table.shape[1]), _ptr(seq_lens), B, 1 if variant == "reconstruct" else 0,
            ctypes.byref(mod._args()), _ptr(out), _ptr(ws), ws.numel() * ws.element_size(),
            _stream(stream)))

    def prefill_attn(self, q, cu_chunk_lens, block_table, seq_lens, out=None, workspace=None,
                     stream=None, variant: str = "auto", mod=None):
        """q: [sum chunk][H][d] fp16; cu_chunk_lens: [B+1] int32; seq_lens include the chunk;
        mod: None or a ScoreMod.

        variant: "rank" (joint-coefficient contraction per head), "reconstruct" (dense values
        C_v W_v rebuilt once per key), or "auto": reconstruct when chunks average at least
        RECONSTRUCT_MIN_CHUNK rows.  The multiply-add count favours reconstruction above
        prefill_crossover_rows() (147 for R = 1024, d = 128); measured on GB300 it is the
        faster variant from 16-row chunks on (priors 4096 to 32768), because a chunk shorter
        than one 128-row tile costs the rank-space kernel a whole tile per R slice.  Under a mod
        that modifies anything "auto" is rank for one request of up to 128 rows on fp16 pages,
        else reconstruct."""
        if out is None:
            out = _empty_like(q, stream)
        H, d = self.shape["num_heads"], self.shape["head_dim"]
        rows, B = _validate_prefill(self.device, H, d, q, cu_chunk_lens, block_table, seq_lens,
                                    out)
        mb = int(block_table.shape[1])
        variant = self._prefill_variant(variant, rows, B, mod)
        ws = self._prefill_scratch(workspace, variant, rows, B, mb, stream)
        if mod is not None:
            self._prefill_mod(mod, None, q, cu_chunk_lens, block_table, seq_lens, out, ws, stream,
                              variant)
            return out
        if variant == "rank":
            fn, name = self._lib.rcp_prefill_attn, "rcp_prefill_attn"
        else:
            fn, name = self._lib.rcp_prefill_attn_reconstruct, "rcp_prefill_attn_reconstruct"
        _lib.check(name, fn(
            self._h, _ptr(q), _ptr(cu_chunk_lens), rows, _ptr(block_table), mb, _ptr(seq_lens), B,
            _ptr(out), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))
        return out

    def prefill_step(self, k, v, slot_mapping, q, cu_chunk_lens, block_table, seq_lens,
                     out=None, workspace=None, stream=None, variant: str = "auto", mod=None):
        """append_kv(k, v, slot_mapping) then prefill_attn(q, cu_chunk_lens, ..., mod=mod), queued
        as one step (the chunk's query projection shares the append's launch).  Arguments and
        variant choice as the two calls."""
        if out is None:
            out = _empty_like(q, stream)
        H, d = self.shape["num_heads"], self.shape["head_dim"]
        T = _validate_append(self.device, H, d, k, v, slot_mapping)
        rows, B = _validate_prefill(self.device, H, d, q, cu_chunk_lens, block_table, seq_lens,
                                    out)
        mb = int(block_table.shape[1])
        variant = self._prefill_variant(variant, rows, B, mod)
        ws = self._prefill_scratch(workspace, variant, rows, B, mb, stream)
        if mod is not None:
            self._prefill_mod(mod, (k, v, slot_mapping), q, cu_chunk_lens, block_table, seq_lens,
                              out, ws, stream, variant)
            return out
        _lib.check("rcp_prefill_step", self._lib.rcp_prefill_step(
            self._h, _ptr(k), _ptr(v), _ptr(slot_mapping), T, _ptr(q), _ptr(cu_chunk_lens), rows,
            _ptr(block_table), mb, _ptr(seq_lens), B, 1 if variant == "reconstruct" else 0,
            _ptr(out), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))
        return out
