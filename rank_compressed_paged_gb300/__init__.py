"""Rank-compressed paged attention on GB300 (sm_103a).

A thin Python layer over the C ABI of ``librcp.so`` (``include/rcp.h``): it passes torch
device pointers and the current CUDA stream through ctypes and does nothing else; every
step of the path runs in the library's CUDA kernels.

    cache = PagedCoeffCache(num_heads=32, head_dim=128, rank_k=64, rank_v=1024,
                            num_blocks=..., U_k=U, W_v=W)       # U, W: fp16 CUDA tensors
    cache.append_kv(k, v, slot_mapping)                          # project + scatter
    cache.append_kv(k, v, slot_mapping, rotary=Rotary(table, k_positions=pos))   # rotated keys
    out = cache.decode_attn(q, block_table, seq_lens)            # [B][H][d] fp16
    out = cache.prefill_attn(q, cu_chunk_lens, block_table, seq_lens)
    out = cache.decode_attn(q, block_table, seq_lens, mod=ScoreMod(softcap=30.0, window=4096))
    out = cache.decode_attn(q, block_table, seq_lens, diff=DiffHeads(lam, norm_weight=w))
    child, = cache.fork_sequence(ids, length)                    # shares pages, copies the last
    new_lens = cache.compact_tokens(block_table, seq_lens, keep) # drops tokens in place
    scores, tokens, parents, ended = beam_select(logits, scores, eos=2)    # best of beams x vocabulary
    block_table, seq_lens = cache.reorder_sequences(block_table, seq_lens, parents.view(-1), spare)
"""
from __future__ import annotations

import ctypes
import operator

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
    if (x.dtype is dtype and (shape is None or x.shape == shape or _fits(x.shape, shape))
            and x.is_contiguous() and (device is None or x.device == device)):
        return
    if x.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {x.dtype}")
    if shape is not None and not _fits(x.shape, shape):
        want = "[" + ", ".join("*" if e is None else str(e) for e in shape) + "]"
        raise ValueError(f"{name} must have shape {want}, got {list(x.shape)}")
    if not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and x.device != device:
        raise ValueError(f"{name} must be on {device}, got {x.device}")


def _plain(device, dtype, *tensors) -> bool:
    """Whether every one is a contiguous tensor of ``dtype`` on ``device`` (a CUDA one): what _need
    checks beside the shape, at once."""
    import torch
    index = device.index
    for x in tensors:
        if not (isinstance(x, torch.Tensor) and x.dtype is dtype and x.get_device() == index
                and x.is_contiguous()):
            return False
    return True


def _validate_append(device, H: int, d: int, k, v, slot_mapping) -> int:
    """k, v: [T][H][d] fp16; slot_mapping: [T] int64.  Returns T."""
    import torch
    if _plain(device, torch.float16, k, v) and _plain(device, torch.int64, slot_mapping):
        T = slot_mapping.shape[0] if slot_mapping.dim() == 1 else -1
        if k.shape == v.shape == (T, H, d):
            return T
    _need("slot_mapping", slot_mapping, torch.int64, (None,), device)
    T = int(slot_mapping.shape[0])
    _need("k", k, torch.float16, (T, H, d), device)
    _need("v", v, torch.float16, (T, H, d), device)
    return T


def _validate_decode(device, H: int, d: int, q, block_table, seq_lens, out) -> int:
    """q, out: [B][H][d] fp16; block_table: [>= B][max_blocks] int32; seq_lens: [B] int32.
    Returns B."""
    import torch
    if _plain(device, torch.float16, q, out) and _plain(device, torch.int32, block_table, seq_lens):
        B = seq_lens.shape[0] if seq_lens.dim() == 1 else -1
        if (q.shape == out.shape == (B, H, d) and block_table.dim() == 2
                and block_table.shape[0] >= B and block_table.shape[1] >= 1):
            return B
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


def _validate_rotary(device, d: int, rotary, tokens=None, rows=None) -> None:
    """The tensors of a Rotary for a call with ``tokens`` new tokens and ``rows`` query rows (None:
    the call has none, and their positions are not looked at)."""
    import torch
    if not isinstance(rotary, Rotary):
        raise ValueError(f"rotary must be a Rotary, got {type(rotary).__name__}")
    table, kp, qp = rotary.table, rotary.k_positions, rotary.q_positions
    if (_plain(device, torch.float32, table) and table.dim() == 2
            and 1 <= table.shape[0] < 2**31 and 16 <= table.shape[1] <= d and table.shape[1] % 16 == 0
            and (tokens is None or kp is None
                 or (_plain(device, torch.int32, kp) and kp.shape == (tokens,)))
            and (rows is None or qp is None
                 or (_plain(device, torch.int32, qp) and qp.shape == (rows,)))):
        return
    _need("table", rotary.table, torch.float32, (None, None), device)
    n, rot = rotary.table.shape
    if n < 1 or n >= 2**31 or rot < 16 or rot % 16 or rot > d:
        raise ValueError(f"table must have shape [positions, a multiple of 16 up to {d}], got "
                         f"{list(rotary.table.shape)}")
    if tokens is not None and rotary.k_positions is not None:
        _need("k_positions", rotary.k_positions, torch.int32, (tokens,), device)
    if rows is not None and rotary.q_positions is not None:
        _need("q_positions", rotary.q_positions, torch.int32, (rows,), device)


def _validate_diff(device, H: int, d: int, diff) -> None:
    """The tensors of a DiffHeads."""
    import torch
    if not isinstance(diff, DiffHeads):
        raise ValueError(f"diff must be a DiffHeads, got {type(diff).__name__}")
    _need("lam", diff.lam, torch.float32, (H // 2,), device)
    if diff.norm_weight is not None:
        _need("norm_weight", diff.norm_weight, torch.float32, (2 * d,), device)


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


def _validate_reorder(device, block_table, seq_lens, parents, tail_blocks, new_table,
                      new_lens) -> tuple[int, int]:
    """block_table: [>= rows][max_blocks] int32; seq_lens: [rows] int32; parents, tail_blocks,
    new_lens: [n] int32; new_table: [>= n][max_blocks] int32.  Returns (rows, n)."""
    import torch
    if (_plain(device, torch.int32, seq_lens, parents, block_table, tail_blocks, new_table, new_lens)
            and seq_lens.dim() == parents.dim() == 1 and block_table.dim() == new_table.dim() == 2
            and parents.shape == tail_blocks.shape == new_lens.shape):
        rows, n = seq_lens.shape[0], parents.shape[0]
        (have, mb), (new, new_mb) = block_table.shape, new_table.shape
        if have >= rows and mb >= 1 and new >= n and new_mb == mb and max(rows, n, mb) < 2**31:
            return rows, n
    _need("seq_lens", seq_lens, torch.int32, (None,), device)
    _need("parents", parents, torch.int32, (None,), device)
    rows, n = int(seq_lens.shape[0]), int(parents.shape[0])
    _need("block_table", block_table, torch.int32, (None, None), device)
    mb = int(block_table.shape[1])
    if block_table.shape[0] < rows or mb < 1:
        raise ValueError(f"block_table needs at least {rows} rows and one column, "
                         f"got {list(block_table.shape)}")
    _need("tail_blocks", tail_blocks, torch.int32, (n,), device)
    _need("new_table", new_table, torch.int32, (None, mb), device)
    if new_table.shape[0] < n:
        raise ValueError(f"new_table needs at least {n} rows, got {list(new_table.shape)}")
    _need("new_lens", new_lens, torch.int32, (n,), device)
    if max(rows, n, mb) >= 2**31:
        raise ValueError(f"{rows} rows to {n} rows of {mb} blocks are too many for a call")
    return rows, n


def _validate_beams(logits, scores, eos) -> tuple[int, int, int, int]:
    """logits: [B][K][V] fp16, bf16 or fp32, starting on 16 bytes; scores: [B][K] fp32.  Returns
    (B, K, V, dtype)."""
    import torch
    code = _logits_code(logits.dtype) if isinstance(logits, torch.Tensor) else None
    if (code is not None and logits.dim() == 3 and logits.is_contiguous() and not _ptr(logits) & 15
            and isinstance(scores, torch.Tensor) and scores.dtype is torch.float32
            and scores.is_contiguous() and scores.get_device() == logits.get_device() >= 0):
        B, K, V = logits.shape
        if scores.shape == (B, K) and (eos is None or (type(eos) is int and 0 <= eos < V)):
            return B, K, V, code
    if code is None:
        raise ValueError("logits must be a torch.Tensor of float16, bfloat16 or float32, got "
                         f"{getattr(logits, 'dtype', type(logits).__name__)}")
    _need("logits", logits, logits.dtype, (None, None, None))
    B, K, V = logits.shape
    if _ptr(logits) & 15:
        raise ValueError("logits must start on a 16-byte boundary (a slice of a larger tensor may not: "
                         f"clone it), got address {_ptr(logits):#x}")
    _need("scores", scores, torch.float32, (B, K), logits.device)
    if eos is not None and not (hasattr(type(eos), "__index__") and 0 <= operator.index(eos) < V):
        raise ValueError(f"eos must be a token of the vocabulary of {V}, got {eos}")
    return B, K, V, code


def _on_current(device) -> None:
    """The library launches on the current device, which has to be the cache's."""
    import torch
    if torch._C._cuda_getDevice() != device.index:
        raise ValueError(f"the call's tensors are on {device}, the current device is "
                         f"cuda:{torch.cuda.current_device()}")


def _ids(ids):
    if any(not -2**31 <= i < 2**31 for i in ids):   # ctypes would keep the low 32 bits
        raise ValueError("block ids must fit 32 bits")
    return (ctypes.c_int32 * max(len(ids), 1))(*ids)


def _stream(stream=None) -> int:
    import torch
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _empty_like(x, stream, dtype=None):
    """A result of a call on ``stream``: its memory is that stream's, because other streams' may
    still be read or written by what was queued there before it was freed."""
    import torch
    if stream is None:
        return torch.empty_like(x, dtype=dtype)
    with torch.cuda.stream(stream):
        return torch.empty_like(x, dtype=dtype)


def _empty(shape, dtype, device, stream):
    """As _empty_like, for a shape."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


_logits_types = {}   # torch dtype -> RCP_LOGITS_*
_beam_bytes = {}     # (B, K, V, dtype) -> workspace bytes


def _logits_code(dtype):
    """RCP_LOGITS_* of a torch dtype, or None."""
    if not _logits_types:
        import torch
        _logits_types.update({torch.float16: _lib.RCP_LOGITS_FP16,
                              torch.bfloat16: _lib.RCP_LOGITS_BF16,
                              torch.float32: _lib.RCP_LOGITS_FP32})
    return _logits_types.get(dtype)


def beam_workspace_bytes(batch: int, beams: int, vocab: int, dtype) -> int:
    """Bytes of workspace of a beam_select on logits [batch][beams][vocab] of a torch dtype."""
    key = (batch, beams, vocab, dtype)
    need = _beam_bytes.get(key)   # a function of the shape alone
    if need is None:
        code = _logits_code(dtype)
        if code is None:
            raise ValueError(f"logits must be of float16, bfloat16 or float32, got {dtype}")
        if max(batch, beams, vocab) >= 2**31:
            raise ValueError(f"[{batch}, {beams}, {vocab}] is too large for a selection")
        n = ctypes.c_size_t()
        _lib.check("rcp_beam_workspace_size", _lib.load().rcp_beam_workspace_size(
            batch, beams, vocab, code, ctypes.byref(n)))
        need = n.value
        if len(_beam_bytes) < 4096:
            _beam_bytes[key] = need
    return need


def beam_select(logits, scores, eos=None, workspace=None, stream=None):
    """Beam search's selection.  logits: [B][K][V] fp16, bf16 or fp32, as the model left them, starting
    on a 16-byte boundary; scores: [B][K] fp32, the beams' sums of log-probabilities (-inf: a dead
    beam, such as all but the first in the first step).  A candidate (i, t) has the total scores[i]
    + log_softmax(logits[i])[t].  Returns (next_scores [B][K] fp32, tokens [B][K] int32, parents
    [B][K] int32, ended [B][K] fp32): the best K candidates that do not end in token ``eos``, best
    first, equal totals in the order of (i, t), with parents as rows b * K + i of the batch (for
    reorder_sequences); and for each beam the total of its end, if fewer than K of all candidates
    come before it, else -inf.  Missing candidates are (-inf, -1, -1).  K up to 32, V up to
    2**18."""
    import torch
    B, K, V, dtype = _validate_beams(logits, scores, eos)
    dev = logits.device
    if dev.type != "cuda":
        raise ValueError(f"logits must be on a CUDA device, got {dev}")
    _on_current(dev)
    lib = _lib.load()
    need = beam_workspace_bytes(B, K, V, logits.dtype)
    if workspace is None:
        workspace = _empty(need, torch.uint8, dev, stream)
    else:
        _validate_workspace(dev, workspace)
    next_scores, ended = _empty_like(scores, stream), _empty_like(scores, stream)
    tokens = _empty_like(scores, stream, torch.int32)
    parents = _empty_like(scores, stream, torch.int32)
    _lib.check("rcp_beam_select", lib.rcp_beam_select(
        _ptr(logits), dtype, _ptr(scores), B, K, V, -1 if eos is None else int(eos),
        _ptr(next_scores), _ptr(tokens), _ptr(parents), _ptr(ended), _ptr(workspace),
        workspace.numel(), _stream(stream)))
    return next_scores, tokens, parents, ended


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


class DiffHeads:
    """Differential attention (include/rcp.h, rcp_diff_heads): heads 2 p and 2 p + 1 are two maps,
    softmax(s_2p) - lam[p] softmax(s_2p+1) is applied to the values of both heads, and where
    norm_weight is given the pair's 2 d outputs are divided by their root mean square and take
    the weight; all times ``scale``.

    lam: [H / 2] float32; norm_weight: None or [2 d] float32, the same for every pair; eps: added to
    the mean square.  The tensors are read by the kernels, on the call's stream.  A prefill
    runs in the reconstructing variant.
    """

    __slots__ = ("lam", "norm_weight", "eps", "scale")

    def __init__(self, lam, norm_weight=None, eps: float = 1e-5, scale: float = 1.0):
        self.lam = lam
        self.norm_weight = norm_weight
        self.eps = float(eps)
        self.scale = float(scale)

    def _args(self):
        return _lib.DiffHeadsArgs(_ptr(self.lam),
                                  None if self.norm_weight is None else _ptr(self.norm_weight),
                                  self.eps, self.scale)


def rotary_table(num_positions: int, rot_dim: int, base: float = 10000.0, scale: float = 1.0,
                 device=None):
    """A table for Rotary: row pos holds cos(a_j), then sin(a_j), with a_j = pos / scale *
    base**(-2 j / rot_dim), j < rot_dim / 2.  Angles in 64 bits (in 32 those of far positions are
    off by whole units of the last place of pos), stored in fp32."""
    import torch
    m = rot_dim // 2
    freq = base ** (-torch.arange(m, dtype=torch.float64, device=device) / m)
    a = torch.arange(num_positions, dtype=torch.float64, device=device)[:, None] / scale * freq
    return torch.cat([a.cos(), a.sin()], 1).to(torch.float32)


class Rotary:
    """Rotation of positions (include/rcp.h, rcp_rotary), applied to new keys before they are
    projected into the cache, and to the queries that meet them: pair j of a head's elements turns
    by the angle whose cosine and sine are table[pos][j] and table[pos][rot_dim / 2 + j].  Pairs
    are (j, j + rot_dim / 2), or (2 j, 2 j + 1) where ``interleaved``; elements from rot_dim on stay.

    table: [positions][rot_dim] float32 (rotary_table makes one), rot_dim a multiple of 16 up to
    the head dim; k_positions: [T] int32, the new tokens' positions, None: keys come as they are;
    q_positions: [query rows] int32, None: queries stay.  Positions are the model's, whatever
    place a token has in the cache.  One outside the table sets a device error bit: its token is
    not appended, its query counts as zero.  The tensors are read by the kernels, on the call's
    stream.
    """

    __slots__ = ("table", "k_positions", "q_positions", "interleaved")

    def __init__(self, table, k_positions=None, q_positions=None, interleaved: bool = False):
        self.table = table
        self.k_positions = k_positions
        self.q_positions = q_positions
        self.interleaved = bool(interleaved)

    def _args(self):
        def at(x):
            return None if x is None else _ptr(x)
        n, rot = self.table.shape
        return _lib.RotaryArgs(_ptr(self.table), n, rot, int(self.interleaved),
                               at(self.k_positions), at(self.q_positions))


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

    def reorder_sequences(self, block_table, seq_lens, parents, tail_blocks, new_table=None,
                          new_lens=None, stream=None):
        """Row j of the new block table is a copy of row parents[j] of ``block_table`` that goes on by
        itself: full pages are shared, a partly filled last page stays with the first row of
        its parent and is copied to tail_blocks[j] for the others.  parents, tail_blocks: [n]
        int32, -1 as a parent gives an empty row.  Returns (new_table [n][max_blocks], -1 past a
        row's pages, new_lens [n]).  tail_blocks: a block for each row that is not in use,
        from alloc_blocks for instance.  References follow once the new table has been read:
        fork_blocks of each new row's entries, then free_blocks of each old row's and of the
        tail blocks (a call per row)."""
        import torch
        if new_table is None:
            if not (isinstance(block_table, torch.Tensor) and block_table.dim() == 2):
                _need("block_table", block_table, torch.int32, (None, None), self.device)
            if not (isinstance(parents, torch.Tensor) and parents.dim() == 1):
                _need("parents", parents, torch.int32, (None,), self.device)
            n, mb = parents.shape[0], block_table.shape[1]
            new_table = (_empty_like(block_table, stream) if n == block_table.shape[0]
                         else _empty((n, mb), torch.int32, self.device, stream))
        if new_lens is None:
            new_lens = _empty_like(parents, stream)
        rows, n = _validate_reorder(self.device, block_table, seq_lens, parents, tail_blocks,
                                    new_table, new_lens)
        _on_current(self.device)
        _lib.check("rcp_reorder_sequences", self._lib.rcp_reorder_sequences(
            self._h, _ptr(block_table), rows, int(block_table.shape[1]), _ptr(seq_lens),
            _ptr(parents), _ptr(tail_blocks), n, _ptr(new_table), _ptr(new_lens),
            _stream(stream)))
        return new_table, new_lens

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

    def reconstruct_workspace_bytes(self, rows: int, batch: int, max_blocks_per_seq: int,
                                    diff: bool = True) -> int:
        """Bytes of workspace of a reconstructing prefill.  diff=False: of calls that are given no
        DiffHeads, which take less on 4-bit pages."""
        n = ctypes.c_size_t()
        if diff:
            _lib.check("rcp_prefill_reconstruct_workspace_size",
                       self._lib.rcp_prefill_reconstruct_workspace_size(
                           self._h, rows, batch, max_blocks_per_seq, ctypes.byref(n)))
        else:
            _lib.check("rcp_prefill_step_workspace_size",
                       self._lib.rcp_prefill_step_workspace_size(
                           self._h, rows, batch, max_blocks_per_seq, None, ctypes.byref(n)))
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
    def append_kv(self, k, v, slot_mapping, stream=None, rotary=None) -> None:
        """k, v: [T][H][d] fp16; slot_mapping: [T] int64 (all on the cache's device); rotary: None or
        a Rotary, whose k_positions the keys are rotated to."""
        H, d = self.shape["num_heads"], self.shape["head_dim"]
        T = _validate_append(self.device, H, d, k, v, slot_mapping)
        if rotary is not None:
            _validate_rotary(self.device, d, rotary, tokens=T)
            _on_current(self.device)
            _lib.check("rcp_append_kv_rotary", self._lib.rcp_append_kv_rotary(
                self._h, _ptr(k), _ptr(v), _ptr(slot_mapping), T, ctypes.byref(rotary._args()),
                _stream(stream)))
            return
        _lib.check("rcp_append_kv", self._lib.rcp_append_kv(
            self._h, _ptr(k), _ptr(v), _ptr(slot_mapping), T, _stream(stream)))

    def _options(self, mod, rotary, diff, B: int, rows: int, tokens):
        """rcp_step_options of checked arguments."""
        opt = _lib.StepOptions()
        if mod is not None:
            _validate_mod(self.device, self.shape["num_heads"], B, rows, mod)
            opt.mod = ctypes.pointer(mod._args())
        if rotary is not None:
            _validate_rotary(self.device, self.shape["head_dim"], rotary, tokens, rows)
            opt.rotary = ctypes.pointer(rotary._args())
        if diff is not None:
            _validate_diff(self.device, self.shape["num_heads"], self.shape["head_dim"], diff)
            opt.diff = ctypes.pointer(diff._args())
        _on_current(self.device)
        return ctypes.byref(opt)

    def _decode_opt(self, mod, rotary, diff, app, q, block_table, seq_lens, out, ws, stream):
        """rcp_decode_step_opt; app: (k, v, slot_mapping), or None for the attention alone."""
        B = int(seq_lens.shape[0])
        k, v, slots, T = (None, None, None, 0) if app is None else (
            _ptr(app[0]), _ptr(app[1]), _ptr(app[2]), int(app[2].shape[0]))
        opt = self._options(mod, rotary, diff, B, B, None if app is None else T)
        _lib.check("rcp_decode_step_opt", self._lib.rcp_decode_step_opt(
            self._h, k, v, slots, T, _ptr(q), _ptr(block_table), int(block_table.shape[1]),
            _ptr(seq_lens), B, opt, _ptr(out), _ptr(ws), ws.numel() * ws.element_size(),
            _stream(stream)))

    def decode_attn(self, q, block_table, seq_lens, out=None, workspace=None, stream=None,
                    mod=None, rotary=None, diff=None):
        """q: [B][H][d] fp16; block_table: [B][max_blocks] int32; seq_lens: [B] int32; mod: None
        or a ScoreMod; rotary: None or a Rotary, whose q_positions the queries are rotated to;
        diff: None or a DiffHeads."""
        if out is None:
            out = _empty_like(q, stream)
        H, d = self.shape["num_heads"], self.shape["head_dim"]
        B = _validate_decode(self.device, H, d, q, block_table, seq_lens, out)
        ws = self._scratch(workspace, B, stream)
        if mod is not None or rotary is not None or diff is not None:
            self._decode_opt(mod, rotary, diff, None, q, block_table, seq_lens, out, ws, stream)
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
                    stream=None, mod=None, rotary=None, diff=None):
        """append_kv(k, v, slot_mapping, rotary=rotary) then decode_attn(q, ..., mod=mod,
        rotary=rotary, diff=diff), queued as one step."""
        if out is None:
            out = _empty_like(q, stream)
        H, d = self.shape["num_heads"], self.shape["head_dim"]
        _validate_append(self.device, H, d, k, v, slot_mapping)
        B = _validate_decode(self.device, H, d, q, block_table, seq_lens, out)
        ws = self._scratch(workspace, B, stream)
        if mod is not None or rotary is not None or diff is not None:
            self._decode_opt(mod, rotary, diff, (k, v, slot_mapping), q, block_table, seq_lens, out,
                             ws, stream)
            return out
        _lib.check("rcp_decode_step", self._lib.rcp_decode_step(
            self._h, _ptr(k), _ptr(v), _ptr(slot_mapping), int(slot_mapping.shape[0]), _ptr(q),
            _ptr(block_table), int(block_table.shape[1]), _ptr(seq_lens), B, _ptr(out), _ptr(ws),
            ws.numel() * ws.element_size(), _stream(stream)))
        return out

    def _prefill_variant(self, variant: str, rows: int, B: int, mod=None, diff=None) -> str:
        if variant == "auto" and diff is not None:
            variant = "reconstruct"
        if variant == "rank" and diff is not None:
            raise ValueError("differential attention has no rank-space prefill")
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

    def _prefill_scratch(self, workspace, variant: str, rows: int, B: int, mb: int, stream, diff=None):
        # quantized pages are widened into the workspace first (both variants)
        if workspace is not None or (variant == "rank" and self.page_format == "fp16"):
            return self._scratch(workspace, rows, stream)
        return self.workspace(rows, self.reconstruct_workspace_bytes(rows, B, mb, diff is not None),
                              stream)

    def _prefill_opt(self, mod, rotary, diff, app, q, cu_chunk_lens, block_table, seq_lens, out,
                     ws, stream, variant: str):
        """rcp_prefill_step_opt; app: (k, v, slot_mapping), or None for the attention alone."""
        B, rows = int(seq_lens.shape[0]), int(q.shape[0])
        k, v, slots, T = (None, None, None, 0) if app is None else (
            _ptr(app[0]), _ptr(app[1]), _ptr(app[2]), int(app[2].shape[0]))
        opt = self._options(mod, rotary, diff, B, rows, None if app is None else T)
        _lib.check("rcp_prefill_step_opt", self._lib.rcp_prefill_step_opt(
            self._h, k, v, slots, T, _ptr(q), _ptr(cu_chunk_lens), rows, _ptr(block_table),
            int(block_table.shape[1]), _ptr(seq_lens), B, 1 if variant == "reconstruct" else 0,
            opt, _ptr(out), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))

    def prefill_attn(self, q, cu_chunk_lens, block_table, seq_lens, out=None, workspace=None,
                     stream=None, variant: str = "auto", mod=None, rotary=None, diff=None):
        """q: [sum chunk][H][d] fp16; cu_chunk_lens: [B+1] int32; seq_lens include the chunk;
        mod: None or a ScoreMod; rotary: None or a Rotary, whose q_positions the queries are
        rotated to; diff: None or a DiffHeads (reconstruct is then the variant).

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
        variant = self._prefill_variant(variant, rows, B, mod, diff)
        ws = self._prefill_scratch(workspace, variant, rows, B, mb, stream, diff)
        if mod is not None or rotary is not None or diff is not None:
            self._prefill_opt(mod, rotary, diff, None, q, cu_chunk_lens, block_table, seq_lens, out,
                              ws, stream, variant)
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
                     out=None, workspace=None, stream=None, variant: str = "auto", mod=None,
                     rotary=None, diff=None):
        """append_kv(k, v, slot_mapping, rotary=rotary) then prefill_attn(q, cu_chunk_lens, ...,
        mod=mod, rotary=rotary, diff=diff), queued as one step (the chunk's query projection
        shares the append's launch).  Arguments and variant choice as the two calls."""
        if out is None:
            out = _empty_like(q, stream)
        H, d = self.shape["num_heads"], self.shape["head_dim"]
        T = _validate_append(self.device, H, d, k, v, slot_mapping)
        rows, B = _validate_prefill(self.device, H, d, q, cu_chunk_lens, block_table, seq_lens,
                                    out)
        mb = int(block_table.shape[1])
        variant = self._prefill_variant(variant, rows, B, mod, diff)
        ws = self._prefill_scratch(workspace, variant, rows, B, mb, stream, diff)
        if mod is not None or rotary is not None or diff is not None:
            self._prefill_opt(mod, rotary, diff, (k, v, slot_mapping), q, cu_chunk_lens, block_table,
                              seq_lens, out, ws, stream, variant)
            return out
        _lib.check("rcp_prefill_step", self._lib.rcp_prefill_step(
            self._h, _ptr(k), _ptr(v), _ptr(slot_mapping), T, _ptr(q), _ptr(cu_chunk_lens), rows,
            _ptr(block_table), mb, _ptr(seq_lens), B, 1 if variant == "reconstruct" else 0,
            _ptr(out), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))
        return out
