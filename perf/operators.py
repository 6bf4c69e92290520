"""Cases of the cache operators: score-modified attention over the paged coefficient cache
(decode and chunked prefill), page copies and token compaction, each with a plain form.

The cache holds, per token, r_k key coefficients per head and R joint value coefficients, in
pages of 16 tokens ([block][H][16][r_k] and [block][16][R]; fp16, E4M3 codes or 4-bit codes
with fp16 scales).  For a query row at position pos of a request with L cached tokens

    s_t = (U_k,h q_h) . c_k[t,h] / sqrt(d)
    s_t = cap tanh(s_t / cap)                       (cap > 0)
    s_t = s_t - slope_h |pos - t|                   (distance bias)
    t is visible iff t < L and (t < prefix or (begin <= t <= pos and t > pos - window))
    o_h = W_v[:, h d:(h+1) d]^T sum_t softmax(s)_t c_v[t]   (nothing visible: 0)

A case's lengths, chunk sizes and document borders follow from the case alone; the values
follow from the seed.
"""
import math

import torch

own = False   # True: run() makes the calls a user makes instead of the plain forms

BS = 16
# (H, d, r_k, R) of the two cache shapes
SHAPES = {"mha32": (32, 128, 64, 1024), "tiny": (4, 64, 16, 64)}


def _case(name, op, shape="mha32", pages="fp16", batch=1, length=1, chunk=0, cap=0.0, alibi=False,
          window=0, prefix=0, docs=0, keep=0.0, ragged=False):
    return dict(name=name, op=op, shape=shape, pages=pages, batch=batch, length=length, chunk=chunk,
                cap=cap, alibi=alibi, window=window, prefix=prefix, docs=docs, keep=keep,
                ragged=ragged)


def listed():
    return [
        # one short conversation: launch latency
        _case("decode_cap_alibi_b1_l1000", "decode", batch=1, length=1000, cap=30.0, alibi=True),
        # the full batch-64 x 8192 step with capped scores: every cached byte is read
        _case("decode_cap_b64_l8192", "decode", batch=64, length=8192, cap=50.0),
        # streaming conversations: attention sinks and the last tokens, E4M3 pages
        _case("decode_window_b64_l8192_e4m3", "decode", pages="fp8_e4m3", batch=64, length=8192,
              window=1000, prefix=20, ragged=True),
        # long packed contexts, each query inside its own document, 4-bit pages
        _case("decode_docs_cap_b20_l32768_int4", "decode", pages="int4", batch=20, length=32768,
              docs=9001, cap=20.0, alibi=True, ragged=True),
        # a few speculated tokens per request
        _case("prefill_cap_b4_l777_c5", "prefill", batch=4, length=777, chunk=5, cap=15.0,
              ragged=True),
        # the batch-16 x (4096 + 256) chunk with capped scores and a distance bias
        _case("prefill_cap_alibi_b16_l4352_c256", "prefill", batch=16, length=4352, chunk=256,
              cap=30.0, alibi=True),
        # packed documents, prefilled at once
        _case("prefill_docs_b2_l4096_c4096", "prefill", batch=2, length=4096, chunk=4096, docs=700),
        # one long context: a chunk that sees a shared prefix and a window, E4M3 pages
        _case("prefill_window_prefix_b1_l33000_c500_e4m3", "prefill", pages="fp8_e4m3", batch=1,
              length=33000, chunk=500, window=4000, prefix=130, cap=50.0),
        # the last page of one forked sequence
        _case("copy_1_page", "copy", batch=1),
        # copy-on-write of a batch's pages
        _case("copy_4096_pages", "copy", batch=4096),
        # one long request drops two tokens of five, 4-bit pages
        _case("compact_b1_l30001_int4", "compact", pages="int4", batch=1, length=30001, keep=0.6),
        # a batch drops half of its tokens
        _case("compact_b64_l8192", "compact", batch=64, length=8192, keep=0.5, ragged=True),
    ]


def _spread(rng, lo, hi):
    """An integer whose logarithm is uniform over [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "prefill", "prefill", "copy", "compact"])
    c = _case("", op, shape=rng.choice(["mha32", "mha32", "mha32", "tiny"]),
              pages=rng.choice(["fp16", "fp8_e4m3", "int4"]), ragged=rng.random() < 0.6)
    del c["name"]
    if op == "copy":
        c["batch"] = _spread(rng, 1, 4000)
        return c
    if op == "compact":
        c["batch"] = _spread(rng, 1, 64)
        c["length"] = _spread(rng, 1, min(32768, 500000 // c["batch"]))
        c["keep"] = round(rng.uniform(0.05, 0.98), 3)
        return c
    if op == "decode":
        c["batch"] = _spread(rng, 1, 64)
        c["length"] = _spread(rng, 1, min(32768, 500000 // c["batch"]))
    else:
        c["batch"] = _spread(rng, 1, 16)
        c["chunk"] = _spread(rng, 1, min(2048, 4096 // c["batch"]))
        most = min(16384, 65000 // c["batch"], 16000000 // (c["batch"] * c["chunk"]))
        c["length"] = c["chunk"] + _spread(rng, 1, most) - 1
    if rng.random() < 0.6:
        c["cap"] = float(rng.choice([5.0, 15.0, 30.0, 50.0]))
    c["alibi"] = rng.random() < 0.5
    if rng.random() < 0.5:
        c["window"] = _spread(rng, 1, 2 * c["length"])
    if rng.random() < 0.5:
        c["prefix"] = _spread(rng, 1, c["length"])
    if rng.random() < 0.4:
        c["docs"] = _spread(rng, 2, 2 * c["length"])
    return c


# ------------------------------------------------------------------------- sizes of a case

def _lens(c):
    """Cached tokens of each request (ragged: between half the length and all of it)."""
    L = c["length"]
    return [L - (b * 7919 + 13) % (L // 2 + 1) if c["ragged"] and b else L
            for b in range(c["batch"])]


def _chunks(c):
    """Query rows of each request of a prefill (ragged: between half the chunk and all of it)."""
    n = c["chunk"]
    return [min(L, n - (b * 104729 + 5) % (n // 2 + 1) if c["ragged"] and b else n)
            for b, L in enumerate(_lens(c))]


def _doc_start(docs, pos):
    """Start of the document that holds position pos: documents of docs/2 and docs tokens in
    turn (docs 0: one document)."""
    if docs == 0:
        return 0
    half = max(1, docs // 2)
    k, r = divmod(pos, half + docs)
    return k * (half + docs) + (half if r >= half else 0)


def _visible(c, L, pos):
    """(keys of the prefix, first and one past the last of the keys behind it) of a row."""
    pre = min(c["prefix"], L)
    lo = max(_doc_start(c["docs"], pos), pos - c["window"] + 1 if c["window"] else 0, 0)
    return pre, max(lo, pre), max(pos + 1, pre)


def _token_bytes(c):
    H, d, rk, R = SHAPES[c["shape"]]
    if c["pages"] == "int4":
        return (H * rk + R) // 2 + 2 * (H + R // 64)
    return (H * rk + R) * (2 if c["pages"] == "fp16" else 1)


def work(c):
    H, d, rk, R = SHAPES[c["shape"]]
    tok = _token_bytes(c)
    if c["op"] == "copy":
        return {"bytes": 2 * BS * tok * c["batch"] + 8 * c["batch"], "flops": 0}
    lens = _lens(c)
    if c["op"] == "compact":
        kept = c["keep"] * sum(lens)
        return {"bytes": 2 * tok * kept + sum(lens) + 12 * c["batch"], "flops": 0}
    rows = _chunks(c) if c["op"] == "prefill" else [1] * c["batch"]
    keys = pairs = values = 0
    for L, n in zip(lens, rows):
        seen, lo_all, hi_all = 0, L, 0
        for i in range(n):
            pre, lo, hi = _visible(c, L, L - n + i)
            seen += pre + max(0, hi - lo)
            lo_all, hi_all = min(lo_all, lo), max(hi_all, hi)
        k = min(c["prefix"], L) + max(0, hi_all - lo_all)
        keys += k
        pairs += seen
        # values: contracted in rank space, or rebuilt once per key
        values += min(2 * H * R * seen + 2 * H * R * d * n, 2 * R * H * d * k + 2 * H * d * seen)
    nq = sum(rows)
    flops = 2 * H * rk * d * nq + 2 * H * rk * pairs + values
    return {"bytes": keys * tok + 4 * H * d * nq + 2 * (H * rk * d + R * H * d) + keys // BS * 4,
            "flops": flops}


# ------------------------------------------------------------------------------- the inputs

def _pages(c, num_blocks, g):
    """Pages of N(0, 1) coefficients in the case's format."""
    H, d, rk, R = SHAPES[c["shape"]]
    dev = "cuda"
    if c["pages"] == "int4":
        def packed(codes, groups):
            b = torch.randint(0, 225, (num_blocks, codes // 2), generator=g, device=dev,
                              dtype=torch.int16)
            lo, hi = torch.div(b, 15, rounding_mode="floor") - 7, b % 15 - 7
            b = ((lo & 15) | ((hi & 15) << 4)).to(torch.uint8)
            s = (0.15 + 0.15 * torch.rand((num_blocks, groups), generator=g, device=dev)).half()
            return torch.cat([b, s.view(torch.uint8)], 1).contiguous()
        return packed(H * BS * rk, H * BS), packed(BS * R, BS * (R // 64))
    k = torch.empty((num_blocks, H, BS, rk), dtype=torch.float16, device=dev).normal_(generator=g)
    v = torch.empty((num_blocks, BS, R), dtype=torch.float16, device=dev).normal_(generator=g)
    if c["pages"] == "fp8_e4m3":
        k, v = (x.to(torch.float8_e4m3fn).view(torch.uint8) for x in (k, v))
    return k, v


def prepare(c, seed):
    H, d, rk, R = SHAPES[c["shape"]]
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": c}
    if c["op"] == "copy":
        n = c["batch"]
        num_blocks = 2 * n + 3
        ids = torch.randperm(num_blocks, generator=g, device="cuda")[:2 * n].to(torch.int32)
        s["pairs"] = ids.view(n, 2).contiguous()
    else:
        lens = _lens(c)
        need = [(L + BS - 1) // BS for L in lens]
        mb = max(need)
        num_blocks = sum(need) + 3
        perm = torch.randperm(num_blocks, generator=g, device="cuda")
        ids, s["spare"] = perm[:sum(need)].to(torch.int32), perm[sum(need)]
        nd = torch.tensor(need, device="cuda")
        table = torch.full((len(lens), mb), -1, dtype=torch.int32, device="cuda")
        table[torch.arange(mb, device="cuda")[None, :] < nd[:, None]] = ids
        s["table"] = table
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["k_pages"], s["v_pages"] = _pages(c, num_blocks, g)
    s["U"] = (torch.randn((H, rk, d), generator=g, device="cuda") / math.sqrt(d)).half()
    s["W"] = (torch.randn((R, H * d), generator=g, device="cuda") / math.sqrt(H * d)).half()
    if c["op"] == "compact":
        s["keep"] = (torch.rand((len(lens), mb * BS), generator=g, device="cuda")
                     < c["keep"]).to(torch.uint8)
    if c["op"] in ("decode", "prefill"):
        rows = _chunks(c) if c["op"] == "prefill" else [1] * c["batch"]
        s["max_chunk"] = max(rows)
        cu = [0]
        for n in rows:
            cu.append(cu[-1] + n)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        # scores of a few units, so that caps and biases matter
        s["q"] = (4 * torch.randn((cu[-1], H, d), generator=g, device="cuda")).half()
        s["slopes"] = None
        if c["alibi"]:
            s["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)],
                                       device="cuda")
        s["prefix"] = s["begin"] = None
        if c["prefix"]:
            s["prefix"] = torch.full((len(lens),), c["prefix"], dtype=torch.int32, device="cuda")
        if c["docs"]:
            s["begin"] = torch.tensor([_doc_start(c["docs"], L - n + i)
                                       for L, n in zip(lens, rows) for i in range(n)],
                                      dtype=torch.int32, device="cuda")
    if own:
        from rank_compressed_paged_gb300 import PagedCoeffCache, ScoreMod
        s["cache"] = PagedCoeffCache(H, d, rk, R, num_blocks, s["U"], s["W"],
                                     k_pages=s["k_pages"], v_pages=s["v_pages"],
                                     page_format=c["pages"])
        if c["op"] in ("decode", "prefill"):
            s["mod"] = ScoreMod(softcap=c["cap"], alibi_slopes=s["slopes"], window=c["window"],
                                prefix_lens=s["prefix"], row_begin=s["begin"])
    return s


# ------------------------------------------------------------------------------ plain forms

def _raw(x):
    return x if x.dtype == torch.uint8 else x.view(torch.int16)


def _unpack(pages, codes, group):
    """4-bit pages to fp32: codes (two per byte, even index in the low nibble, two's
    complement) then fp16 scales, one per group."""
    b = pages[..., :codes // 2].to(torch.int32)
    nib = torch.stack([b & 15, b >> 4], -1).flatten(-2)
    val = ((nib ^ 8) - 8).float()
    sc = pages[..., codes // 2:].contiguous().view(torch.float16).float()
    return val * sc.repeat_interleave(group, -1)


def _gather(s):
    """Coefficients of every table entry: keys [B, H, T, r_k], values [B, T, R], fp32."""
    c = s["case"]
    H, d, rk, R = SHAPES[c["shape"]]
    table = s["table"].clamp(min=0).long()
    B, mb = table.shape
    k, v = s["k_pages"][table], s["v_pages"][table]
    if c["pages"] == "int4":
        k, v = _unpack(k, H * BS * rk, rk), _unpack(v, BS * R, 64)
    elif c["pages"] == "fp8_e4m3":
        k, v = k.view(torch.float8_e4m3fn).float(), v.view(torch.float8_e4m3fn).float()
    else:
        k, v = k.float(), v.float()
    k = k.view(B, mb, H, BS, rk).permute(0, 2, 1, 3, 4).reshape(B, H, mb * BS, rk)
    return k, v.reshape(B, mb * BS, R)


def _attend(s):
    c = s["case"]
    H, d, rk, R = SHAPES[c["shape"]]
    k, v = _gather(s)
    B, T = v.shape[:2]
    C = s["max_chunk"]
    cu = s["cu"].long()
    n = cu[1:] - cu[:-1]
    row = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), row, right=True)
    i = row - cu[b]
    q = torch.zeros((B, C, H, d), device="cuda")
    q[b, i] = s["q"].float()
    pos = (s["lens"] - n)[:, None] + torch.arange(C, device="cuda")          # [B, C]
    t = torch.arange(T, device="cuda")
    seen = t <= pos[:, :, None]
    if c["window"]:
        seen = seen & (t > pos[:, :, None] - c["window"])
    if s["begin"] is not None:
        begin = torch.zeros((B, C), dtype=torch.long, device="cuda")
        begin[b, i] = s["begin"].long()
        seen = seen & (t >= begin[:, :, None])
    if s["prefix"] is not None:
        seen = seen | (t < s["prefix"][:, None, None])
    seen = (seen & (t < s["lens"][:, None, None]))[:, None]                  # [B, 1, C, T]
    qt = torch.einsum("bchd,hkd->bhck", q, s["U"].float())
    x = qt @ k.transpose(2, 3) / math.sqrt(d)                                # [B, H, C, T]
    if c["cap"]:
        x = c["cap"] * torch.tanh(x / c["cap"])
    if s["slopes"] is not None:
        x = x - s["slopes"][:, None, None] * (pos[:, :, None] - t).abs()[:, None]
    x = x.masked_fill(~seen, float("-inf"))
    m = x.max(-1, keepdim=True).values
    e = torch.exp(x - m.masked_fill(m == float("-inf"), 0.0))
    p = e / e.sum(-1, keepdim=True).clamp(min=1e-30)
    z = torch.einsum("bhct,btr->bchr", p, v)
    o = torch.einsum("bchr,rhd->bchd", z, s["W"].float().view(R, H, d))
    return o[b, i].half()


def _copy(s):
    src, dst = s["pairs"][:, 0].long(), s["pairs"][:, 1].long()
    s["k_pages"][dst] = s["k_pages"][src]
    s["v_pages"][dst] = s["v_pages"][src]


def _move(rows, blk, off, src):
    """rows [..., block, 16, width]: every table position takes the row of position src."""
    sb, so = blk.gather(1, src), off.gather(1, src)
    moved = rows[sb, :, so]
    rows[blk, :, off] = moved


def _compact(s):
    """Every position below the new length takes the kept token of that rank, the others
    keep their own."""
    c = s["case"]
    H, d, rk, R = SHAPES[c["shape"]]
    table = s["table"].clamp(min=0).long()
    B, mb = table.shape
    T = mb * BS
    t = torch.arange(T, device="cuda")
    kept = (s["keep"] != 0) & (t < s["lens"][:, None])
    new = kept.sum(1)
    order = torch.argsort((~kept).to(torch.uint8), dim=1, stable=True)
    src = torch.where(t < new[:, None], order, t)
    # positions behind a request's pages write a page that no table holds
    have = t < ((s["lens"] + BS - 1) // BS * BS)[:, None]
    blk = torch.where(have, table.repeat_interleave(BS, 1), s["spare"])
    src = torch.where(have, src, t)
    off = (t % BS).expand(B, T)
    nb = s["k_pages"].shape[0]
    if c["pages"] == "int4":
        kc, vc = H * BS * rk // 2, BS * R // 2
        k, v = s["k_pages"], s["v_pages"]
        _move(k[:, :kc].view(nb, H, BS, rk // 2), blk, off, src)
        _move(k[:, kc:].view(nb, H, BS, 2), blk, off, src)
        _move(v[:, :vc].view(nb, 1, BS, R // 2), blk, off, src)
        _move(v[:, vc:].view(nb, 1, BS, R // 32), blk, off, src)
    else:
        _move(s["k_pages"], blk, off, src)
        _move(s["v_pages"].view(nb, 1, BS, R), blk, off, src)
    return new.to(torch.int32)


def run(s):
    op = s["case"]["op"]
    if op == "decode":
        if own:
            return s["cache"].decode_attn(s["q"], s["table"], s["lens"], mod=s["mod"])
        return _attend(s)
    if op == "prefill":
        if own:
            return s["cache"].prefill_attn(s["q"], s["cu"], s["table"], s["lens"], mod=s["mod"])
        return _attend(s)
    if op == "copy":
        if own:
            s["cache"].copy_blocks(s["pairs"])
        else:
            _copy(s)
        return _raw(s["k_pages"]), _raw(s["v_pages"])
    if own:
        new = s["cache"].compact_tokens(s["table"], s["lens"], s["keep"])
    else:
        new = _compact(s)
    return new, _raw(s["k_pages"]), _raw(s["v_pages"])


# ------------------------------------------------------------------- definition in 64 bits

def _token(pages, codes, group, width, slot, heads):
    """Coefficients of the tokens at slots (block * 16 + offset) as fp64 [n, heads, width]."""
    blk, off = slot // BS, slot % BS
    row = torch.arange(heads, device="cuda")[None, :] * BS + off[:, None]     # [n, heads]
    if pages.dtype == torch.float16:
        return pages.view(-1, heads * BS, width)[blk[:, None], row].double()
    if codes == 0:
        codes8 = pages.view(-1, heads * BS, width)[blk[:, None], row]
        return codes8.view(torch.float8_e4m3fn).float().double()
    b = pages[:, :codes // 2].reshape(-1, heads * BS, width // 2)[blk[:, None], row].double()
    hi = torch.floor(b / 16)
    two = torch.stack([b - 16 * hi, hi], -1).flatten(-2)
    two = torch.where(two > 7, two - 16, two)
    sc = pages[:, codes // 2:].contiguous().view(torch.float16)
    sc = sc.view(-1, heads * BS, width // group)[blk[:, None], row].double()
    return (two.view(*two.shape[:-1], width // group, group) * sc[..., None]).flatten(-2)


def exact(c, seed):
    if c["op"] in ("copy", "compact"):
        return None
    s = prepare(c, seed)
    H, d, rk, R = SHAPES[c["shape"]]
    U, W = s["U"].double(), s["W"].double()
    i4 = c["pages"] == "int4"
    lens = _lens(c)
    rows = _chunks(c) if c["op"] == "prefill" else [1] * c["batch"]
    out = torch.zeros((sum(rows), H, d), dtype=torch.float64, device="cuda")
    at = 0
    for b, (L, n) in enumerate(zip(lens, rows)):
        # the tokens some row sees
        lo = torch.tensor([_visible(c, L, L - n + i) for i in range(n)], device="cuda")
        pre, first, last = lo[:, 0], lo[:, 1], lo[:, 2]
        t = torch.arange(L, device="cuda")
        tok = t[(t < pre.max()) | ((t >= first.min()) & (t < last.max()))]
        slot = s["table"][b].long()[tok // BS] * BS + tok % BS
        ck = _token(s["k_pages"], H * BS * rk if i4 else 0, rk, rk, slot, H)     # [t, H, r_k]
        cv = _token(s["v_pages"], BS * R if i4 else 0, 64, R, slot, 1)[:, 0]     # [t, R]
        pos = torch.arange(L - n, L, device="cuda")
        see = (tok < pre[:, None]) | ((tok >= first[:, None]) & (tok < last[:, None]))  # [n, t]
        for h in range(H):
            x = (s["q"][at:at + n, h].double() @ U[h].T) @ ck[:, h].T / math.sqrt(d)
            if c["cap"]:
                x = c["cap"] * torch.tanh(x / c["cap"])
            if c["alibi"]:
                x = x - 2.0 ** (-8.0 * (h + 1) / H) * (pos[:, None] - tok).abs()
            x = torch.where(see, x, torch.full_like(x, -math.inf))
            p = torch.where(see.any(1, keepdim=True), torch.softmax(x, 1), torch.zeros_like(x))
            Wh = W[:, h * d:(h + 1) * d]
            # the cheaper order of the two products
            few = n * R * (len(tok) + d) < len(tok) * d * (R + n)
            out[at:at + n, h] = (p @ cv) @ Wh if few else p @ (cv @ Wh)
        at += n
    return out
