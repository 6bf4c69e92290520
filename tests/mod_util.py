"""Caches of every page format and the rounding bound of the score-modified attention tests."""
import numpy as np

import workloads as wl
from oracle import rcp_oracle as orc
from tests.gpu_util import t


def encode(pages, k, v):
    """Pages of fp16 coefficients in a format: (K, V) as the library holds them."""
    if pages == "fp16":
        return k, v
    if pages == "fp8_e4m3":
        return orc.e4m3_encode(k.astype(np.float64)), orc.e4m3_encode(v.astype(np.float64))
    return orc.int4_pack_pages(*orc.int4_pages(k, v))


def values(pages, shape, k, v, widened_keys):
    """Coefficients the kernels attend: fp16(code * scale) for the values of 4-bit pages, and for
    their keys where a prefill widens them first (the documented reading of the format)."""
    if pages == "fp16":
        return k, v
    if pages == "fp8_e4m3":
        return orc.e4m3_decode(k), orc.e4m3_decode(v)
    H, rk, R = shape["num_heads"], shape["rank_k"], shape["rank_v"]
    kc, vc = orc.int4_page_coefficients(k, v, H, rk, R)
    return (wl.fp16(kc) if widened_keys else kc), wl.fp16(vc)


def cache_of(pages, shape, U, W, k, v):
    from rank_compressed_paged_gb300 import PagedCoeffCache
    return PagedCoeffCache(shape["num_heads"], shape["head_dim"], shape["rank_k"],
                           shape["rank_v"], k.shape[0], t(U), t(W), k_pages=t(k.copy()),
                           v_pages=t(v.copy()), page_format=pages)


def score_mod(mod):
    """ScoreMod of a dict of host values (the oracle's keyword arguments)."""
    from rank_compressed_paged_gb300 import ScoreMod
    dev = {"alibi_slopes": np.float32, "prefix_lens": np.int32, "row_begin": np.int32}
    return ScoreMod(**{k: t(np.asarray(x, dev[k])) if k in dev and x is not None else x
                       for k, x in mod.items()})


def assert_within(got, ref, what):
    """|got - ref| within the roundings of the path, element by element.

    With A = sum_t p_t |V^_t| of the element and S the row's largest sum_k |q~_k c_k| / sqrt(d):
    * the weights enter the value product in fp16 (half a step: 2^-11 of each weight), and the
      decode normalises by the sum of the rounded ones (2^-11);
    * the reconstructing prefill stores V^ in fp16 (2^-11 of each value);
    * the output is rounded to fp16 (2^-11 of it, at most 2^-11 A): together 4 * 2^-11 A;
    * weights below fp16's normal range (the running maximum is followed to within 2^8) are
      off by at most 2^-25 each, relative to a largest weight of at least one; A counts
      weights that sum to one, so per token 2^-25 of its value: with N visible tokens
      N 2^-25 max|V^|, where max|V^| <= 8 for the N(0, 1) coefficients of these tests;
    * a query entry is off by at most 2^-16 of itself (split into four E4M3 terms; fp32 or
      an fp16 pair elsewhere), a score by 2^-16 S, a weight by twice that: 2^-15 S A; the
      cap and the bias are computed in fp32 (cap at most 64 here: below 2^-16 of a unit).
    """
    out, mag, prod, n = ref
    got = np.asarray(got, np.float64)
    assert got.shape == out.shape
    assert np.all(np.isfinite(got)), f"{what}: non-finite output"
    bound = (4 * 2.0 ** -11 + 2.0 ** -15 * (prod + 1)[:, None, None]) * mag \
        + 8 * n * 2.0 ** -25 + 2.0 ** -25
    over = np.abs(got - out) - bound
    assert np.all(over <= 0), (f"{what}: off by up to {np.abs(got - out).max():.3e}, "
                               f"{(over > 0).sum()} elements past the bound by up to "
                               f"{over.max():.3e}")
    assert np.all(got[mag.sum(axis=(1, 2)) == 0] == 0), f"{what}: a row without keys is not zero"
