"""Steps whose new tokens and query rows differ in number: they store and give what their append and
attention calls do, bit for bit (needs a GB300)."""
import functools

import numpy as np
import pytest
import torch

import workloads as wl
from rank_compressed_paged_gb300 import Rotary, rotary_table
from tests.gpu_util import t
from tests.mod_util import cache_of
from tests.test_gpu_rotary import FORMATS, SHAPES, empty_pages

pytestmark = pytest.mark.gpu


@functools.lru_cache(maxsize=None)
def factors(shape_name):
    return wl.make_factors(np.random.default_rng(11), *(
        SHAPES[shape_name][x] for x in ("num_heads", "head_dim", "rank_k", "rank_v")))


def inputs(shape, T, rows, seed):
    """New tokens' keys and values, and queries."""
    gen = torch.Generator("cuda").manual_seed(seed)
    return [torch.randn((n, shape["num_heads"], shape["head_dim"]), generator=gen, device="cuda",
                        dtype=torch.float16) for n in (T, T, rows)]


def same_pages(a, b):
    return torch.equal(a.k_pages.view(torch.uint8), b.k_pages.view(torch.uint8)) and \
        torch.equal(a.v_pages.view(torch.uint8), b.v_pages.view(torch.uint8))


# tokens and rows on either side of every change of kernel, tile or split
COUNTS = [(1, 20), (16, 17), (3, 200), (10, 400), (17, 193), (40, 250), (64, 65), (70, 192), (70, 300),
          (150, 260), (192, 193), (192, 500), (193, 20), (200, 256), (256, 257), (256, 700), (257, 300),
          (300, 40), (300, 2000), (600, 601), (900, 300), (2000, 1)]


@pytest.mark.parametrize("pages", FORMATS)
@pytest.mark.parametrize("shape_name", ["tiny", "main"])
@pytest.mark.parametrize("turned", ["keys and queries", "queries", "keys"])
def test_prefill_steps_store_what_their_append_does(shape_name, pages, turned):
    shape = SHAPES[shape_name]
    table = t(rotary_table(3000, shape["head_dim"]).numpy())
    for T, rows in COUNTS:
        k, v, q = inputs(shape, T, rows, seed=T + rows)
        length = max(T, rows) + 5
        blocks = (length + 15) // 16
        a, b = (cache_of(pages, shape, *factors(shape_name), *empty_pages(shape, pages, blocks)) for _ in range(2))
        kp = t(np.arange(length - T, length).astype(np.int32)) if "keys" in turned else None
        qp = t(np.arange(length - rows, length).astype(np.int32)) if "queries" in turned else None
        rot = Rotary(table, kp, qp)
        new = k, v, t(np.arange(length - T, length))
        att = (q, t(np.array([0, rows], np.int32)), t(np.arange(blocks, dtype=np.int32)[None]),
               t(np.array([length], np.int32)))
        one = a.prefill_step(*new, *att, rotary=rot)
        b.append_kv(*new, rotary=rot)
        two = b.prefill_attn(*att, rotary=rot)
        assert same_pages(a, b), (T, rows)
        if qp is not None:    # (queries as they are have a projection of their own in the attention call)
            assert torch.equal(one, two), (T, rows)
        assert a.read_device_error() == b.read_device_error() == 0


@pytest.mark.parametrize("shape_name", ["tiny", "main"])
@pytest.mark.parametrize("turned", ["keys and queries", "queries"])
def test_decode_steps_store_what_their_append_does(shape_name, turned):
    """As drafted tokens are: more new tokens than requests, or fewer; captured and replayed."""
    shape = SHAPES[shape_name]
    table = t(rotary_table(3000, shape["head_dim"]).numpy())
    for T, B in [(4, 200), (70, 250), (150, 300), (200, 70), (300, 17), (256, 260)]:
        k, v, q = inputs(shape, T, B, seed=T + 3 * B)
        lens = 20 + np.arange(B) % 12
        bt = np.arange(2 * B, dtype=np.int32).reshape(B, 2)
        spots = np.concatenate([32 * i + np.arange(n) for i, n in enumerate(lens)])
        slots = np.random.default_rng(T).permutation(spots)[:T]
        a, b = (cache_of("fp16", shape, *factors(shape_name), *empty_pages(shape, "fp16", 2 * B)) for _ in range(2))
        rot = Rotary(table, t((7 * np.arange(T)).astype(np.int32)) if "keys" in turned else None,
                     t((11 * np.arange(B)).astype(np.int32) % 3000))
        new, att = (k, v, t(slots)), (q, t(bt), t(lens.astype(np.int32)))
        one = a.decode_step(*new, *att, rotary=rot)
        b.append_kv(*new, rotary=rot)
        two = b.decode_attn(*att, rotary=rot)
        assert same_pages(a, b) and torch.equal(one, two), (T, B)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            again = a.decode_step(*new, *att, rotary=rot)
        a.k_pages.zero_(), a.v_pages.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same_pages(a, b) and torch.equal(again, two), (T, B)
        assert a.read_device_error() == b.read_device_error() == 0
