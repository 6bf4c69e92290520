"""Beam selection where totals of different beams are equal: they keep the order of (beam, token),
whatever 16-byte boundaries their rows of logits start on (needs a GB300)."""
import numpy as np
import pytest
import torch

from rank_compressed_paged_gb300 import beam_select
from tests.gpu_util import t
from tests.test_gpu_beam import DTYPES, check, logits_of

pytestmark = pytest.mark.gpu


def rows(B, V, seed, scale=3.0):
    """A row of logits for each request, two of them large."""
    x = scale * np.random.default_rng(seed).standard_normal((B, V))
    x[:, V // 2], x[:, V - 1] = 4 * scale + 2, 4 * scale + 1
    return x


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("V", [2, 3, 5, 7, 1001, 1002, 9001, 50003, 131071, 262143])
@pytest.mark.parametrize("B,K", [(1, 8), (3, 5)])
def test_beams_that_are_equal_keep_their_order(dtype, V, B, K):
    """Every beam of a request is the same row with the same score, as where a prompt is expanded to
    its beams: each rank of the vocabulary comes from beam 0, 1, .. in turn."""
    if B * K * V > 2 ** 21 and dtype != "bf16":
        K = 4
    x = np.repeat(rows(B, V, seed=V)[:, None], K, axis=1)
    s = np.full((B, K), -1.25)
    held = logits_of(x, dtype)[1][:, 0].astype(np.float64)
    order = np.argsort(-held, axis=1, kind="stable")
    best, second = order[:, :1], order[:, 1:2]
    top = -np.sort(-held, axis=1)[:, :3]
    alone = np.all(top[:, 1:] < top[:, :-1], axis=1)    # requests whose three largest differ in the dtype
    assert alone.any()
    own = np.arange(B * K).reshape(B, K)
    got = check(x, s, dtype, what="no end")
    assert np.all((got[1] == best)[alone]) and np.array_equal(got[2][alone], own[alone])
    for eos in (int(best[0, 0]), int(second[0, 0])):
        got = check(x, s, dtype, eos=eos, what=eos)
        assert np.all((got[1] == np.where(best == eos, second, best))[alone])
        assert np.array_equal(got[2][alone], own[alone])
        # all ends of a request are among its best K, or none is
        assert np.all((np.isfinite(got[3]) == (best == eos))[alone])
        assert np.all(got[3] == got[3][:, :1])


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("V", [5, 4099, 9001])
def test_pairs_of_equal_beams_among_others(dtype, V):
    """Beams 0 and 3, 1 and 4 are equal, 2 and 5 alone, and the best K end within a pair's ends."""
    x = rows(2, V, seed=V + 1)[:, None].repeat(6, axis=1)
    x[:, [1, 4]] = np.roll(x[:, [1, 4]], 2, axis=2)
    x[:, 2] *= 0.5
    x[:, 5] *= 0.25
    s = np.tile([-1.0, -1.5, -1.25, -1.0, -1.5, -2.0], (2, 1))
    check(x, s, dtype)
    for eos in range(0, V, max(1, V // 7)):
        check(x, s, dtype, eos=eos)
    check(x, s, dtype, eos=V // 2)
    check(x, s, dtype, eos=(V // 2 + 2) % V)


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("name", ["equal", "sorted", "blocks"])
def test_equal_beams_whose_lists_overflow(dtype, name):
    """Equal scores beside rows on which many candidates reach the bound, at an odd vocabulary."""
    V, K = 40001, 6
    v = np.arange(V)
    x = {"equal": np.full(V, 1.5), "sorted": v * 2.0 ** -10, "blocks": (v // 5000) * 0.5}[name]
    x = np.repeat(x[None, None], K, axis=1)
    for s in (np.full((1, K), -0.5), np.array([[0, 0, -0.125, 0, -0.125, -0.25]])):
        check(x, s, dtype, what=name)
        check(x, s, dtype, eos=V - 1, what=name)
        check(x, s, dtype, eos=0, what=name)


@pytest.mark.parametrize("dtype", sorted(DTYPES))
def test_a_row_alone_and_among_others(dtype):
    """What a request gives does not depend on its place in the batch, to the last bit."""
    V, K, B = 4099, 3, 9
    r = np.random.default_rng(8)
    one, s = 3 * r.standard_normal((1, K, V)), r.standard_normal((1, K))
    g, _ = logits_of(np.repeat(one, B, axis=0), dtype)
    sc = t(np.repeat(s, B, axis=0).astype(np.float32))
    many = beam_select(g, sc, eos=17)
    for a, b in zip(many, beam_select(g[:1], sc[:1], eos=17)):
        off = torch.zeros_like(a)
        if a is many[2]:
            off += K * torch.arange(B, device="cuda", dtype=a.dtype)[:, None]
        assert torch.equal(a, b.expand(B, K) + off)
