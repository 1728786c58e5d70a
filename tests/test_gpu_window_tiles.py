"""moe_window_attention in each of its kinds of tile: up to 16 and up to 32 rows a cache head (keys shared out to the waves), up to 64 and
more (keys through LDS, rows shared out), at every width of heads, with what each has to leave out. Tolerances: window_util.attend_ref."""
import math

import numpy as np
import pytest
import torch

from moe_routed_expert_route_amd import binding as B
from tests.test_gpu_window import TYPES, check_attention, randn
from tests.window_util import BF16, DEV, F16, I8, Place, attend_ref, host, tree

pytestmark = pytest.mark.gpu

# tokens of the longest window, query heads a cache head
TILES = [(4, 4), (4, 7), (13, 5), (40, 4)]


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("d", [16, 48, 64, 80, 112, 128, 144, 192, 240, 256])
@pytest.mark.parametrize("tokens,group", TILES)
def test_head_sizes(tokens, group, d, dtype, cache):
    lengths = [tokens, 1, max(1, tokens // 2)]
    p = Place(lengths, [70, 0, 33], n_kv=2, d=d, cache=cache, seen=tree(lengths, d)[0], pad=1)
    check_attention(p, 2 * group, dtype, key=d)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("d", [80, 128, 256])
@pytest.mark.parametrize("tokens,group", TILES)
def test_lengths_of_several_steps_and_runs(tokens, group, d, dtype, cache):
    for ctx in (31, 290, 1100):
        check_attention(Place([tokens], [ctx], n_kv=1, d=d, cache=cache, page=48, seen=tree([tokens], ctx)[0]), group, dtype, key=ctx, lse=ctx != 31)


@pytest.mark.parametrize("order", ["slots", "wide", "both"])
@pytest.mark.parametrize("d", [80, 128, 208])
@pytest.mark.parametrize("tokens,group", TILES)
def test_cache_orders(tokens, group, d, order):
    check_attention(Place([tokens, 2], [130, 77], n_kv=3, d=d, page=32, order=order), 3 * group, BF16, ld=5)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("d", [64, 80, 144, 256])
@pytest.mark.parametrize("tokens,group", TILES)
def test_whatever_masked_places_hold(tokens, group, d, dtype, cache):
    """NaN and infinities past the last key, in pages of no sequence and in a token that only itself sees: the other rows' bits stay."""
    lengths, ctx = [tokens, 3], [70, 9]
    seen = [1 << j if j == 2 else ((2 << j) - 1) & ~4 for t in lengths for j in range(t)]
    p = Place(lengths, ctx, n_kv=1, d=d, cache=cache, seen=seen, key=4)
    q = randn((p.n, group * d), dtype, 1, 5)
    lse = [torch.zeros((p.n, group), device=DEV) for _ in range(2)]
    clean = B.moe_window_attention(p.cache, p.window, q, d ** -0.5, lse=lse[0])
    want, _, tol, _ = attend_ref(p, q, group, d ** -0.5)
    assert (np.abs(host(clean) - want) <= tol).all()
    keep = {(int(a), b) for s in range(2) for a, b in (p.key_at(s, i) for i in range(lengths[s] + ctx[s]))}
    poison, pools = [math.nan, math.inf, -math.inf], (p.k_scale, p.v_scale) if cache is I8 else (p.k, p.v)
    for i, (a, b) in enumerate((a, b) for a in range(p.n_pages) for b in range(p.page) if (a, b) not in keep):
        for pool in pools:
            pool[a, :, b] = poison[i % 3]
    out = B.moe_window_attention(p.cache, p.window, q, d ** -0.5, lse=lse[1])
    assert torch.equal(out, clean) and torch.equal(*lse)
    a, b = p.key_at(0, 72)
    pools[0][a, :, b], pools[1][a, :, b] = 1.0, math.nan
    out = B.moe_window_attention(p.cache, p.window, q, d ** -0.5)
    rows = [r for r in range(p.n) if r != 2]
    assert torch.equal(out[rows], clean[rows]) and torch.isnan(out[2]).all()
    if cache is not I8:
        p.v[a, :, b] = 1.0
        p.v[a, 0, b, d - 3] = -math.inf
        out = B.moe_window_attention(p.cache, p.window, q, d ** -0.5).view(p.n, group, d)
        assert torch.equal(out[rows], clean.view(p.n, group, d)[rows]) and (out[2, :, d - 3] == -math.inf).all()
        assert torch.isfinite(out[2, :, :d - 3]).all() and torch.isfinite(out[2, :, d - 2:]).all()
    pools[0][a, :, b] = math.nan     # a key that is not a number, of the token that only itself sees
    out = B.moe_window_attention(p.cache, p.window, q, d ** -0.5)
    assert torch.equal(out[rows], clean[rows]) and torch.isnan(out[2]).all()


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("d", [64, 80, 256])
@pytest.mark.parametrize("tokens,group", TILES)
def test_pages_out_of_range(tokens, group, d, dtype, cache):
    """Pages that are none, the first, one in the middle and those of the window's own keys, beside sound ones in the same step."""
    p = Place([tokens, 2], [200, 50], n_kv=1, d=d, cache=cache)
    last = (199 + tokens) // 16
    bad = [(0, 0, p.n_pages), (0, 5, -1), (0, last, 2 ** 31 - 1), (1, 1, -2 ** 31)]
    for s, c, page in bad:
        p.window.pages[s, c] = page
    check_attention(p, group, dtype, left_out=[(s, 16 * c, 16 * c + 16) for s, c, _ in bad], errors=256)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("d", [48, 128, 144])
@pytest.mark.parametrize("tokens,group", TILES)
def test_rows_that_see_nothing(tokens, group, d, dtype, cache):
    """Empty contexts and tokens of no bits, or of bits past the window alone; then the same behind a context."""
    seen = [(0 if j % 3 == 0 else 1 << 63 if j % 3 == 1 else (2 << j) - 1) for j in range(tokens)]
    for ctx in (0, 5):
        p = Place([tokens], [ctx], n_kv=1, d=d, cache=cache, seen=seen)
        out, lse = check_attention(p, group, dtype)
        if ctx == 0:
            blank = [j for j in range(tokens) if j % 3 != 2]
            assert not out[blank].any() and torch.isneginf(lse[blank]).all()


@pytest.mark.parametrize("n_seqs", [64, 65, 300])
@pytest.mark.parametrize("d,dtype,cache", [(64, BF16, BF16), (80, F16, I8), (128, F16, F16), (256, BF16, BF16), (256, BF16, I8)])
@pytest.mark.parametrize("tokens,group", TILES)
def test_many_sequences(tokens, group, d, dtype, cache, n_seqs):
    """More sequences than lanes: their items are listed in LDS, behind the ring of keys where there is one."""
    rng = np.random.default_rng(n_seqs)
    lengths = np.where(rng.random(n_seqs) < 0.1, tokens, rng.integers(0, 3, n_seqs))
    lengths[n_seqs // 2] = tokens
    p = Place(lengths, rng.integers(0, 60, n_seqs), n_kv=1, d=d, cache=cache, pad=2, max_window=tokens)
    check_attention(p, group, dtype)


@pytest.mark.parametrize("d,dtype,cache,tokens,n_heads", [(64, BF16, BF16, 1, 2), (128, BF16, BF16, 3, 8), (128, BF16, BF16, 20, 2), (256, F16, F16, 20, 4),
                                                          (256, F16, I8, 40, 2), (16, F16, I8, 64, 1)])
def test_the_most_sequences(d, dtype, cache, tokens, n_heads):
    """4096 sequences, most of one token or none."""
    rng = np.random.default_rng(5)
    lengths = rng.integers(0, 2, 4096)
    lengths[[7, 2047, 4095]] = tokens
    p = Place(lengths, [0] * 4096, n_kv=1, d=d, cache=cache, max_window=tokens)
    out = check_attention(p, n_heads, dtype)[0]
    again = B.moe_window_attention(p.cache, p.window, randn((p.rows, n_heads * d), dtype, 1, 5), d ** -0.5)
    assert torch.equal(out, again)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("tokens,group", TILES)
def test_keys_that_end_at_every_place_of_a_step(tokens, group, d, dtype, cache):
    """Windows that begin and end at each of the 32 keys of a step, of tokens that see themselves, the context and some others: each
    place of a tile masked for some rows, or past the last key, where the slots hold NaN."""
    lengths = [1 + s % min(tokens, 7) for s in range(40)]
    rng = np.random.default_rng(d + tokens)
    seen = [int(rng.integers(0, 1 << t)) | 1 << j for t in lengths for j in range(t)]
    p = Place(lengths, [s if s < 8 else 57 + s for s in range(40)], n_kv=1, d=d, cache=cache, seen=seen, max_window=tokens)
    keep = {(int(a), b) for s in range(40) for a, b in (p.key_at(s, i) for i in range(lengths[s] + p.ctx[s]))}
    bad = [(a, b) for a in range(p.n_pages) for b in range(p.page) if (a, b) not in keep]
    for pool in (p.k_scale, p.v_scale) if cache is I8 else (p.k, p.v):
        pool[[a for a, _ in bad], :, [b for _, b in bad]] = math.nan
    check_attention(p, group, dtype, key=d)
