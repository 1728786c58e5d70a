"""The calls on windows at the edges of what they accept: lists of rows that go back, contexts next to the largest, scales, weights
and values far apart. Tolerances are window_util.attend_ref's, or stand at the test."""
import numpy as np
import pytest
import torch

from moe_routed_expert_route_amd import binding as B
from tests.test_gpu_window import check_logprobs, randn
from tests.window_util import BF16, DEV, F16, F32, HALF_STEP, I8, TINY, Place, attend_ref, host

pytestmark = pytest.mark.gpu


def owned(starts, n):
    """The rows of each sequence of a list of starts: none where its rows do not ascend within [0, n), or where it starts below
    an earlier entry."""
    out = []
    for s in range(len(starts) - 1):
        a, b = starts[s], starts[s + 1]
        out.append(range(a, b) if 0 <= a <= b <= n and a >= max(starts[:s + 1]) else range(0))
    return out


def back(n_seqs, at):
    """A list of n_seqs sequences of two rows each that falls back to row 1 after sequence `at`."""
    starts = [2 * s for s in range(n_seqs + 1)]
    starts[at + 1:] = [1 + 2 * s for s in range(n_seqs - at)]
    return starts


LISTS = [[0, 5, 3, 8], [100, 104, 0, 4], [4, 0, 8], [0, 3, 3, -2, 1, 4, 9], [-5, 2, 6], [0, 4, 1000, 8, 12], [7, 6, 5, 0], [0, 5, 3, 4, 5, 9],
         back(64, 40), back(65, 62), back(200, 70), back(300, 255), back(600, 511), [0] + [2] * 300 + [1, 3], [9] * 100 + [0, 4] + [9, 12]]


@pytest.mark.parametrize("dtype,cache,tokens", [(BF16, BF16, 1), (F16, I8, 1), (BF16, BF16, 12)])
@pytest.mark.parametrize("starts", LISTS, ids=lambda s: f"{len(s) - 1}:{s[:6]}")
def test_lists_of_rows_that_go_back(starts, dtype, cache, tokens):
    """A sequence that starts below an earlier entry is left out by every call; the others are as without it, and no row but theirs is
    written. `tokens` = 12: the same with windows of twelve times the rows (keys through LDS)."""
    n = tokens * max(12, min(max(starts), 700))
    starts = [tokens * a for a in starts]
    rows = owned(starts, n)
    assert any(len(r) != starts[s + 1] - starts[s] for s, r in enumerate(rows))
    rng = np.random.default_rng(len(starts))
    p = Place([len(r) for r in rows], rng.integers(100, 150, len(rows)), n_kv=1, d=64, cache=cache)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)
    p.start, p.n, p.rows = np.array(starts, dtype=np.int64), n, n
    p.window = B.Window(ints(starts), p.window.ctx_len, p.window.pages, n, 8 if tokens == 1 else 64)
    mine = torch.zeros(n, dtype=torch.bool)
    for r in rows:
        mine[r.start:r.stop] = True
    pools = [t.clone() for t in (p.k, p.v)]
    q, k, v = randn((n, 128), dtype, 1), randn((n, 64), dtype, 2), randn((n, 64), dtype, 3)
    q_out = torch.full_like(q, 5.0)
    B.moe_window_append(p.cache, p.window, q, k, v, q_out=q_out)
    assert p.window.errors() == 128
    assert torch.equal(q_out[mine], q[mine]) and (q_out[~mine] == 5.0).all()
    written = torch.zeros(p.k.shape[0], p.k.shape[2], dtype=torch.bool)
    for s, r in enumerate(rows):
        for j in range(len(r)):
            page, slot = p.key_at(s, p.ctx[s] + j)
            written[page, slot] = True
            if cache is not I8:
                assert torch.equal(p.k[page, 0, slot], k[r.start + j]) and torch.equal(p.v[page, 0, slot], v[r.start + j])
    for pool, old in zip((p.k, p.v), pools):
        assert torch.equal(pool[:, 0].cpu()[~written], old[:, 0].cpu()[~written])
    p.window.err.zero_()
    out, lse = torch.full_like(q, 5.0), torch.full((n, 2), 5.0, device=DEV)
    B.moe_window_attention(p.cache, p.window, q, 0.125, out=out, lse=lse)
    assert p.window.errors() == 128
    want, want_lse, tol, lse_tol = attend_ref(p, q, 2, 0.125)
    assert (np.abs(host(out) - want)[mine] <= tol[mine]).all() and (np.abs(host(lse) - want_lse)[mine] <= lse_tol[mine]).all()
    assert (out[~mine] == 5.0).all() and (lse[~mine] == 5.0).all()


@pytest.mark.parametrize("dtype,tokens", [(BF16, 2), (F16, 40)])
def test_contexts_next_to_the_largest(dtype, tokens):
    """2^31 - 1064 keys, of which the table shares all but the last 984 in one page. A query of zeros takes the mean of the values:
    sums of ones and zeros that float32 holds, so that the rounding of the quotient (2^-24 twice), of exp2 (1 for 0) and of the
    output remain; a query of ones one key of the last page alone. Slots past the last key hold NaN."""
    page, cols = 1024, (1 << 21) - 1
    keys = page * cols - 40
    k, v = (torch.zeros((2, 1, page, 16), dtype=dtype, device=DEV) for _ in range(2))
    v[0, 0, ::4, ::2] = 1.0
    k[1, 0, 100], v[1, 0, 100] = 30.0, 5.0
    for pool in (k, v):
        pool[1, 0, page - 40:] = float("nan")
    table = torch.zeros((1, cols), dtype=torch.int32, device=DEV)
    table[0, -1] = 1
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
    seen = torch.full((tokens,), -1, dtype=torch.int64, device=DEV)
    w = B.Window(ints(0, tokens), ints(keys - tokens), table, tokens, tokens, seen=seen)
    q = torch.zeros((tokens, 16), dtype=dtype, device=DEV)
    q[1::2] = 1.0
    lse = torch.zeros((tokens, 1), device=DEV)
    out = B.moe_window_attention(B.KVCache(k, v), w, q, 1.0, lse=lse)
    assert w.errors() == 0
    out, lse = host(out), host(lse)[:, 0]
    mean = (np.where(np.arange(16) % 2 == 0, (cols - 1) * (page // 4), 0) + 5.0) / keys
    assert (np.abs(out[::2] - mean) <= mean * (HALF_STEP[dtype] + 2.0 ** -22) + TINY[dtype]).all()
    assert (out[1::2] == 5.0).all()
    assert (np.abs(lse[::2] - np.log(keys)) <= 2.0 ** -20 * 22).all() and (np.abs(lse[1::2] - 480.0) <= 480 * 2.0 ** -22).all()


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_log_probabilities_of_the_largest_scale(dtype):
    """Logits apart by 2^-14 and more: a score of 0 and of less than -2^112, so probabilities of one, of a half where two are largest,
    and of none."""
    x = torch.tensor([[1.0, 2.0, 2.0 ** -14, -1.0], [0.5, 0.5, 0.0, -0.5], [-1.0, -2.0, -3.0, -4.0]], device=DEV).to(dtype)
    logp, h, ids, top = B.moe_token_logprobs(x, tokens=torch.tensor([[1, 0], [1, 2], [0, 3]], dtype=torch.int32, device=DEV), k=2, entropy=True,
                                             scale=2.0 ** 127)
    assert ids.tolist() == [[1, 0], [0, 1], [0, 1]]
    half = -float(np.log(2))
    assert logp[0, 0] == 0 and logp[2, 0] == 0 and abs(float(logp[1, 0]) - half) < 2.0 ** -22
    assert (logp[:, 1] < -2.0 ** 112).all() and h[0] == 0 and abs(float(h[1]) + half) < 2.0 ** -22 and h[2] == 0
    assert top[0, 0] == 0 and abs(float(top[1, 1]) - half) < 2.0 ** -22 and top[2, 1] < -2.0 ** 112


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("tokens", [2, 40])
def test_attention_of_the_largest_scale(tokens, dtype):
    """One key of 2^-14 times a query of 2^-8: a score of 2^105 beside zeros, which alone counts; a query of zeros beside it."""
    p = Place([tokens], [50], n_kv=1, d=64, cache=dtype)
    p.k.zero_()
    for i in range(50 + tokens):
        page, slot = p.key_at(0, i)
        p.k[page, 0, slot, 0] = 2.0 ** -14 if i == 17 else 0.0
    q = torch.zeros((tokens, 64), dtype=dtype, device=DEV)
    q[:, 0] = torch.where(torch.arange(tokens, device=DEV) % 2 == 0, 2.0 ** -8, 0.0)
    lse = torch.zeros((tokens, 1), device=DEV)
    out = B.moe_window_attention(p.cache, p.window, q, 2.0 ** 127, lse=lse)
    page, slot = p.key_at(0, 17)
    assert torch.equal(out[::2], p.v[page, 0, slot].expand_as(out[::2])) and (lse[::2, 0] == 2.0 ** 105).all()
    want, want_lse, tol, lse_tol = attend_ref(p, q, 1, 2.0 ** 127)
    assert (np.abs(host(out) - want)[1::2] <= tol[1::2]).all() and (np.abs(host(lse) - want_lse)[1::2] <= lse_tol[1::2]).all()


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("scale", [1e-38, 2.5e-37])
@pytest.mark.parametrize("n", [12, 5000, 70000])
def test_log_probabilities_of_infinities_under_a_small_scale(n, scale, dtype):
    """Infinity counts as the largest float32, also where the scale makes a score of a few units of it."""
    x = randn((6, n), F32, n, 4, scale=1e38).clamp(-3e38, 3e38)
    x[0, 3] = x[1, 2] = x[1, n - 1] = x[1, n // 2] = x[3, 5] = float("inf")
    x[2, 7], x[3, 1], x[4, 4], x[4, 0] = 3.4028234663852886e38, 3.4028234663852886e38, float("nan"), float("-inf")
    x[5, ::2] = float("inf")
    check_logprobs(x.to(dtype), torch.tensor([[3, 1, 5, 7, 0, n - 1]] * 6, dtype=torch.int32, device=DEV), min(n, 20), scale)


@pytest.mark.parametrize("layout", [0, 3, (1 << 32) + 1, -(1 << 32) + 2])
def test_layouts_that_are_none(layout):
    p = Place([2], [3], d=64)
    q, k, v = (randn((2, 128), BF16, i) for i in range(3))
    k0 = p.k.clone()
    with pytest.raises(ValueError, match="layout"):
        B.moe_window_append(p.cache, p.window, q, k, v, freq=torch.ones(32, device=DEV), layout=layout)
    assert torch.equal(p.k, k0)


@pytest.mark.parametrize("tokens", [[1] * 65, [1] * 300, [64, 1, 40], [3] * 30])
def test_windows_of_a_length_that_is_not_given(tokens):
    """Batches of more rows than a window may have, without a longest window."""
    p = Place(tokens, [5 * (s % 40) for s in range(len(tokens))], n_kv=1, d=64)
    p.window = B.Window(p.window.row_start, p.window.ctx_len, p.window.pages, p.rows)
    q = randn((p.rows, 256), BF16, 2)
    out = B.moe_window_attention(p.cache, p.window, q, 0.125)
    want, _, tol, _ = attend_ref(p, q, 4, 0.125)
    assert (np.abs(host(out) - want) <= tol).all() and p.window.errors() == 0


def test_a_window_that_is_too_long_without_its_length():
    """Alone it is refused, among others left out and flagged; append takes windows of any length."""
    for tokens in ([65], [65, 2]):
        p = Place(tokens, [0] * len(tokens), n_kv=1, d=64)
        w = B.Window(p.window.row_start, p.window.ctx_len, p.window.pages, p.rows)
        q = randn((p.rows, 64), BF16, 2)
        B.moe_window_append(p.cache, w, q, q, q)
        assert w.errors() == 0
        out = torch.full_like(q, 5.0)
        if len(tokens) == 1:
            with pytest.raises(RuntimeError):
                B.moe_window_attention(p.cache, w, q, 0.125, out=out)
        else:
            B.moe_window_attention(p.cache, w, q, 0.125, out=out)
            assert w.errors() == 128 and (out[:65] == 5.0).all() and not (out[65:] == 5.0).all()


@pytest.mark.parametrize("dtype,cache", [(BF16, BF16), (F16, I8)])
@pytest.mark.parametrize("tokens", [[3, 0, 2], [300, 20, 400]])
def test_rows_of_no_sequence_count_for_nothing(tokens, dtype, cache):
    """NaN and infinities in padded rows behind the last sequence, which append and attention may read: the same bits everywhere, and
    the padded rows of the outputs as they were."""
    got = []
    for bad in (0.0, float("nan"), float("inf")):
        p = Place(tokens, [9, 4, 0], d=64, cache=cache, pad=7)
        q, k, v = randn((p.rows, 256), dtype, 1), randn((p.rows, 128), dtype, 2), randn((p.rows, 128), dtype, 3)
        q[p.n:], k[p.n:], v[p.n:] = bad, bad, bad
        q_out, out, lse = torch.full_like(q, 5.0), torch.full_like(q, 5.0), torch.full((p.rows, 4), 5.0, device=DEV)
        w = torch.ones(64, dtype=dtype, device=DEV)
        B.moe_window_append(p.cache, p.window, q, k, v, freq=torch.ones(16, device=DEV), q_weight=w, k_weight=w, q_out=q_out)
        if max(tokens) <= 64:
            B.moe_window_attention(p.cache, p.window, q, 0.125, out=out, lse=lse)
        assert p.window.errors() == 0 and all((t[p.n:] == 5.0).all() for t in (q_out, out, lse))
        got.append([q_out, out, lse, p.k, p.v] + ([p.k_scale, p.v_scale] if cache is I8 else []))
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))


# a head's rows in each kind of tile: up to 16, up to 32, up to 64 and more (n_heads / n_kv times the longest window)
TILES = [(1, 4), (3, 8), (10, 4), (40, 4)]


@pytest.mark.parametrize("tokens,n_heads,dtype", [(*t, BF16) for t in TILES[:2]] + [(*t, F16) for t in TILES])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_weights_over_int8_rows_keep_more_than_16_bits(tokens, n_heads, d, dtype):
    """A weight times its value's scale, in two bfloat16 parts (of up to 32 rows a head, and for float16 queries), is off by 2^-16
    at most: twice 8 bits. The bound for queries of float32 counts all but that and the rounding of the output."""
    p = Place([tokens, 1], [700, 90], n_kv=1, d=d, cache=I8, key=d)
    q = randn((p.n, n_heads * d), dtype, 7, scale=0.3)
    out = B.moe_window_attention(p.cache, p.window, q, d ** -0.5)
    want, _, tol, _ = attend_ref(p, q.float(), n_heads, d ** -0.5)
    most = float((p.v.double() * p.v_scale.double()[..., None]).abs().max())
    tol += 2.0 ** -16 * most + np.abs(want) * HALF_STEP[dtype] + TINY[dtype]
    assert (np.abs(host(out) - want) <= tol).all(), float((np.abs(host(out) - want) / tol).max())


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("tokens,n_heads", TILES[1:])
def test_values_scales_far_apart(tokens, n_heads, dtype):
    """int8 rows whose scales are far above the others': that of a token which only itself sees changes nothing of the rows that do not see
    it; that of a key which the softmax all but leaves out (2^-60 next to 1) counts by its weight."""
    d, ctx = 64, 100
    seen = [1 << j if j == 1 else ((2 << j) - 1) & ~2 for j in range(tokens)]
    p = Place([tokens], [ctx], n_kv=1, d=d, cache=I8, seen=seen)
    q = randn((tokens, n_heads * d), dtype, 3, scale=0.2)
    clean = B.moe_window_attention(p.cache, p.window, q, 0.125)
    rows = [j for j in range(tokens) if j != 1]
    page, slot = p.key_at(0, ctx + 1)
    p.v_scale[page, 0, slot] = 2.0 ** 60
    out = B.moe_window_attention(p.cache, p.window, q, 0.125)
    assert torch.equal(out[rows], clean[rows]) and torch.isfinite(clean).all()
    # a key whose codes are 127 where q's are negative: a score of -60 log 2 beside zeros
    p = Place([tokens], [ctx], n_kv=1, d=d, cache=I8)
    p.k.zero_()
    page, slot = p.key_at(0, 37)
    p.k[page, 0, slot, 0], p.k_scale[page, 0, slot], p.v_scale[page, 0, slot] = 60, 1.0, 2.0 ** 40
    q = torch.zeros((tokens, n_heads * d), dtype=dtype, device=DEV)
    q.view(tokens, n_heads, d)[:, :, 0] = -1.0
    scale = float(np.float32(np.log(2.0)))
    out = B.moe_window_attention(p.cache, p.window, q, scale)
    want, _, tol, _ = attend_ref(p, q, n_heads, scale)
    assert (np.abs(host(out) - want) <= tol).all() and np.abs(want).max() < 10


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("tokens,n_heads", TILES[1:])
def test_values_that_are_none_reach_rows_that_hardly_weigh_them(tokens, n_heads, dtype):
    """int8 rows whose scale is NaN (a row with an infinity in it) have values that are NaN: of every row that sees the token, also where
    its weight, exp(-200) beside 1, is 0 in float32."""
    seen = [1 << j if j == 1 else ((2 << j) - 1) & ~(2 if j % 2 else 0) for j in range(tokens)]
    p = Place([tokens], [100], n_kv=1, d=64, cache=I8, seen=seen)
    p.k.zero_()
    page, slot = p.key_at(0, 101)
    p.k[page, 0, slot, 0], p.k_scale[page, 0, slot], p.v_scale[page, 0, slot] = -100, 2.0, float("nan")
    q = torch.zeros((tokens, n_heads * 64), dtype=dtype, device=DEV)
    q.view(tokens, n_heads, 64)[:, :, 0] = 1.0
    out = B.moe_window_attention(p.cache, p.window, q, 1.0)
    for j in range(tokens):
        assert torch.isnan(out[j]).all() if seen[j] & 2 else torch.isfinite(out[j]).all()


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("n", [1, 3, 5000, 70000])
def test_no_log_probability_is_above_none(n, dtype):
    """Rows that are sure of a token: its log probability is 0 to 2^-50 (64-bit roundings next to 1) and no more than 0."""
    x = randn((300, n), dtype, n, 9, scale=3.0)
    x[:, 0] += 90.0 + torch.arange(300, device=DEV).to(dtype) / 7
    for scale in (0.7, 1.0, 1000.0):
        logp, _, _, top = B.moe_token_logprobs(x, tokens=torch.zeros((300, 1), dtype=torch.int32, device=DEV), k=1, scale=scale)
        for y in (logp, top):
            assert (y <= 0).all() and (y >= -2.0 ** -50 - n * np.exp(-60 * scale)).all()
