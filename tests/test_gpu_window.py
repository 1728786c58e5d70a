"""The calls on windows of tokens over a paged cache (moe_window_append, moe_window_attention) and moe_token_logprobs
against 64-bit references in numpy, through the binding.

Tolerances, from the definitions (a rounding is off by at most half a step, HALF_STEP of the value):
* queries, and 16-bit rows of the cache: evaluated in 64 bits, rounded to float32 and then to their type: the sum of the two half
  steps; where the two terms of a rotation cancel, the 64-bit evaluation itself counts, 2^-46 of the terms.
* int8 rows: |code - y / d| <= 1/2 + 2^-16 with d = max|y| / 127 (y within 2^-24, the quotient within 2^-24 of at most 128), and d
  within 2^-22 (the rounding of y and its own, and the 64-bit evaluation).
* attention: window_util.attend_ref.
* log probabilities: test_logprobs' comment.
"""
import math

import numpy as np
import pytest
import torch

from moe_routed_expert_route_amd import binding as B
from moe_routed_expert_route_amd import synth
from tests.window_util import BF16, DEV, F16, F32, HALF_STEP, I8, TINY, Place, attend_ref, host, tree

pytestmark = pytest.mark.gpu


def randn(shape, dtype, *key, scale=1.0):
    return torch.from_numpy(scale * synth.rng(*key).standard_normal(shape)).to(dtype).to(DEV)


# ------------------------------------------------------------------ append ----------------------

def angles(n_rot, base=10000.0):
    i = np.arange(n_rot // 2)
    return torch.from_numpy((base ** (-2.0 * i / max(n_rot, 1))).astype(np.float32)).to(DEV)


def turned(x, weight, freq, pos, layout, amp, eps):
    """Rows x [n, heads, d] normed and rotated, and the size of the terms of each value."""
    y = x.copy()
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * weight
    size = np.abs(y)
    if freq is not None:
        half = len(freq)
        a, b = (np.arange(half), half + np.arange(half)) if layout == B.ROPE_HALF else (2 * np.arange(half), 2 * np.arange(half) + 1)
        t = pos[:, None].astype(np.float64) * freq[None].astype(np.float64)
        c, s = amp * np.cos(t)[:, None], amp * np.sin(t)[:, None]
        p, r = y[..., a].copy(), y[..., b].copy()
        y[..., a], y[..., b] = p * c - r * s, r * c + p * s
        size[..., a] = size[..., b] = abs(amp) * (np.abs(p) + np.abs(r))
    return y, size


def close(got, want, size, dtype):
    bound = np.abs(want) * (HALF_STEP[dtype] + 2 * HALF_STEP[F32]) + size * 2.0 ** -46 + TINY[dtype]
    assert (np.abs(got - want) <= bound).all()


def check_append(p, n_heads, in_type, out_type, n_rot, layout=B.ROPE_HALF, amp=1.0, norm=True, eps=1e-6, w_type=None, ld=None,
                 in_place=False, key=1):
    d, kv, n = p.d, p.n_kv, p.rows
    wide = (n_heads + 2 * kv) * d
    buf = randn((n, ld or wide), in_type, key, 1)
    q, k, v = buf[:, :n_heads * d], buf[:, n_heads * d:(n_heads + kv) * d], buf[:, (n_heads + kv) * d:wide]
    w_type = w_type or in_type
    qw, kw = (randn((d,), w_type, key, 2) + 1, randn((d,), w_type, key, 3) + 1) if norm else (None, None)
    freq = angles(n_rot) if n_rot else None
    q_out = q if in_place else randn((n, n_heads * d + 16), out_type, key, 4)[:, :n_heads * d]
    before, rows0 = q_out.clone(), buf.clone()
    pools = [t.clone() if t is not None else None for t in (p.k, p.v, p.k_scale, p.v_scale)]
    ret = B.moe_window_append(p.cache, p.window, q, k, v, freq=freq, layout=layout, amp=amp, q_weight=qw, k_weight=kw, eps=eps, q_out=q_out)
    assert ret is q_out and p.window.errors() == 0
    x = host(rows0)[:p.n, :wide].reshape(p.n, n_heads + 2 * kv, d)
    at = np.concatenate([[c + j for j in range(t)] for t, c in zip(p.tokens, p.ctx)] + [[]]).astype(np.int64)
    pos = np.asarray(p.pos) if p.pos is not None else at
    f = None if freq is None else freq.cpu().numpy()
    wq, wk = (None, None) if not norm else (host(qw), host(kw))
    want, size = turned(x[:, :n_heads], wq, f, pos, layout, amp, eps)
    close(host(q_out)[:p.n].reshape(want.shape), want, size, q_out.dtype)
    assert torch.equal(q_out[p.n:], before[p.n:])            # rows of no sequence
    if not in_place:
        assert torch.equal(buf, rows0)
    rows = {"k": turned(x[:, n_heads:n_heads + kv], wk, f, pos, layout, amp, eps), "v": (x[:, n_heads + kv:], np.abs(x[:, n_heads + kv:]))}
    seq = np.repeat(np.arange(len(p.tokens)), p.tokens)
    page = torch.from_numpy(p.table[seq, at // p.page].astype(np.int64)).to(DEV)
    slot = torch.from_numpy(at % p.page).to(DEV)
    for i, name in enumerate("kv"):
        pool, old, (want, size) = (p.k, p.v)[i], pools[i], rows[name]
        got = host(pool[page, :, slot])
        if p.dtype is I8:
            scale = (p.k_scale, p.v_scale)[i]
            dd = host(scale[page, :, slot])
            exact = np.abs(want).max(-1) / 127
            assert (np.abs(dd - exact) <= exact * 2.0 ** -22 + TINY[F32]).all()
            quotient = np.divide(want, dd[..., None], out=np.zeros_like(want), where=dd[..., None] > 0)
            assert (np.abs(got - quotient) <= 0.5 + 2.0 ** -16).all() and np.abs(got).max() <= 127
            scale[page, :, slot] = pools[2 + i][page, :, slot]
            assert torch.equal(scale, pools[2 + i])
        else:
            close(got, want, size, p.dtype)
        pool[page, :, slot] = old[page, :, slot]             # every other row as it was
        assert torch.equal(pool, old)


@pytest.mark.parametrize("cache", [BF16, F16, I8])
@pytest.mark.parametrize("d,n_rot,layout", [(64, 64, B.ROPE_HALF), (128, 128, B.ROPE_HALF), (128, 128, B.ROPE_PAIRS), (80, 36, B.ROPE_PAIRS),
                                            (80, 38, B.ROPE_HALF), (16, 2, B.ROPE_HALF), (16, 14, B.ROPE_PAIRS), (96, 0, B.ROPE_HALF),
                                            (112, 62, B.ROPE_HALF), (192, 96, B.ROPE_HALF), (256, 250, B.ROPE_HALF), (256, 256, B.ROPE_PAIRS),
                                            (240, 6, B.ROPE_HALF)])
def test_append(d, n_rot, layout, cache):
    p = Place([3, 0, 1, 17, 2], [5, 9, 0, 30, 16], d=d, cache=cache, pad=2, key=d + n_rot)
    check_append(p, 6, BF16 if cache is I8 else cache, F16 if cache is F16 else BF16, n_rot, layout, amp=1.0 if d < 100 else 1.25)


@pytest.mark.parametrize("in_type,out_type,w_type", [(F32, BF16, F32), (F32, F32, F32), (BF16, F32, F32), (F16, F16, BF16), (BF16, F16, F16)])
@pytest.mark.parametrize("cache", [BF16, F16, I8])
def test_append_types(in_type, out_type, w_type, cache):
    check_append(Place([2, 5], [7, 100], d=128, cache=cache), 4, in_type, out_type, 64, w_type=w_type)


@pytest.mark.parametrize("order", ["heads", "slots", "wide", "both"])
@pytest.mark.parametrize("page", [16, 48, 256])
def test_append_cache_orders_and_pages(order, page):
    check_append(Place([20, 1, 60], [12, 0, 40], n_kv=3, d=96, page=page, order=order, pad=1), 9, BF16, BF16, 96)


@pytest.mark.parametrize("ld,norm,in_place", [(None, False, True), (8 * 128 + 3, True, False), (8 * 128 + 1, False, False), (2048, True, True)])
def test_append_strides_in_place_and_without_norm(ld, norm, in_place):
    check_append(Place([9, 4], [0, 3], d=128), 4, BF16, BF16, 128, ld=ld, norm=norm, in_place=in_place)


def test_append_one_token_and_many_sequences():
    check_append(Place([1], [0], n_kv=1, d=128), 1, F16, F16, 128)
    rng = synth.rng(5)
    check_append(Place(rng.integers(0, 3, 200), rng.integers(0, 50, 200), n_kv=1, d=64, pad=3), 2, BF16, BF16, 64)


def test_append_far_positions_and_given_ones():
    bits, depth = tree([6, 9], 3)
    pos = [c + e for c, e in zip([1 << 20] * 6 + [(1 << 31) - 20] * 9, depth)]
    check_append(Place([6, 9], [40, 3], d=128, pos=pos), 4, F32, F32, 128)
    check_append(Place([3], [4], d=64, pos=[-1, -100000, 0]), 2, F32, F32, 64)


def test_append_keys_alone():
    p = Place([4], [10], d=64)
    k, v = randn((4, 128), BF16, 1), randn((4, 128), BF16, 2)
    assert B.moe_window_append(p.cache, p.window, None, k, v) is None
    page, slot = zip(*(p.key_at(0, 10 + j) for j in range(4)))
    assert torch.equal(p.k[list(page), :, list(slot)], k.view(4, 2, 64)) and torch.equal(p.v[list(page), :, list(slot)], v.view(4, 2, 64))


def test_append_not_finite():
    p = Place([4], [0], d=64, cache=I8)
    k, v = randn((4, 128), F32, 1), randn((4, 128), F32, 2)
    v[0, 3], v[1, 64], v[2, :64] = math.inf, math.nan, 0.0
    B.moe_window_append(p.cache, p.window, None, k, v)
    page = p.table[0, 0]
    codes, scale = p.v[page].cpu(), p.v_scale[page].cpu()
    assert math.isnan(scale[0, 0]) and math.isnan(scale[1, 1]) and not codes[0, 0].any() and not codes[1, 1].any()
    assert scale[0, 2] == 0 and not codes[0, 2].any() and scale[1, 0] > 0 and scale[0, 3] > 0
    p = Place([1], [0], n_kv=1, d=64)
    q, k, v = torch.ones(1, 64, dtype=F32, device=DEV), k[:1, :64], v[3:, :64]
    out = B.moe_window_append(p.cache, p.window, q, k, v, freq=torch.tensor([math.inf, 2.0 ** 41, 0.5], device=DEV))
    assert p.pos is None and not torch.isfinite(out[0, 0]) and torch.isfinite(out[0, 2])   # infinity times key 0
    p = Place([1], [1], n_kv=1, d=64)
    out = B.moe_window_append(p.cache, p.window, q, k, v, freq=torch.tensor([math.inf, 2.0 ** 41, 0.5], device=DEV))
    assert torch.isnan(out[0, [0, 1, 3, 4]]).all() and torch.isfinite(out[0, [2, 5, 6]]).all()


# ------------------------------------------------------------------ attention -------------------

def check_attention(p, n_heads, dtype, key=1, scale=None, sharp=1.0, ld=0, lse=True, left_out=(), errors=0):
    scale = p.d ** -0.5 if scale is None else scale
    wide = n_heads * p.d
    q = randn((p.rows, wide + ld), dtype, key, 5, scale=sharp)[:, :wide]
    out = randn((p.rows, wide + ld), dtype, key, 6)[:, :wide]
    got_lse = randn((p.rows, n_heads), F32, key, 7) if lse else None
    before, lse0 = out.clone(), got_lse.clone() if lse else None
    ws = B.window_workspace(p.cache, p.window, n_heads)
    ws.fill_(255)
    assert B.moe_window_attention(p.cache, p.window, q, scale, out=out, lse=got_lse, ws=ws) is out
    assert p.window.errors() == errors
    want, want_lse, tol, lse_tol = attend_ref(p, q[:p.n], n_heads, scale, left_out=left_out)
    err = np.abs(host(out)[:p.n] - want)
    assert (err <= tol).all(), float((err / tol).max())
    assert torch.equal(out[p.n:], before[p.n:])
    if lse:
        got = host(got_lse)[:p.n]
        none = np.isneginf(want_lse)
        assert np.array_equal(np.isneginf(got), none) and (np.abs(got[~none] - want_lse[~none]) <= lse_tol[~none]).all()
        assert torch.equal(got_lse[p.n:], lse0[p.n:])
    return out, got_lse


TYPES = [(BF16, BF16), (F16, F16), (BF16, I8), (F16, I8)]


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("d", [16, 48, 64, 80, 96, 128, 144, 192, 256])
def test_attention_head_sizes(d, dtype, cache):
    check_attention(Place([3, 1], [70, 0], d=d, cache=cache), 6, dtype, key=d)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("n_heads,n_kv", [(1, 1), (3, 3), (5, 1), (16, 2), (17, 1), (40, 2)])
@pytest.mark.parametrize("tokens", [[1], [4, 1], [7, 0, 5]])
def test_attention_heads_and_windows(tokens, n_heads, n_kv, dtype, cache):
    p = Place(tokens, [33 * (i + 1) for i in range(len(tokens))], n_kv=n_kv, d=64, cache=cache, pad=1, seen=tree(tokens)[0])
    check_attention(p, n_heads, dtype, key=n_heads)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("ctx", [0, 1, 15, 16, 17, 63, 64, 255, 256, 257, 511, 513, 1023, 1024, 1025])
def test_attention_lengths(ctx, dtype, cache):
    check_attention(Place([2], [ctx], n_kv=1, d=64, cache=cache, page=32), 3, dtype, key=ctx)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("ctx,tokens,n_heads", [(20000, 1, 4), (20000, 64, 1), (2500, 40, 4), (40000, 2, 4), (5000, 33, 2)])
def test_attention_long(ctx, tokens, n_heads, dtype, cache):
    check_attention(Place([tokens, 1], [ctx, ctx // 3], n_kv=1, d=64, cache=cache, page=64, seen=tree([tokens, 1])[0]), n_heads, dtype)


@pytest.mark.parametrize("order", ["heads", "slots", "wide", "both"])
@pytest.mark.parametrize("page", [16, 48, 256])
def test_attention_cache_orders_and_pages(order, page):
    check_attention(Place([5, 2], [300, 77], n_kv=3, d=96, page=page, order=order, pad=1), 6, BF16, ld=3)


@pytest.mark.parametrize("tokens", [64, 63, 33])
@pytest.mark.parametrize("dtype,cache", TYPES)
def test_attention_largest_windows(tokens, dtype, cache):
    bits, _ = tree([tokens, 3, tokens], 9)
    check_attention(Place([tokens, 3, tokens], [200, 0, 0], d=128, cache=cache, seen=bits), 16, dtype)


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_attention_rows_that_see_nothing(dtype, cache):
    seen = [0, 1, 2, 0, 0, 1 << 40 | 1]      # bits past the window count nothing
    p = Place([4, 2], [0, 0], d=64, cache=cache, seen=seen)
    out, lse = check_attention(p, 4, dtype)
    assert not out[[0, 3, 4]].any() and torch.isneginf(lse[[0, 3, 4]]).all()
    check_attention(Place([4, 2], [3, 20], d=64, cache=cache, seen=seen), 4, dtype, lse=False)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("sharp", [0.0, 30.0])
def test_attention_flat_and_sharp(sharp, dtype, cache):
    check_attention(Place([3], [600], d=128, cache=cache), 8, dtype, sharp=sharp)
    check_attention(Place([3], [600], d=128, cache=cache), 8, dtype, scale=-0.3)


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_attention_whatever_masked_places_hold(dtype, cache):
    """Infinities and NaN in slots past the last key, in other pages, and in tokens that a row does not see."""
    tokens, ctx = [5, 3], [70, 9]
    seen = [1, 3, 5, 9, 17, 1, 2, 5]
    p = Place(tokens, ctx, d=64, cache=cache, seen=seen, key=4)
    clean, clean_lse = check_attention(p, 4, dtype)
    keep = {(int(a), b) for s in range(2) for a, b in (p.key_at(s, i) for i in range(tokens[s] + ctx[s]))}
    bad = [(a, b) for a in range(p.n_pages) for b in range(p.page) if (a, b) not in keep]
    poison = [math.nan, math.inf, -math.inf]
    for i, (a, b) in enumerate(bad):
        for pool in ((p.k_scale, p.v_scale) if cache is I8 else (p.k, p.v)):
            pool[a, :, b] = poison[i % 3]
    out, lse = check_attention(p, 4, dtype)
    assert torch.equal(out, clean) and torch.equal(lse, clean_lse)
    # token 4 of the first sequence is seen by itself alone
    a, b = p.key_at(0, 74)
    for pool, value in zip((p.k_scale, p.v_scale) if cache is I8 else (p.k, p.v), (1.0, math.nan)):
        pool[a, :, b] = value
    q = randn((8, 256), dtype, 1, 5)
    out = B.moe_window_attention(p.cache, p.window, q, 0.125)
    rows = [0, 1, 2, 3, 5, 6, 7]
    assert torch.equal(out[rows], clean[rows]) and torch.isnan(out[4]).all()
    if cache is not I8:      # one infinite value: that value of the rows that see it
        p.v[a, :, b] = 1.0
        p.v[a, 0, b, 7] = math.inf
        out = B.moe_window_attention(p.cache, p.window, q, 0.125).view(8, 4, 64)
        assert torch.equal(out[rows], clean.view(8, 4, 64)[rows])
        assert (out[4, :2, 7] == math.inf).all() and torch.isfinite(out[4, 2:]).all() and torch.isfinite(out[4, :2, 8:]).all()


def test_attention_pages_out_of_range():
    p = Place([3, 2], [100, 50], d=64)
    p.window.pages[0, 2], p.window.pages[1, 0] = p.n_pages, -1
    check_attention(p, 4, BF16, left_out=[(0, 32, 48), (1, 0, 16)], errors=256)


def test_sequences_out_of_range_are_left_out():
    """Each bad sequence keeps its rows; the others are as without it."""
    for change in (dict(ctx=-1), dict(ctx=10 ** 6), dict(ctx=2 ** 31 - 1), dict(max_window=2), dict(end=4)):
        p = Place([2, 3, 2], [40, 20, 30], d=64, max_window=change.get("max_window", 3))
        q = randn((7, 256), BF16, 2)
        want = B.moe_window_attention(p.cache, B.Window(p.window.row_start, p.window.ctx_len, p.window.pages, 7, 64), q, 0.1)
        if "ctx" in change:
            p.window.ctx_len[1] = change["ctx"]
        n = change.get("end", 7)
        w = B.Window(p.window.row_start, p.window.ctx_len, p.window.pages, n, p.window.max_window)
        out = torch.full((n, 256), 5.0, dtype=BF16, device=DEV)
        B.moe_window_attention(p.cache, w, q[:n], 0.1, out=out)
        assert w.errors() == 128 and torch.equal(out[:2], want[:2])
        assert (out[2:min(n, 5)] == 5).all()
        if n == 7:
            assert torch.equal(out[5:], want[5:])
        if "max_window" not in change:
            k, v = randn((n, 128), BF16, 3), randn((n, 128), BF16, 4)
            q_out, k0 = torch.full((n, 256), 5.0, dtype=BF16, device=DEV), p.k.clone()
            w = B.Window(p.window.row_start, p.window.ctx_len, p.window.pages, n, 1)
            B.moe_window_append(p.cache, w, q[:n], k, v, q_out=q_out)
            assert w.errors() == 128 and (q_out[2:min(n, 5)] == 5).all() and torch.equal(q_out[:2], q[:2])
            assert int((p.k != k0).any(-1).any(1).sum()) == (4 if n == 7 else 2)


def test_append_page_out_of_range_writes_nothing_there():
    p = Place([3], [14], d=64)
    p.window.pages[0, 1] = p.n_pages
    k0 = p.k.clone()
    q = randn((3, 128), BF16, 1)
    out = B.moe_window_append(p.cache, p.window, q, randn((3, 128), BF16, 2), randn((3, 128), BF16, 3))
    assert torch.equal(out, q) and p.window.errors() == 256
    changed = (p.k != k0).any(-1).any(1).nonzero().tolist()
    assert changed == [[int(p.table[0, 0]), 14], [int(p.table[0, 0]), 15]]


# ------------------------------------------------------------------ log probabilities -----------

def logprobs_ref(x, scale, tokens, k):
    """In 64 bits, with a bound of the error of a log of the sum and of the entropy."""
    x = np.where(np.isnan(x), -np.inf, np.minimum(x, np.finfo(np.float32).max))
    rows, n = x.shape
    out = dict(logp=np.full(tokens.shape, -np.inf), entropy=np.zeros(rows), ids=np.zeros((rows, k), int), top=np.full((rows, k), -np.inf))
    size, spread = np.zeros(rows), np.zeros(rows)
    for r in range(rows):
        out["ids"][r] = np.lexsort((np.arange(n), -x[r]))[:k]
        live = np.isfinite(x[r])
        if not live.any():
            continue
        top = x[r][live].max()
        z = np.where(live, (np.where(live, x[r], 0) - top) * scale, -np.inf)
        e = np.exp(z)
        p = e / e.sum()
        lp = z - np.log(e.sum())
        zz = np.where(p > 0, z, 0)
        out["entropy"][r] = np.log(e.sum()) - (p * zz).sum()
        size[r], spread[r] = np.abs(p * zz).sum(), (p * zz * zz).sum()
        out["top"][r] = lp[out["ids"][r]]
        out["logp"][r] = [lp[t] if 0 <= t < n else -np.inf for t in tokens[r]]
    return out, size, spread


def check_logprobs(x, tokens=None, k=0, scale=1.0, entropy=True):
    """A term exp(z) is off by 2^-22 |z| (the argument in float32) and 2^-22 (exp2), a sum of up to 256 by 2^-16: the log
    of the sum by 2^-16 + 2^-22 (1 + mean|z|). The mean of z: by its terms' errors (mean of z^2 and |z|) and the sums'."""
    rows, n = x.shape
    logp, h, ids, top = B.moe_token_logprobs(x, tokens=tokens, k=k, entropy=entropy, scale=scale)
    t = tokens.cpu().numpy() if tokens is not None else np.zeros((rows, 0), int)
    want, size, spread = logprobs_ref(host(x), scale, t, k)
    tol = 2.0 ** -16 + 2.0 ** -22 * (1 + size)
    if k:
        assert np.array_equal(ids.cpu().numpy(), want["ids"])
    for got, name in ((logp, "logp"), (top, "top")):
        if got is None:
            continue
        got, w = host(got), want[name]
        none = np.isneginf(w)
        assert np.array_equal(np.isneginf(got), none)
        err = np.abs(np.where(none, 0, got) - np.where(none, 0, w))
        assert (err <= tol[:, None] + np.where(none, 0, np.abs(w)) * 2.0 ** -22).all()
    if entropy:
        bound = tol * (2 + 2 * size) + 2.0 ** -22 * (spread + 2 * size) + np.abs(want["entropy"]) * 2.0 ** -23
        assert (np.abs(host(h) - want["entropy"]) <= bound).all()
    else:
        assert h is None
    return logp, h, ids, top


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows,n,k", [(1, 1, 1), (3, 2, 2), (2, 31, 31), (5, 64, 32), (3, 257, 8), (4, 1000, 1), (2, 4095, 20), (2, 4097, 5),
                                      (1, 8192, 32), (3, 16385, 20), (2, 50021, 8), (1, 131072, 32), (70, 300, 3), (1, 262147, 5)])
def test_logprobs(rows, n, k, dtype):
    x = randn((rows, n), dtype, rows, n, scale=3.0)
    tokens = torch.from_numpy(synth.rng(n).integers(0, n, (rows, 3)).astype(np.int32)).to(DEV)
    tokens[:, 1] = n - 1
    check_logprobs(x, tokens, k)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("scale", [0.37, 2.5, 1e-3])
def test_logprobs_scaled_in_padded_rows(scale, dtype):
    buf = torch.full((9, 5003), math.nan, dtype=dtype, device=DEV)
    x = buf[:, 1:5001]
    x.copy_(randn(x.shape, dtype, 8, scale=4.0))
    tokens = torch.tensor([[-1, 5000, 0, 4999, -2 ** 31, 2 ** 31 - 1]] * 9, dtype=torch.int32, device=DEV)
    logp = check_logprobs(x, tokens, 4, scale)[0]
    assert torch.isneginf(logp[:, [0, 1, 4, 5]]).all() and torch.isfinite(logp[:, 2:4]).all()


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("n", [40, 5000, 40000])
def test_logprobs_ties_orders_and_masks(n, dtype):
    i = torch.arange(n, device=DEV)
    rows = [torch.zeros(n, device=DEV), torch.full((n,), -math.inf, device=DEV), i.float() / 64, -i.float() / 64, (i % 7).float(),
            torch.where(i == n - 1, 0.0, -math.inf), torch.where(i % 3 == 1, -math.inf, 1.0), torch.where(i % 2 == 0, -0.0, 0.0),
            torch.where(i < n // 2, math.nan, -1.0), torch.where(i == 3, 60.0, 0.0), torch.full((n,), math.nan, device=DEV),
            torch.where(i < 5, -math.inf, -65000.0), torch.where(i % 11 == 5, 8.0, (i % 5).float()),
            torch.where(i % 1000 < 24, 20.0 + i / n, 0.0)]
    x = torch.stack(rows).to(dtype)
    out = check_logprobs(x, torch.tensor([[0, n - 1]] * len(rows), dtype=torch.int32, device=DEV), 32)
    assert torch.isneginf(out[0][1]).all() and out[1][1] == 0 and torch.isneginf(out[3][1]).all() and out[2][1].tolist() == list(range(32))
    assert out[2][0].tolist() == list(range(32)) and out[2][7].tolist() == list(range(32))


def test_logprobs_infinities_and_the_largest():
    x = torch.tensor([[1.0, math.inf, 2.0, math.nan], [math.inf, math.inf, 0.0, -math.inf], [3.0e38, 3.4e38, 0.0, 1.0]], device=DEV)
    logp, h, ids, top = B.moe_token_logprobs(x, tokens=torch.tensor([[1, 3], [0, 3], [1, 0]], dtype=torch.int32, device=DEV), k=4, entropy=True)
    assert ids.tolist() == [[1, 2, 0, 3], [0, 1, 2, 3], [1, 0, 3, 2]]
    assert logp[0, 0] == 0 and torch.isneginf(logp[0, 1]) and abs(float(logp[1, 0]) + math.log(2)) < 1e-6 and logp[2, 0] == 0
    assert h[0] == 0 and abs(float(h[1]) - math.log(2)) < 1e-6 and h[2] == 0


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("n", [900, 32000, 100000])
def test_logprobs_of_rows_that_are_sure(n, dtype):
    """The sum is 1 and a little more: the terms beside the largest alone are off by 2^-22 |z| and 2^-22 each, their sum by
    2^-16, so that what is left of entropy and log probability keeps its relative precision: 2^-15 (1 + |z|), |z| < 64. The sum
    itself stands in 64 bits next to 1, where some four roundings of 2^-53 are absolute: 2^-50."""
    x = randn((6, n), dtype, n, scale=1.5)
    top = torch.arange(6, device=DEV) * (n // 6) + 3
    x[torch.arange(6, device=DEV), top] = torch.tensor([16.0, 20.0, 24.0, 30.0, 40.0, 55.0], device=DEV).to(dtype)
    logp, h, ids, best = B.moe_token_logprobs(x, tokens=top.int()[:, None], k=2, entropy=True)
    z = x.double() - x.double().amax(1, keepdim=True)
    e = torch.exp(z)
    rest = torch.where(z < 0, e, torch.zeros_like(e)).sum(1)
    want = torch.log1p(rest) - (e * z).sum(1) / (1 + rest)
    assert ((h.double() - want).abs() <= want * 2.0 ** -15 * 65 + 2.0 ** -50).all() and (ids[:, 0] == top).all()
    assert ((logp[:, 0].double() + torch.log1p(rest)).abs() <= torch.log1p(rest) * 2.0 ** -15 + 2.0 ** -50).all() and (h >= 0).all()


@pytest.mark.parametrize("given,k,entropy", [(0, 3, False), (2, 0, False), (0, 0, True), (64, 32, True)])
def test_logprobs_outputs_asked_for(given, k, entropy):
    x = randn((6, 9000), BF16, 3, scale=2.0)
    tokens = torch.randint(0, 9000, (6, given), dtype=torch.int32, device=DEV) if given else None
    check_logprobs(x, tokens, k, entropy=entropy)


def test_logprobs_rows_alone_and_among_others():
    x = randn((41, 30011), BF16, 5, scale=3.0)
    t = torch.arange(41, dtype=torch.int32, device=DEV)[:, None] * 100
    every = B.moe_token_logprobs(x, tokens=t, k=20, entropy=True)
    for r in (0, 17, 40):
        for a, b in zip(every, B.moe_token_logprobs(x[r:r + 1], tokens=t[r:r + 1], k=20, entropy=True)):
            assert torch.equal(a[r:r + 1], b)


def test_append_keeps_an_amplitude_that_float32_does_not_hold():
    """At angles of zero a turned value is the product with amp, of 64 bits, rounded once: bit for bit."""
    p = Place([3, 2], [5, 0], d=64, cache=I8)
    q, k, v = randn((p.rows, 256), F32, 31), randn((p.rows, p.n_kv * 64), F32, 32), randn((p.rows, p.n_kv * 64), F32, 33)
    out = B.moe_window_append(p.cache, p.window, q, k, v, freq=torch.zeros(32, device=DEV), amp=1.2, q_out=torch.empty_like(q))
    assert torch.equal(out[:p.n], (q[:p.n].double() * 1.2).float())
