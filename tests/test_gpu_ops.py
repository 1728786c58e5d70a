"""The calls around the layer (moe_add_rmsnorm, moe_route_scores, moe_swiglu_i8, moe_matmul_i8) against
64-bit references in numpy, through the binding.

Tolerances, from the definitions (a rounding is off by at most half a step: relative 2^-24 in float32,
2^-8 in bfloat16, 2^-11 in float16; SLACK covers the 64-bit evaluation itself, some tens of operations of
2^-53 each):
* y and w: evaluated in 64 bits, rounded to float32 (and y then to its type).
* codes of y: exact, by the rule in float32 on the call's own float32 y.
* codes of h, which is not returned: |q - h / d| <= 1/2 + 2^-16. h is within 2^-24 of the 64-bit value, the
  float32 quotient within 2^-24 of the true one, and |h / d| < 128, so 128 * 2 * 2^-24 = 2^-16 covers both;
  d = float32(max|h| / 127) is within 2^-23 of its 64-bit value (the rounding of h, then its own).
* products: bit for bit, since the integer sum is exact and each float32 step is stated.
"""
import numpy as np
import pytest
import torch

import oracle
from moe_routed_expert_route_amd import binding as B
from moe_routed_expert_route_amd import synth

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
HALF_STEP = {F32: 2.0 ** -24, BF16: 2.0 ** -8, F16: 2.0 ** -11}
SLACK = 2.0 ** -44
TINY = {F32: 2.0 ** -149, BF16: 2.0 ** -133, F16: 2.0 ** -24}   # a step of the smallest values
DEV = "cuda:0"


def randn(shape, dtype, *key, scale=1.0):
    return torch.from_numpy(scale * synth.rng(*key).standard_normal(shape)).to(dtype).to(DEV)


def rows_in(rows, n, dtype, ld=None, offset=0, fill=None):
    """A [rows, n] view with row stride ld inside a larger buffer (returned too), `offset` elements in."""
    ld = ld or n
    buf = torch.full((offset + (rows + 1) * ld,), fill if fill is not None else 0, dtype=dtype, device=DEV)
    return buf.as_strided((rows, n), (ld, 1), offset), buf


def host(t):
    return t.detach().cpu().double().numpy()


def code_rule(y, axis):
    """Codes and float32 scale of float32 values: quotient in float32, halves away from zero."""
    y = y.astype(np.float32)
    d = (np.abs(y).max(axis, keepdims=True) / np.float32(127)).astype(np.float32)
    v = np.divide(y, d, out=np.zeros_like(y), where=d > 0).astype(np.float64)
    t = np.trunc(v)
    return np.clip(t + np.where(np.abs(v - t) >= 0.5, np.sign(v), 0), -127, 127).astype(np.int8), d.squeeze(axis)


# ------------------------------------------------------------------ norm ------------------------

def norm_ref(r, weight, eps):
    return r / np.sqrt((r * r).mean(1) + eps)[:, None] * weight[None]


def check_norm(x, weight, res=None, eps=1e-6, y_dtype=F32, want_q81=False, res_out=None):
    rows, n = x.shape
    x0, res0 = x.clone(), None if res is None else res.clone()
    y, _ = rows_in(rows, n, F32)
    q, d = B.i8_rows(rows, n, DEV)
    blocks = torch.empty((rows, n // 32 * 36), dtype=torch.uint8, device=DEV) if want_q81 else None
    out = res_out if res_out is not None else torch.empty_like(x0)
    B.moe_add_rmsnorm(x, weight, eps, res=res, res_out=out, y=y, q=q, scale=d, q8_1=blocks)
    r = x0 if res0 is None else (x0.cpu().float() + res0.cpu().float()).to(x0.dtype).to(DEV)
    assert torch.equal(out, r)
    want = norm_ref(host(r), host(weight), eps)
    got = host(y)
    assert (np.abs(got - want) <= np.abs(want) * (HALF_STEP[F32] + SLACK) + TINY[F32]).all()
    codes, scale = code_rule(y.cpu().numpy(), 1)
    assert np.array_equal(q.cpu().numpy(), codes)
    assert np.array_equal(d.cpu().numpy(), scale)
    if want_q81:
        assert np.array_equal(blocks.cpu().numpy(), oracle.quantize_q8_1(y.cpu().numpy()).reshape(blocks.shape))
        assert torch.equal(blocks, B.moe_quantize_q8_1(y))
    if y_dtype != F32:
        x.copy_(x0)
        if res is not None:
            res.copy_(res0)
        y2 = torch.empty((rows, n), dtype=y_dtype, device=DEV)
        B.moe_add_rmsnorm(x, weight, eps, res=res, y=y2)
        assert torch.equal(y2.cpu(), y.cpu().to(y_dtype))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows,n", [(1, 1), (3, 2), (2, 31), (5, 64), (3, 257), (4, 1000), (2, 2560), (3, 4097), (2, 8192),
                                    (1, 16383), (2, 16384), (70, 96)])
def test_norm(rows, n, dtype):
    x, res = randn((rows, n), dtype, rows, n, 1), randn((rows, n), dtype, rows, n, 2, scale=3.0)
    w = randn((n,), dtype, n, 3) + 1
    check_norm(x, w, res, y_dtype=dtype, want_q81=n % 32 == 0)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_norm_without_residual_with_float_weight(dtype):
    check_norm(randn((9, 640), dtype, 4), randn((640,), F32, 5), y_dtype=BF16, want_q81=True)


@pytest.mark.parametrize("onto", ["x", "res"])
def test_norm_in_place(onto):
    x, res = randn((6, 1536), BF16, 6), randn((6, 1536), BF16, 7)
    check_norm(x, randn((1536,), BF16, 8), res, res_out=x if onto == "x" else res)


@pytest.mark.parametrize("dtype,ld,offset", [(F32, 131, 1), (BF16, 133, 3), (F16, 136, 8), (BF16, 1 << 12, 5)])
def test_norm_strides_and_untouched_bytes(dtype, ld, offset):
    rows, n = 7, 130
    x, _ = rows_in(rows, n, dtype, ld, offset)
    x.copy_(randn((rows, n), dtype, 9))
    res, _ = rows_in(rows, n, dtype, ld + 3, offset)
    res.copy_(randn((rows, n), dtype, 10))
    w = randn((n + 1,), dtype, 11)[1:]
    out, out_buf = rows_in(rows, n, dtype, ld + 1, offset, 7)
    y, y_buf = rows_in(rows, n, F16, ld + 2, offset, 7)
    q, q_buf = rows_in(rows, n, torch.int8, ld, offset, 99)
    d = torch.full((rows + 2,), 5.0, device=DEV)
    B.moe_add_rmsnorm(x, w, 1e-5, res=res, res_out=out, y=y, q=q, scale=d[1:-1])
    r = (x.float() + res.float()).to(dtype)
    assert torch.equal(out, r)
    want = torch.from_numpy(norm_ref(host(r), host(w), 1e-5).astype(np.float32))
    # float16 of float32 of the 64-bit value; a second rounding may differ where the first one does
    assert (np.abs(host(y) - host(want)) <= np.abs(host(want)) * (2.0 ** -11 + 2.0 ** -23) + TINY[F16]).all()
    codes, scale = code_rule(want.numpy(), 1)
    assert np.abs(q.cpu().numpy().astype(int) - codes).max() <= 1 and (q.cpu().numpy() != codes).mean() < 0.01
    assert d[0] == 5 and d[-1] == 5 and np.allclose(d[1:-1].cpu().numpy(), scale, rtol=2.0 ** -22, atol=0)
    for view, buf, fill in ((out, out_buf, 7), (y, y_buf, 7), (q, q_buf, 99)):
        view.fill_(fill)
        assert (buf == fill).all()


def test_norm_rows_alone_and_among_others():
    x, w = randn((37, 2560), BF16, 12), randn((2560,), BF16, 13)
    q, d = B.i8_rows(37, 2560, DEV)
    y = torch.empty((37, 2560), device=DEV)
    B.moe_add_rmsnorm(x, w, 1e-6, y=y, q=q, scale=d)
    q1, d1 = B.i8_rows(1, 2560, DEV)
    y1 = torch.empty((1, 2560), device=DEV)
    B.moe_add_rmsnorm(x[36:], w, 1e-6, y=y1, q=q1, scale=d1)
    assert torch.equal(q1, q[36:]) and torch.equal(d1, d[36:]) and torch.equal(y1, y[36:])


def test_norm_rows_of_zeros_infinities_and_nans():
    x = randn((6, 96), F32, 14)
    x[1] = 0
    x[2, 5] = float("inf")
    x[3, 7] = float("nan")
    x[4] = 2.0 ** -140 * x[4].sign()
    x[5] = 1e30 * x[5].sign()
    w = torch.ones(96, device=DEV)
    y = torch.empty_like(x)
    q, d = B.i8_rows(6, 96, DEV)
    blocks = torch.empty((6, 108), dtype=torch.uint8, device=DEV)
    B.moe_add_rmsnorm(x, w, 1e-6, y=y, q=q, scale=d, q8_1=blocks)
    q, d, yh = q.cpu().numpy(), d.cpu().numpy(), y.cpu().numpy()
    assert not q[1].any() and d[1] == 0 and not yh[1].any()
    assert not q[2].any() and np.isnan(d[2]) and not q[3].any() and np.isnan(d[3])
    assert np.isnan(yh[3]).all() and np.isnan(yh[2, 5]) and not yh[2, :5].any()
    for i in (0, 4, 5):
        codes, scale = code_rule(yh[i:i + 1], 1)
        assert np.array_equal(q[i], codes[0]) and d[i] == scale[0]
    assert (np.abs(yh[5]) == 1).all()
    assert torch.equal(blocks, B.moe_quantize_q8_1(y))
    w[3] = float("nan")   # a NaN among finite values, in every row
    w[4] = float("inf")
    B.moe_add_rmsnorm(x, w, 1e-6, y=y, q8_1=blocks)
    assert torch.equal(blocks, B.moe_quantize_q8_1(y))


def test_norm_rows_side_by_side_in_one_buffer():
    """x, its sum, float rows and int8 rows as column ranges of one buffer: no byte is shared."""
    buf = torch.zeros((5, 512), device=DEV)
    x, r, y = buf[:, :100], buf[:, 100:200], buf[:, 200:300]
    q = buf.view(torch.int8)[:, 1200:1300]
    x.copy_(randn((5, 100), F32, 15))
    keep, d, w = x.clone(), torch.empty(5, device=DEV), randn((100,), F32, 16)
    B.moe_add_rmsnorm(x, w, 1e-6, res_out=r, y=y, q=q, scale=d)
    assert torch.equal(x, keep) and torch.equal(r, keep) and not buf[:, 325:].any()
    codes, scale = code_rule(y.cpu().numpy(), 1)
    assert np.array_equal(q.cpu().numpy(), codes) and np.array_equal(d.cpu().numpy(), scale)
    with pytest.raises(RuntimeError, match="bad argument"):
        B.moe_add_rmsnorm(x, w, 1e-6, y=buf[:, 50:150])


# ------------------------------------------------------------------ router ----------------------

def route_ref(logits, k, score, bias, n_groups, keep, top, renorm, factor):
    """One token at a time, in 64 bits."""
    ids_all, w_all = [], []
    for l in logits:
        live = ~np.isnan(l) & (l != -np.inf)
        l = np.minimum(l, 3.4028234663852886e38)
        E = len(l)
        s = np.zeros(E)
        if live.any():
            with np.errstate(over="ignore"):
                s[live] = np.exp(l[live] - l[live].max()) if score == B.SCORE_SOFTMAX else 1 / (1 + np.exp(-l[live]))
            if score == B.SCORE_SOFTMAX:
                s /= s.sum()
        c = s + bias if bias is not None else s
        per = E // n_groups
        group = []
        for g in range(n_groups):
            best = sorted((c[e] for e in range(g * per, (g + 1) * per) if live[e]), reverse=True)[:top]
            group.append(sum(best) if best else -np.inf)
        kept = sorted(range(n_groups), key=lambda g: (-group[g], g))[:keep]
        order = c if bias is not None else l
        pool = [e for g in kept for e in range(g * per, (g + 1) * per)]
        ids = sorted(pool, key=lambda e: (not live[e], -order[e] if live[e] else 0.0, e))[:k]
        w = s[ids]
        if renorm and w.sum() > 0:
            w = w / w.sum()
        ids_all.append(ids)
        w_all.append(w * factor)
    return np.array(ids_all, np.int32), np.array(w_all)


def check_route(logits, k, score=B.SCORE_SOFTMAX, bias=None, n_groups=1, keep=1, top=1, renorm=True, factor=1.0):
    ids, w = B.moe_route_scores(logits, k, score=score, bias=bias, n_groups=n_groups, keep_groups=keep, group_top=top,
                                renorm=renorm, factor=factor)
    rid, rw = route_ref(host(logits), k, score, None if bias is None else host(bias), n_groups, keep, top, renorm,
                        float(np.float32(factor)))
    assert np.array_equal(ids.cpu().numpy(), rid)
    assert (np.abs(host(w) - rw) <= np.abs(rw) * (HALF_STEP[F32] + SLACK) + TINY[F32]).all()
    return ids, w


SIG, SOFT = B.SCORE_SIGMOID, B.SCORE_SOFTMAX


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("T,E,k,score,bias,groups,keep,top,renorm", [
    (1, 1, 1, SOFT, False, 1, 1, 1, True), (1, 128, 8, SOFT, False, 1, 1, 1, True), (4, 128, 8, SIG, False, 1, 1, 1, True),
    (33, 7, 7, SOFT, True, 1, 1, 1, False), (65, 256, 8, SIG, True, 8, 4, 2, True), (5, 63, 32, SOFT, True, 1, 1, 1, True),
    (9, 160, 6, SOFT, False, 8, 3, 1, False), (130, 64, 4, SIG, True, 4, 2, 2, True), (3, 1024, 32, SIG, True, 64, 13, 2, True),
    (3, 1000, 10, SOFT, False, 1, 1, 1, False), (6, 65, 5, SOFT, True, 13, 2, 1, True), (2, 64, 32, SIG, True, 64, 40, 1, True),
    (21, 192, 12, SIG, False, 3, 2, 2, False), (7, 320, 1, SOFT, True, 2, 1, 2, True), (40, 512, 12, SIG, True, 1, 1, 1, True),
    (17, 96, 16, SOFT, False, 1, 1, 1, False), (9, 64, 10, SIG, True, 4, 2, 2, True), (6, 128, 9, SOFT, True, 16, 5, 2, True),
    (5, 500, 16, SOFT, True, 4, 1, 1, False), (11, 256, 11, SIG, False, 8, 3, 2, True), (3, 16, 16, SIG, True, 16, 16, 1, True)])
def test_route(T, E, k, score, bias, groups, keep, top, renorm, dtype):
    logits = randn((T, E), dtype, T, E, k, scale=2.0)
    b = randn((E,), F32, E, 1, scale=0.1) if bias else None
    check_route(logits, k, score, b, groups, keep, top, renorm, factor=1.0 if T % 2 else 2.5)


@pytest.mark.parametrize("score", [SIG, SOFT])
@pytest.mark.parametrize("E,k,groups", [(256, 8, 8), (200, 12, 1), (128, 8, 2), (512, 10, 16)])
def test_route_few_tokens_and_among_many(E, k, groups, score):
    """The bits of a token's choice do not depend on the call's tokens (which may take another kernel)."""
    logits, b = randn((2600, E), F32, E, 28, scale=2.0), randn((E,), F32, E, 29, scale=0.05)
    logits[5, ::3] = float("-inf")
    for renorm in (True, False):
        kw = dict(score=score, bias=b, n_groups=groups, keep_groups=max(1, groups // 2), group_top=2, renorm=renorm)
        ids, w = B.moe_route_scores(logits, k, **kw)
        for rows in (slice(0, 1), slice(3, 9), slice(0, 1000), slice(100, 2000)):
            i, v = B.moe_route_scores(logits[rows], k, **kw)
            assert torch.equal(i, ids[rows]) and torch.equal(v, w[rows])
    check_route(logits[:40], k, score, b, groups, max(1, groups // 2), 2, False)


def test_route_many_tokens_agree_with_the_softmax_router():
    logits = randn((3000, 128), F32, 20, scale=2.0)
    ids, w = B.moe_route_scores(logits, 8)
    ids0, w0 = B.moe_route_topk(logits, 8)
    assert torch.equal(ids, ids0)
    assert torch.allclose(w, w0, rtol=1e-5, atol=0)


@pytest.mark.parametrize("score", [SIG, SOFT])
@pytest.mark.parametrize("groups,keep,top", [(1, 1, 1), (4, 2, 2), (4, 2, 1)])
def test_route_ties_go_to_the_lower_index(score, groups, keep, top):
    flat = torch.zeros((3, 64), device=DEV)
    flat[1] = torch.arange(64, device=DEV) // 5 % 3
    flat[2, 40:] = 1.0
    check_route(flat, 8, score, None, groups, keep, top)
    check_route(flat, 8, score, torch.full((64,), 0.25, device=DEV), groups, keep, top)


@pytest.mark.parametrize("E,k", [(64, 8), (128, 12), (256, 8), (512, 16), (640, 8), (64, 20)])
def test_route_order_of_64_bits(E, k):
    """Scores that float32 cannot tell apart: logits a step from each other, and biases that leave sums
    apart by less than a float32 step, for either score; and equal scores with equal biases."""
    g = synth.rng(21, E)
    base = np.float32(1.0 + g.random((40, 1)))
    logits = (base + np.float32(2.0 ** -23) * g.permuted(np.tile(np.arange(E), (40, 1)), axis=1)).astype(np.float32)
    lt = torch.from_numpy(logits).to(DEV)
    bias = torch.from_numpy((0.5 + 2.0 ** -24 * g.permutation(E)).astype(np.float32)).to(DEV)
    for score in (SIG, SOFT):
        check_route(lt, k, score)
        check_route(lt, k, score, bias)
        check_route(lt, k, score, bias, 8, 3, 2)
        check_route(lt.bfloat16(), k, score, torch.zeros_like(bias))
        check_route(randn((40, E), BF16, E, 27, scale=2.0), k, score, torch.full_like(bias, 0.125), 4, 2, 2)
    # saturated sigmoids order by logit as long as no bias is given
    check_route(lt * 30 + 40, k, SIG)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("score,bias", [(SOFT, False), (SIG, True), (SOFT, True)])
@pytest.mark.parametrize("groups,keep,top", [(1, 1, 1), (8, 3, 2), (8, 2, 1)])
def test_route_masked_experts(dtype, score, bias, groups, keep, top):
    logits = randn((12, 64), dtype, 22, scale=2.0)
    inf = float("inf")
    logits[0] = -inf                      # every expert masked
    logits[1, 3:] = -inf                  # fewer live than k
    logits[2, ::2] = float("nan")
    logits[3, 8:] = -inf                  # whole groups masked
    logits[4, :] = -inf
    logits[4, 63] = 0.5                   # one live expert, in the last group
    logits[5, 17] = inf
    logits[6, [1, 40]] = inf
    logits[7, :32] = -inf
    logits[8, 1::8] = -inf
    check_route(logits, 6, score, randn((64,), F32, 23, scale=0.3) if bias else None, groups, keep, top)


def test_route_extreme_logits():
    logits = randn((8, 96), F32, 24, scale=1.0)
    logits[0] *= 1e4
    logits[1] = 3.4e38 * logits[1].sign()
    logits[2] = -200.0 + logits[2]
    logits[3] = 100.0 + logits[3]
    logits[4, 5:] = -1e30
    check_route(logits[:3], 8, SOFT)
    check_route(logits[4:], 8, SOFT, None, 4, 2, 2, False)
    check_route(logits[2:], 8, SIG)


def test_route_strides_and_untouched_rows():
    view, _ = rows_in(9, 100, BF16, 131, 3, 100.0)
    view.copy_(randn((9, 100), BF16, 25))
    ids = torch.full((11, 6), 77, dtype=torch.int32, device=DEV)
    w = torch.full((11, 6), 7.0, device=DEV)
    B.moe_route_scores(view, 6, ids=ids[1:10], w=w[1:10])
    rid, rw = route_ref(host(view), 6, SOFT, None, 1, 1, 1, True, 1.0)
    assert np.array_equal(ids[1:10].cpu().numpy(), rid)
    assert (ids[[0, 10]] == 77).all() and (w[[0, 10]] == 7).all()


# ------------------------------------------------------------------ SwiGLU ----------------------

def check_codes(q, d, want):
    """Codes and scales of rows against the 64-bit values `want` (bounds: the module's docstring)."""
    q, d, amax = q.cpu().numpy().astype(np.float64), host(d), np.abs(want).max(1)
    assert (np.abs(d - amax / 127) <= amax / 127 * (2.0 ** -23 + SLACK) + 2.0 ** -149).all()
    big = d > 2.0 ** -100
    assert (np.abs(q[big] - np.clip(want[big] / d[big][:, None], -127, 127)) <= 0.5 + 2.0 ** -16).all()
    assert not q[d == 0].any()


def swiglu_ref(g, u):
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-g)) * u


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows,n", [(1, 1), (2, 3), (4, 64), (3, 255), (4, 768), (5, 1001), (2, 2560), (2, 5461), (1, 16384),
                                    (2, 16383), (66, 130)])
def test_swiglu(rows, n, dtype):
    gu = randn((rows, 2 * n), dtype, rows, n, 30, scale=1.5)
    g, u = gu[:, :n], gu[:, n:]
    q, d = B.moe_swiglu_i8(g, u)
    check_codes(q, d, swiglu_ref(host(g), host(u)))


def test_swiglu_wide_gates():
    """Gates from where exp overflows to where it vanishes."""
    g = torch.cat([torch.linspace(-750, 750, 1501), torch.linspace(-110, -80, 300), torch.linspace(-1e-3, 1e-3, 99)])
    g = g.to(DEV)[None].repeat(2, 1)
    u = randn((2, g.shape[1]), F32, 31)
    u[1] = u[1] * torch.exp(-g[1].clamp(max=0).clamp(min=-80))   # brings the small gates' values to the row's scale
    q, d = B.moe_swiglu_i8(g, u)
    check_codes(q, d, swiglu_ref(host(g), host(u)))


def test_swiglu_strides_rows_and_untouched_bytes():
    g, _ = rows_in(5, 77, BF16, 101, 1)
    u, _ = rows_in(5, 77, BF16, 90, 3)
    g.copy_(randn((5, 77), BF16, 32))
    u.copy_(randn((5, 77), BF16, 33))
    q, buf = rows_in(5, 77, torch.int8, 83, 5, 99)
    d = torch.full((7,), 5.0, device=DEV)
    B.moe_swiglu_i8(g, u, q, d[1:6])
    check_codes(q, d[1:6], swiglu_ref(host(g), host(u)))
    q1, d1 = B.moe_swiglu_i8(g[4:], u[4:])
    assert torch.equal(q1, q[4:]) and torch.equal(d1, d[5:6])
    q.fill_(99)
    assert (buf == 99).all() and d[0] == 5 and d[6] == 5


def test_swiglu_rows_of_zeros_infinities_and_nans():
    g, u = randn((5, 40), F32, 34), randn((5, 40), F32, 35)
    g[1] = 0
    u[2, 3] = float("inf")
    g[3, 9] = float("nan")
    g[4], u[4] = 3e38, 3e38          # the product passes float32's range
    q, d = B.moe_swiglu_i8(g, u)
    assert not q[1:].any() and d[1] == 0 and torch.isnan(d[2:]).all() and d[0] > 0


# ------------------------------------------------------------------ product ---------------------

def i8(shape, *key):
    return torch.from_numpy(synth.rng(*key).integers(-128, 128, shape, dtype=np.int8)).to(DEV)


def matmul_ref(a, sa, b, sb, dtype, c0=None):
    s = (a.cpu().double() @ b.cpu().double().t()).numpy()          # whole numbers below 2^53: exact
    v = s.astype(np.float32) * sa.cpu().numpy()[:, None] * sb.cpu().numpy()[None]
    if c0 is not None:
        v = v + c0.cpu().float().numpy()
    return torch.from_numpy(v).to(dtype)


def check_matmul(a, b, dtype=F32, c=None, accumulate=False):
    M, N = a.shape[0], b.shape[0]
    sa = (randn((M,), F32, M, 40, scale=0.3) + 1) * 0.01
    sb = (randn((N,), F32, N, 41, scale=0.3) + 1) * 0.002
    want = matmul_ref(a, sa, b, sb, c.dtype if c is not None else dtype, c if accumulate else None)
    got = B.moe_matmul_i8(a, sa, b, sb, c=c, dtype=dtype, accumulate=accumulate)
    assert torch.equal(got.cpu(), want)


SIZES = [(1, 1, 1), (1, 16, 64), (1, 17, 63), (2, 1536, 2560), (3, 100, 1000), (1, 2560, 768), (4, 33, 65), (5, 2561, 1283),
         (7, 64, 8192), (8, 129, 512), (9, 640, 2560), (15, 128, 128), (16, 16, 16), (17, 257, 129), (31, 512, 640), (33, 31, 33),
         (48, 1000, 1001), (64, 1536, 2560), (65, 65, 65), (100, 2560, 768), (127, 129, 255), (128, 128, 128), (129, 300, 2048),
         (200, 640, 1111), (256, 256, 256), (257, 511, 384), (300, 1024, 1024), (509, 517, 523), (520, 2560, 768),
         (100, 2560, 256), (100, 2561, 255), (512, 1536, 256), (500, 1530, 250), (1024, 1536, 384), (1000, 1531, 383),
         (2048, 1536, 320), (2000, 1533, 321), (4096, 1536, 256), (4090, 1531, 257), (4100, 3301, 200), (3330, 4096, 384), (2048, 6400, 129), (4096, 4096, 144), (700, 777, 130), (1030, 1536, 640), (2050, 513, 192), (1, 8200, 4096), (40, 4096, 97)]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_matmul(M, N, K):
    check_matmul(i8((M, K), M, N, K), i8((N, K), M, N, K, 1))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("M,N,K", [(1, 130, 320), (6, 257, 511), (37, 300, 640), (130, 192, 256), (300, 515, 1000), (600, 1024, 512), (3400, 4100, 272),
                                   (100, 2560, 256), (512, 1536, 256), (1024, 1536, 384), (2048, 1536, 320), (4096, 1536, 256),
                                   (3330, 4096, 384), (500, 1532, 250)])
def test_matmul_types_and_accumulation(M, N, K, dtype):
    a, b = i8((M, K), M, 50), i8((N, K), N, 51)
    check_matmul(a, b, dtype)
    check_matmul(a, b, c=randn((M, N), dtype, M, N, 52), accumulate=True)


@pytest.mark.parametrize("M", [1, 5, 40, 300, 1100, 33000])
@pytest.mark.parametrize("lda,ldb,ldc,off", [(261, 259, 201, 1), (272, 288, 208, 16), (264, 268, 204, 4), (512, 257, 1000, 3)])
def test_matmul_strides_and_untouched_bytes(M, lda, ldb, ldc, off):
    N, K = 200, 257
    a, _ = rows_in(M, K, torch.int8, lda, off, 55)
    b, _ = rows_in(N, K, torch.int8, ldb, off, 55)
    a.copy_(i8((M, K), M, 60))
    b.copy_(i8((N, K), N, 61))
    for dtype in (F32, BF16):
        c, buf = rows_in(M, N, dtype, ldc, off, 7)
        check_matmul(a, b, c=c)
        c.fill_(7)
        assert (buf == 7).all()


def test_matmul_largest_sums():
    """K at its limit with codes that bring the sums to the edge of 32 bits."""
    K = 131071
    a = torch.full((3, K), -128, dtype=torch.int8, device=DEV)
    b = torch.full((20, K), -128, dtype=torch.int8, device=DEV)
    b[1] = 127
    a[2, ::2] = 127
    check_matmul(a, b)
    check_matmul(a.repeat(100, 1), b.repeat(30, 1))


def test_matmul_offsets_past_32_bits():
    """Rows 2^30 bytes apart: the fourth starts past 2^31, the sixth past 2^32."""
    step = 1 << 30
    buf = torch.empty(5 * step + 4096, dtype=torch.int8, device=DEV)
    far = buf.as_strided((6, 1000), (step, 1), 16)
    far.copy_(i8((6, 1000), 70))
    near = i8((40, 1000), 71)
    check_matmul(far, near)
    check_matmul(near, far)
    c = buf[:5 * step].view(torch.float32).as_strided((5, 40), (step // 4, 1), 4096)
    check_matmul(i8((5, 640), 72), i8((40, 640), 73), c=c)


def test_row_calls_offsets_past_32_bits():
    step = 1 << 30
    buf = torch.empty(5 * step + 8192, dtype=torch.int8, device=DEV)
    x = buf[:5 * step].view(BF16).as_strided((5, 640), (step // 2, 1), 0)
    x.copy_(randn((5, 640), BF16, 74))
    q = buf.as_strided((5, 640), (step, 1), 4096)
    d = torch.empty(5, device=DEV)
    near = x.contiguous()
    qn, dn = B.i8_rows(5, 640, DEV)
    w = torch.ones(640, device=DEV)
    B.moe_add_rmsnorm(near, w, 1e-6, q=qn, scale=dn)
    y = buf[:5 * step].view(BF16).as_strided((5, 640), (step // 2, 1), 8192)
    yn = torch.empty((5, 640), dtype=BF16, device=DEV)
    B.moe_add_rmsnorm(near, w, 1e-6, y=yn, q=q, scale=d)
    assert torch.equal(q, qn) and torch.equal(d, dn)
    B.moe_add_rmsnorm(near, w, 1e-6, y=y)
    assert torch.equal(y, yn)
    qs, ds = B.moe_swiglu_i8(x, x)
    qt, dt = B.moe_swiglu_i8(near, near)
    assert torch.equal(qs, qt) and torch.equal(ds, dt)
    l = x.as_strided((5, 64), (step // 2, 1), 0)
    assert torch.equal(B.moe_route_scores(l, 8)[0], B.moe_route_scores(near[:, :64].contiguous(), 8)[0])


def test_zero_rows():
    e = torch.empty((0, 64), device=DEV)
    q, d = B.i8_rows(0, 64, DEV)
    B.moe_add_rmsnorm(e, torch.ones(64, device=DEV), 1e-6, y=torch.empty_like(e), q=q, scale=d)
    ids, w = B.moe_route_scores(e, 4)
    assert ids.shape == (0, 4)
    assert B.moe_swiglu_i8(e, e)[0].shape == (0, 64)
    b, sb = i8((32, 64), 75), torch.ones(32, device=DEV)
    assert B.moe_matmul_i8(q, d, b, sb).shape == (0, 32)
    assert B.moe_matmul_i8(b, sb, q, d).shape == (32, 0)


# ------------------------------------------------------------------ together --------------------

class Block:
    """The front and the shared expert of an MoE layer on the prompt path: norm -> router -> routed experts
    (q8_1 rows) and shared expert (int8 rows), both added into Y."""

    def __init__(self, T, n_embd=256, n_ff=128, E=16, k=4, key=0):
        self.T, self.n, self.n_ff, self.E, self.k = T, n_embd, n_ff, E, k
        self.gate, self.up, self.down = synth.experts(synth.Q8_0, synth.Q8_0, E, n_embd, n_ff, key)
        self.layer = B.Layer(n_embd, n_ff, B.Q8_0, B.Q8_0, self.gate, self.up, self.down, device=DEV)
        self.x, self.res = randn((T, n_embd), F32, key, 80), randn((T, n_embd), F32, key, 81)
        self.weight = randn((n_embd,), F32, key, 82, scale=0.1) + 1
        self.router, self.srouter = i8((E, n_embd), key, 83), torch.full((E,), 1e-3, device=DEV)
        self.bias = randn((E,), F32, key, 84, scale=0.1)
        self.wgu, self.sgu = i8((2 * n_ff, n_embd), key, 85), torch.full((2 * n_ff,), 2e-3, device=DEV)
        self.wd, self.sd = i8((n_embd, n_ff), key, 86), torch.full((n_embd,), 1e-3, device=DEV)
        f = dict(device=DEV)
        self.y, self.sum, self.Y = (torch.empty((T, n_embd), **f) for _ in range(3))
        self.q, self.d = B.i8_rows(T, n_embd, DEV)
        self.xq = torch.empty((T, n_embd // 32 * 36), dtype=torch.uint8, **f)
        self.logits = torch.empty((T, E), **f)
        self.ids, self.w = torch.empty((T, k), dtype=torch.int32, **f), torch.empty((T, k), **f)
        self.plan = B.Plan(min(E, T * k), T * k, device=DEV)
        self.ent_of = torch.empty((T, k), dtype=torch.int32, **f)
        self.g, self.u = torch.empty((T * k, n_ff), **f), torch.empty((T * k, n_ff), **f)
        self.hq = torch.empty((T * k, n_ff // 32 * 36), dtype=torch.uint8, **f)
        self.O = torch.empty((T * k, n_embd), **f)
        self.gu = torch.empty((T, 2 * n_ff), **f)
        self.sq, self.ss = B.i8_rows(T, n_ff, DEV)

    def run(self):
        B.moe_add_rmsnorm(self.x, self.weight, 1e-6, res=self.res, res_out=self.sum, y=self.y, q=self.q, scale=self.d,
                          q8_1=self.xq)
        B.moe_matmul_i8(self.q, self.d, self.router, self.srouter, c=self.logits)
        B.moe_route_scores(self.logits, self.k, score=B.SCORE_SIGMOID, bias=self.bias, n_groups=4, keep_groups=2,
                           group_top=2, factor=2.5, ids=self.ids, w=self.w)
        B.moe_prefill_plan(self.ids, self.w, self.plan, self.E, ent_of=self.ent_of)
        B.moe_prefill_gate_up(self.layer, self.plan, self.xq, self.g, self.u)
        B.moe_prefill_swiglu_q8_1(self.plan, self.g, self.u, self.n_ff, self.hq)
        B.moe_prefill_down(self.layer, self.plan, self.hq, self.O)
        torch.mul(self.sum, 1.0, out=self.Y)
        B.moe_prefill_scatter(self.plan, self.ent_of, self.O, self.Y, self.n)
        B.moe_matmul_i8(self.q, self.d, self.wgu, self.sgu, c=self.gu)
        B.moe_swiglu_i8(self.gu[:, :self.n_ff], self.gu[:, self.n_ff:], self.sq, self.ss)
        B.moe_matmul_i8(self.sq, self.ss, self.wd, self.sd, c=self.Y, accumulate=True)

    def outputs(self):
        return [t.clone() for t in (self.sum, self.y, self.q, self.d, self.xq, self.ids, self.w, self.sq, self.ss, self.Y)]


@pytest.mark.parametrize("T", [1, 5, 70])
def test_block_against_the_oracle(T):
    b = Block(T, key=T)
    b.run()
    assert b.plan.errors() == 0
    y = b.y.cpu().numpy()
    rid, rw = route_ref(host(b.logits), b.k, B.SCORE_SIGMOID, host(b.bias), 4, 2, 2, True, 2.5)
    assert np.array_equal(b.ids.cpu().numpy(), rid)
    w32 = b.w.cpu().numpy()
    assert np.abs(w32 - rw).max() <= 2.5 * 2.0 ** -24
    ref = oracle.layer(y, oracle.build_plan(rid, w32, None, b.E, 0), oracle.Q8_0, oracle.Q8_0, b.gate, b.up, b.down, b.n,
                       b.n_ff, b.sum.cpu().numpy(), oracle.Tables())
    gu = matmul_ref(b.q, b.d, b.wgu, b.sgu, F32)
    assert torch.equal(b.gu.cpu(), gu)
    check_codes(b.sq, b.ss, swiglu_ref(host(gu[:, :b.n_ff]), host(gu[:, b.n_ff:])))
    shared = host(matmul_ref(b.sq, b.ss, b.wd, b.sd, F32))
    # the routed part within the library's 2e-5 of the sum of its terms' sizes, then one more float32 sum
    assert (np.abs(host(b.Y) - ref["Y"] - shared) <= 2e-5 * ref["S"] + 2.0 ** -23 * (np.abs(ref["Y"]) + np.abs(shared))).all()


@pytest.mark.parametrize("T", [1, 70])
def test_block_captured_and_replayed(T):
    b = Block(T, key=T)
    b.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        b.run()
        with torch.cuda.graph(graph, stream=side):
            b.run()
    for i in range(4):
        b.x.copy_(randn((T, b.n), F32, i, 90))
        b.res.copy_(randn((T, b.n), F32, i, 91))
        b.run()
        torch.cuda.synchronize()
        want = b.outputs()
        for t in (b.sum, b.y, b.d, b.w, b.ss, b.Y):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for got, w in zip(b.outputs(), want):
            assert torch.equal(got, w)


def test_router_counts_are_refused_before_they_lose_bits():
    l = randn((2, 8), F32, 17)
    for bad in (dict(k=0), dict(k=9), dict(k=(1 << 32) + 1), dict(k=1, n_groups=(1 << 32) + 1), dict(k=1, n_groups=2, keep_groups=3),
                dict(k=1, group_top=(1 << 32) + 1), dict(k=1, keep_groups=0)):
        with pytest.raises(ValueError, match="of 8 experts"):
            B.moe_route_scores(l, **bad)


def test_named_stream_allocates_there_too():
    side = torch.cuda.Stream()
    a, b, s = i8((40, 640), 92), i8((300, 640), 93), torch.ones(300, device=DEV)
    want = B.moe_matmul_i8(a, s[:40], b, s)
    torch.cuda.synchronize()
    for _ in range(20):   # results of the side stream outlive work of the current one that could take their memory
        got = B.moe_matmul_i8(a, s[:40], b, s, stream=side)
        torch.full((40, 300), float("nan"), device=DEV)
        side.synchronize()
        assert torch.equal(got, want)
        del got
    assert torch.cuda.current_stream() != side


def test_two_streams_at_once():
    a, b = Block(33, key=1), Block(34, key=2)
    a.run(), b.run()
    torch.cuda.synchronize()
    want = a.outputs() + b.outputs()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(s1):
            a.run()
        with torch.cuda.stream(s2):
            b.run()
    torch.cuda.synchronize()
    for got, w in zip(a.outputs() + b.outputs(), want):
        assert torch.equal(got, w)


def test_matmul_with_more_channels_than_the_usual_launch_takes():
    """17 tokens past the few-token kernel's channels, and 33 past those of the tile of least cost."""
    for M, N in ((17, 134217712 + 96), (33, 1 << 30)):
        K = 3
        need = 2 * M * N + K * N + 4 * N + (8 << 30)
        if torch.cuda.mem_get_info()[0] < need:
            pytest.skip(f"{need >> 30} GiB of memory are not free")
        g = torch.Generator(device=DEV).manual_seed(M)
        a = torch.randint(-128, 128, (M, K), generator=g, device=DEV, dtype=torch.int8)
        b = torch.randint(-128, 128, (N, K), generator=g, device=DEV, dtype=torch.int8)
        sa, sb = torch.rand(M, generator=g, device=DEV) + 0.5, torch.rand(N, generator=g, device=DEV) + 0.5
        c = torch.full((M, N), float("nan"), dtype=BF16, device=DEV)
        B.moe_matmul_i8(a, sa, b, sb, c=c)
        for n in range(0, N, 1 << 26):
            e = min(N, n + (1 << 26))
            for m in range(M):
                sums = sum(a[m, i].float() * b[n:e, i].float() for i in range(K))   # whole numbers below 2^24
                assert torch.equal(c[m, n:e], (sums * sa[m] * sb[n:e]).to(BF16))
        del a, b, sa, sb, c
        torch.cuda.empty_cache()


# g:u as the bits of float32 values, found by search: h lies 2^-50 to 2^-48 of itself from a float32 rounding border
NEAR_BORDERS = """
    c072d972:3fe4a77a c0d300c6:3fb6113f c0486ecd:3fbee7a5 c0bd25f6:3fb1b527 c0a6ed55:3fadda4b bf840b27:3fd8f94f
    c09056d9:3fa1b680 c0e83ba2:3ff76784 bf87d31c:3fafa216 c0e9097a:3fb29b5d c0d2fb8e:3fc4fdbd bfe12f6e:3fe50595
    bf8261b4:3fcde385 c0a6c65b:3ffaa4e3 c0d25320:3fa15396 c0fe6fb5:3f9688db c0e88e0a:3f8210bf c0e88e0a:3f8799a1
    c0e88e0a:3f8d2283 c0e88e0a:3f92ab65 c0e88e0a:3f983447 c0e88e0a:3f9dbd29 c0e88e0a:3fa3460b c0e88e0a:3fa8ceed
    c0e88e0a:3fae57cf c0e88e0a:3fb3e0b1 c0e88e0a:3fb96993 c0e88e0a:3fbef275 c0e88e0a:3fc47b57 c0e88e0a:3fccc8aa
    c0e88e0a:3fd7da6e c0e88e0a:3fe2ec32 c0e88e0a:3fedfdf6 c0e88e0a:3ff90fba 40fd3151:3fa257d2 c0738925:3ff84e5d
    c0e22195:3f9900d2 c0e22195:3fc4b1d5 40ab697a:3fbd09f5 3fbfbcb9:3f885aaa 40f03471:3ffce735 4061beee:3f889fef
    c1715532:3fb00a54 c09fab02:3fdcb560 c09fab02:3ff9a72e c12c6c71:3fe1505f c09910b5:3fb20f30 c09910b5:3feb3875
    c0dc5444:3fe4026d 3fc07060:3fb9384d c17e0489:3fc0a33d 3f0be38e:3f92e251 c0a3fb05:3fccfc29 bee03084:3fbeccac
    40338a84:3f9fd911 40418082:3fe7a83b c18e0513:3fabf7de 40ee06f8:3f802bf6
"""


def test_swiglu_next_to_rounding_borders():
    """h is within 2^-50 of its exact value before its rounding, so these round as the exact values do (in 80 bits
    here). A row of one value: its scale is float32(|h| / 127)."""
    assert np.finfo(np.longdouble).nmant >= 63
    bits = np.array([[int(v, 16) for v in pair.split(":")] for pair in NEAR_BORDERS.split()], np.uint32)
    g, u = bits.view(np.float32).T.astype(np.longdouble)
    h = np.abs(g / (1 + np.exp(-g)) * u)
    m = np.frexp(h)[0] * np.longdouble(2) ** 24
    assert (np.abs(m - np.floor(m) - 0.5) > m * np.longdouble(2) ** -50).all()
    q, d = B.moe_swiglu_i8(*(torch.from_numpy(x.astype(np.float32)[:, None]).to(DEV) for x in (g, u)))
    assert np.array_equal(d.cpu().numpy(), h.astype(np.float32) / np.float32(127))
    assert np.array_equal(q.cpu().numpy()[:, 0], (127 * np.sign(g)).astype(np.int8))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n", [1, 7, 8, 9, 505, 513, 1025, 2048, 2049, 2056, 2560, 4095, 4097, 5461, 8193, 8200, 16377])
def test_swiglu_rows_of_zeros_between_others(n, dtype):
    """Rows of zeros, of either sign and from either factor, where some threads hold no piece of the row, or one of two."""
    g, u = randn((6, n), dtype, n, 37), randn((6, n), dtype, n, 38)
    g[1], u[2], g[3], u[4] = 0, 0, -0.0, -0.0
    q, d = B.moe_swiglu_i8(g, u)
    assert not q[1:5].any() and not d[1:5].any()
    check_codes(q[::5], d[::5], swiglu_ref(host(g[::5]), host(u[::5])))


def test_router_score_kind_is_refused_before_it_loses_bits():
    l = randn((2, 8), F32, 18)
    for score in (0, 3, -1, (1 << 32) + 1, (1 << 32) + 2):
        with pytest.raises(ValueError, match="score"):
            B.moe_route_scores(l, 2, score=score)


def buffers(b):
    """Every buffer that Block.run writes, but for the plan."""
    return [b.sum, b.y, b.q, b.d, b.xq, b.logits, b.ids, b.w, b.ent_of, b.g, b.u, b.hq, b.O, b.Y, b.gu, b.sq, b.ss]


def test_two_streams_at_once_into_cleared_buffers():
    """Each run has to write every output again."""
    blocks = [Block(33, key=1), Block(34, key=2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    want = []
    for b in blocks:
        b.run()
        torch.cuda.synchronize()
        want.append(b.outputs())
    for _ in range(5):
        for b in blocks:
            for t in buffers(b):
                t.fill_(float("nan") if t.is_floating_point() else 77)
            for got, w in zip(b.outputs(), want[0] if b is blocks[0] else want[1]):
                assert not torch.equal(got, w)
        torch.cuda.synchronize()
        for b, s in zip(blocks, streams):
            with torch.cuda.stream(s):
                b.run()
        torch.cuda.synchronize()
        for b, outs in zip(blocks, want):
            for got, w in zip(b.outputs(), outs):
                assert torch.equal(got, w)


def test_results_on_a_named_stream_are_of_its_memory():
    """A result of the current stream takes the block that was just freed there; one of a named stream does not."""
    a, b, s = i8((900, 640), 94), i8((2900, 640), 95), torch.ones(2900, device=DEV)
    logits, g = randn((9000, 300), F32, 96), randn((900, 2000), BF16, 97)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for call in (lambda **kw: B.moe_matmul_i8(a, s[:900], b, s, **kw), lambda **kw: B.moe_route_scores(logits, 30, **kw)[0],
                 lambda **kw: B.moe_route_scores(logits, 30, **kw)[1], lambda **kw: B.moe_swiglu_i8(g, g, **kw)[0]):
        place = call().data_ptr()
        assert call().data_ptr() == place
        want = call()
        torch.cuda.synchronize()
        keep = want.clone()
        del want
        torch.cuda.synchronize()
        got = call(stream=side)
        assert got.data_ptr() != place
        filled = torch.full_like(keep, 77)       # takes the block again, while the side stream may still run
        assert filled.data_ptr() == place
        torch.cuda.synchronize()
        assert torch.equal(got, keep)
        del got, filled, keep


@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("M,N,K", [(1, 256, 512), (6, 256, 512), (12, 256, 512), (24, 256, 512), (40, 2560, 768), (100, 2560, 256),
                                   (512, 1536, 256), (1024, 1536, 384), (2048, 1536, 320), (4096, 1536, 256), (3330, 4096, 384)])
def test_matmul_captured_and_replayed(M, N, K, off):
    """Each of the kernels, rows aligned and not, in a graph of two products, the second added to the first."""
    a, _ = rows_in(M, K, torch.int8, K + 16 + off, off)
    b, _ = rows_in(N, K, torch.int8, K + 16 + off, off)
    sa, sb = torch.rand(M, device=DEV) + 0.5, torch.rand(N, device=DEV) + 0.5
    c, e = torch.empty((M, N), device=DEV), torch.empty((M, N), device=DEV)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        B.moe_matmul_i8(a, sa, b, sb, c=c)
        B.moe_matmul_i8(a, sa, b, sb, c=c, accumulate=True)
    for i in range(4):
        a.copy_(i8((M, K), M, i, 98))
        b.copy_(i8((N, K), N, i, 99))
        B.moe_matmul_i8(a, sa, b, sb, c=e)
        B.moe_matmul_i8(a, sa, b, sb, c=e, accumulate=True)
        torch.cuda.synchronize()
        c.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c, e) and torch.equal(e, 2 * matmul_ref(a, sa, b, sb, F32).to(DEV))


def same(got, want):
    """Equal bits, any NaN equal to any."""
    g, w = got.cpu(), want.cpu()
    assert g.dtype == w.dtype and g.shape == w.shape
    return bool(((g == w) | (g.isnan() & w.isnan())).all())


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("M,N", [(3, 48), (3, 47), (24, 64), (40, 64), (40, 61), (300, 328), (1100, 1536)])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_matmul_scales_of_every_size(M, N, dtype, accumulate):
    """Products below the smallest normal value, past the largest, infinite and NaN scales, also of sums of zero."""
    K = 80
    a, b = i8((M, K), M, 100), i8((N, K), N, 101)
    a[0], b[0] = 0, 0
    sa = torch.exp2(torch.from_numpy(synth.rng(M, 102).uniform(-100, 40, M)).float()).to(DEV)
    sb = torch.exp2(torch.from_numpy(synth.rng(N, 103).uniform(-60, 60, N)).float()).to(DEV)
    sa[1], sb[1] = float("inf"), float("nan")
    sa[2], sb[2] = 0.0, float("-inf")
    sb[3:9] = 1e-45
    c = randn((M, N), F32, M, N, 104).to(dtype)
    c[:, 5] = float("inf")
    c[-1] = float("-inf")
    c[:, 6] = 0
    with np.errstate(all="ignore"):
        want = matmul_ref(a, sa, b, sb, dtype, c if accumulate else None)
    assert same(B.moe_matmul_i8(a, sa, b, sb, c=c, accumulate=accumulate), want)


def test_rows_of_tiny_and_huge_values():
    """Rows whose scale has no normal float32, and rows next to its largest: the rule in float32 on the call's own values."""
    n = 320
    x = randn((9, n), F32, 105)
    w = torch.ones(n, device=DEV)
    for power in (-149, -146, -140, -133, -127, -120, -100, 0, 100, 125):
        w.fill_(2.0 ** power)
        w[::7] *= 0.5
        y, blocks = torch.empty_like(x), torch.empty((9, n // 32 * 36), dtype=torch.uint8, device=DEV)
        q, d = B.i8_rows(9, n, DEV)
        B.moe_add_rmsnorm(x, w, 1e-6, y=y, q=q, scale=d, q8_1=blocks)
        want = norm_ref(host(x), host(w), float(np.float32(1e-6))).astype(np.float32)
        assert (np.abs(host(y) - want) <= np.abs(want) * 2.0 ** -23 + TINY[F32]).all()
        codes, scale = code_rule(y.cpu().numpy(), 1)
        assert np.array_equal(q.cpu().numpy(), codes) and np.array_equal(d.cpu().numpy(), scale)
        assert torch.equal(blocks, B.moe_quantize_q8_1(y))
        for dtype in (BF16, F16):
            z = torch.empty((9, n), dtype=dtype, device=DEV)
            B.moe_add_rmsnorm(x, w, 1e-6, y=z)
            assert torch.equal(z.cpu(), y.cpu().to(dtype))
        # 1 + exp(-90) is 1 in 64 bits, so h is 90 u there
        g = torch.full_like(y, 90.0)
        q, d = B.moe_swiglu_i8(g, y / 128)
        codes, scale = code_rule((host(y / 128) * 90).astype(np.float32), 1)
        assert np.array_equal(q.cpu().numpy(), codes) and np.array_equal(d.cpu().numpy(), scale)


@pytest.mark.parametrize("k", [6, 20])
@pytest.mark.parametrize("groups,keep,top", [(1, 1, 1), (4, 2, 2)])
def test_route_values_that_64_bits_cannot_tell_apart(groups, keep, top, k):
    """Logits below the smallest normal float32 order as they are; biases that swallow the scores leave ties."""
    g = synth.rng(106)
    tiny = torch.from_numpy((g.integers(-40, 41, (9, 64)) * 2.0 ** -149).astype(np.float32)).to(DEV)
    check_route(tiny, k, SOFT, None, groups, keep, top)
    check_route(tiny, k, SIG, None, groups, keep, top)
    logits = randn((9, 64), F32, 107)
    for value in (1e18, -1e18, 3.4e38, -3.4e38, 2.0 ** 54, 2.0 ** 30):
        bias = torch.full((64,), value, device=DEV)
        bias[::5] = 0.5
        check_route(logits, k, SIG, bias, groups, keep, top)
        check_route(logits, k, SOFT, bias, groups, keep, top, False, -1.5)


def test_as_many_rows_as_a_call_takes():
    rows = 4194303
    g = torch.Generator(device=DEV).manual_seed(108)
    x = torch.randn((rows, 16), generator=g, device=DEV).to(BF16)
    w, part = torch.ones(16, device=DEV), slice(rows - 1000, rows)
    q, d = B.i8_rows(rows, 16, DEV)
    B.moe_add_rmsnorm(x, w, 1e-6, q=q, scale=d)
    q1, d1 = B.i8_rows(1000, 16, DEV)
    B.moe_add_rmsnorm(x[part], w, 1e-6, q=q1, scale=d1)
    assert torch.equal(q[part], q1) and torch.equal(d[part], d1)
    assert bool((q.abs().amax(1) == 127).all())
    q, d = B.moe_swiglu_i8(x, x)
    q1, d1 = B.moe_swiglu_i8(x[part], x[part])
    assert torch.equal(q[part], q1) and torch.equal(d[part], d1)
    assert bool((q.abs().amax(1) == 127).all())
    first = torch.where(x == x.amax(1, keepdim=True), torch.arange(16, device=DEV), 16).amin(1).int()
    for k, groups in ((1, 1), (2, 1), (1, 16), (2, 8)):
        ids, v = B.moe_route_scores(x, k, n_groups=groups, keep_groups=groups)
        assert torch.equal(ids[:, 0], first) and bool((v.sum(1) - 1).abs().max() < 2.0 ** -22)


@pytest.mark.parametrize("M", [1, 4, 5, 8])
@pytest.mark.parametrize("N", [1024, 1025, 2048, 2049, 4095, 4096, 8191, 8192])
@pytest.mark.parametrize("K", [1023, 1024, 2047, 2048, 4095, 4096])
def test_matmul_few_tokens_next_to_the_sizes_that_decide(M, N, K):
    check_matmul(i8((M, K), M, K, 110), i8((N, K), N, K, 111), BF16)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M", [2, 7, 14, 40, 300, 1024])
@pytest.mark.parametrize("offsets", [(0, 1, 0, 0, 0), (1, 0, 0, 0, 0), (0, 0, 4, 0, 0), (0, 0, 0, 8, 0), (0, 0, 0, 0, 4), (3, 2, 16, 16, 1)])
def test_matmul_operands_at_any_place(offsets, M, dtype):
    """Scales, rows and C each at an alignment of its own."""
    N, K = 264, 272
    osa, osb, oa, ob, oc = offsets
    sa, sb = torch.rand(M + osa, device=DEV)[osa:] + 0.5, torch.rand(N + osb + 1, device=DEV)[osb:osb + N]
    a, b = rows_in(M, K, torch.int8, K, oa)[0], rows_in(N, K, torch.int8, K, ob)[0]
    a.copy_(i8((M, K), M, 112))
    b.copy_(i8((N, K), N, 113))
    c, buf = rows_in(M, N, dtype, N, oc, 7)
    B.moe_matmul_i8(a, sa, b, sb, c=c)
    want = matmul_ref(a, sa, b, sb, dtype)
    assert torch.equal(c.cpu(), want)
    B.moe_matmul_i8(a, sa, b, sb, c=c, accumulate=True)
    twice = matmul_ref(a, sa, b, sb, dtype, want)
    assert torch.equal(c.cpu(), twice)
    c.fill_(7)
    assert (buf == 7).all()
