"""A window's answers from its inputs: rows of one product appended, the tree attended, the outputs multiplied with a head of tokens,
and those logits scored. Each step is compared in 64 bits with the formula on what the step before gave, the first on the
inputs, so that an error at any step shows at the size of that step's own roundings.

Bounds: queries and rows of the cache as test_gpu_window has them (an int8 row's value within half a code and 2^-15 of one), attention's
window_util.attend_ref's, a logit by the float32 sum of its n products, n 2^-24 of their sizes, scores of logits as
test_gpu_window.check_logprobs has them."""
import numpy as np
import pytest
import torch

from moe_routed_expert_route_amd import binding as B
from tests.test_gpu_window import check_logprobs, close, turned
from tests.test_gpu_window_chain import Chain, place
from tests.window_util import BF16, F16, I8, attend_ref, host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,cache", [(BF16, BF16), (F16, F16), (BF16, I8), (F16, I8)])
@pytest.mark.parametrize("tokens,ctx", [((1, 1), (300, 0)), ((5, 1, 8), (300, 0, 1200)), ((40, 3, 64), (90, 700, 0))])
def test_answers_from_the_inputs(tokens, ctx, dtype, cache):
    n_heads, eps, scale = 8, 1e-6, 128 ** -0.5
    ch = Chain(place(cache, tokens, ctx), n_heads, dtype, vocab=700)
    p, c = ch.p, ch.cuts
    kv, d, n = p.n_kv, p.d, p.n
    before = [[[x[:ctx[s]] for x in p.keys(s, h)] for h in range(kv)] for s in range(len(tokens))]
    B.moe_window_append(p.cache, p.window, ch.qkv[:, :c[1]], ch.qkv[:, c[1]:c[2]], ch.qkv[:, c[2]:], freq=ch.freq, q_weight=ch.qw,
                        k_weight=ch.kw, eps=eps, q_out=ch.q)
    B.moe_window_attention(p.cache, p.window, ch.q, scale, out=ch.out, lse=ch.lse, ws=ch.ws)
    logits = ch.out.float() @ ch.head.float().t().contiguous()
    got = check_logprobs(logits, ch.tokens, 5)
    again = B.moe_token_logprobs(logits, tokens=ch.tokens, k=5, entropy=True, ws=ch.ws2)
    assert p.window.errors() == 0 and all(torch.equal(a, b) for a, b in zip(got, again))

    x = host(ch.qkv).reshape(n, n_heads + 2 * kv, d)
    parts = [turned(x[:, a:b], host(w), ch.freq.cpu().numpy(), np.asarray(p.pos), B.ROPE_HALF, 1.0, eps)
             for a, b, w in ((0, n_heads, ch.qw), (n_heads, n_heads + kv, ch.kw))]
    close(host(ch.q).reshape(n, n_heads, d), *parts[0], dtype)
    rows = [parts[1], (x[:, n_heads + kv:], np.abs(x[:, n_heads + kv:]))]
    for s in range(len(tokens)):
        own = slice(p.start[s], p.start[s + 1])
        for a in range(kv):
            for i, y in enumerate(p.keys(s, a)):
                assert np.array_equal(y[:ctx[s]], before[s][a][i])
                want, size = (r[own, a] for r in rows[i])
                if cache is I8:
                    step = np.abs(want).max(-1, keepdims=True) / 127
                    assert (np.abs(y[ctx[s]:] - want) <= step * (0.5 + 2.0 ** -15)).all()
                else:
                    close(y[ctx[s]:], want, size, cache)
    want, lse, tol, lse_tol = attend_ref(p, ch.q, n_heads, scale)
    assert (np.abs(host(ch.out) - want) <= tol).all() and (np.abs(host(ch.lse) - lse) <= lse_tol).all()
    out, head = host(ch.out), host(ch.head)
    assert (np.abs(host(logits) - out @ head.T) <= head.shape[1] * 2.0 ** -24 * (np.abs(out) @ np.abs(head).T)).all()
