"""The calls on windows together, as a decoder layer uses them: a window's rows appended, its tree attended, its answers scored;
eagerly and from a captured graph whose inputs change between replays, on two streams, and sequence by sequence.

Tolerance of the whole chain against 64 bits: the queries and keys are rounded to 16 bits once (HALF_STEP relative, twice in a
score: |q| . |k| times two half steps and the products' own), which the bound of window_util.attend_ref takes as an error of the
scores; it is evaluated on the call's own cache and queries, so that only attention's own errors remain.
"""
import numpy as np
import pytest
import torch

from moe_routed_expert_route_amd import binding as B
from tests.test_gpu_window import angles, randn
from tests.window_util import BF16, DEV, F16, F32, I8, Place, attend_ref, host, tree

pytestmark = pytest.mark.gpu


class Chain:
    def __init__(self, p, n_heads, dtype, vocab=5000):
        self.p, self.n_heads, self.vocab = p, n_heads, vocab
        d, kv, n = p.d, p.n_kv, p.rows
        self.cuts = np.cumsum([0, n_heads * d, kv * d, kv * d])
        self.qkv = randn((n, int(self.cuts[3])), dtype, 1, d)
        self.qw, self.kw = randn((d,), dtype, 2) + 1, randn((d,), dtype, 3) + 1
        self.freq = angles(d)
        self.q, self.out = torch.zeros((n, n_heads * d), dtype=dtype, device=DEV), torch.zeros((n, n_heads * d), dtype=dtype, device=DEV)
        self.lse = torch.zeros((n, n_heads), device=DEV)
        self.ws = B.window_workspace(p.cache, p.window, n_heads)
        self.head = randn((vocab, n_heads * d), dtype, 4, scale=0.05)
        self.logits = torch.zeros((n, vocab), dtype=dtype, device=DEV)
        self.tokens = torch.randint(0, vocab, (n, 2), dtype=torch.int32, device=DEV)
        self.ws2 = B.logprobs_workspace(n, vocab, 5)

    def run(self, stream=None):
        p, c = self.p, self.cuts
        B.moe_window_append(p.cache, p.window, self.qkv[:, :c[1]], self.qkv[:, c[1]:c[2]], self.qkv[:, c[2]:], freq=self.freq,
                            q_weight=self.qw, k_weight=self.kw, q_out=self.q, stream=stream)
        B.moe_window_attention(p.cache, p.window, self.q, p.d ** -0.5, out=self.out, lse=self.lse, ws=self.ws, stream=stream)
        return B.moe_token_logprobs(self.logits, tokens=self.tokens, k=5, entropy=True, ws=self.ws2, stream=stream)

    def values(self):
        return [t.clone() for t in (self.q, self.out, self.lse, self.p.k, self.p.v)]


def place(cache, tokens=(5, 1, 8), ctx=(300, 0, 1200), **more):
    bits, depth = tree(tokens, 2)
    pos = [c + e for c, e in zip(np.repeat(ctx, tokens), depth)]
    return Place(list(tokens), list(ctx), n_kv=2, d=128, page=32, cache=cache, seen=bits, pos=pos, key=11, **more)


@pytest.mark.parametrize("dtype,cache", [(BF16, BF16), (F16, F16), (BF16, I8)])
def test_chain(dtype, cache):
    ch = Chain(place(cache), 8, dtype)
    ch.logits.copy_(randn(ch.logits.shape, dtype, 5, scale=2.0))
    logp, h, ids, top = ch.run()
    want, lse, tol, lse_tol = attend_ref(ch.p, ch.q, 8, 128 ** -0.5)
    assert (np.abs(host(ch.out) - want) <= tol).all() and (np.abs(host(ch.lse) - lse) <= lse_tol).all()
    assert ch.p.window.errors() == 0
    x = torch.log_softmax(ch.logits.double(), -1)
    assert torch.allclose(logp.double(), torch.gather(x, 1, ch.tokens.long()), atol=2e-5)
    assert torch.equal(top, torch.gather(x, 1, ids.long()).float()) or torch.allclose(top.double(), torch.gather(x, 1, ids.long()), atol=2e-5)


@pytest.mark.parametrize("dtype,cache", [(BF16, BF16), (F16, I8)])
def test_captured_and_replayed(dtype, cache):
    """Inputs, lengths, pages, positions and masks change between replays; each equals the eager call."""
    ch = Chain(place(cache), 8, dtype)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        ch.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        res = ch.run()
    k0, v0 = ch.p.k.clone(), ch.p.v.clone()
    for i in range(4):
        ch.qkv.copy_(randn(ch.qkv.shape, dtype, 20 + i))
        ch.logits.copy_(randn(ch.logits.shape, dtype, 30 + i, scale=2.0))
        ch.tokens.random_(0, ch.vocab)
        ch.p.window.ctx_len.copy_(torch.tensor([300 - 70 * i, i, 1200 - 299 * i], dtype=torch.int32))
        ch.p.window.seen.bitwise_or_(1 << (i % 3))
        ch.p.window.pos.add_(1)
        ch.p.k.copy_(k0), ch.p.v.copy_(v0), ch.out.fill_(7), ch.ws.fill_(255), ch.ws2.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        got = ch.values() + [t.clone() for t in res]
        ch.p.k.copy_(k0), ch.p.v.copy_(v0), ch.out.fill_(9), ch.ws.fill_(3), ch.ws2.fill_(3)
        eager = ch.run()
        torch.cuda.synchronize()
        for a, b in zip(got, ch.values() + list(eager)):
            assert torch.equal(a, b)
    assert ch.p.window.errors() == 0


def test_two_streams_at_once():
    chains = [Chain(place(c), 8, t) for c, t in ((BF16, BF16), (I8, F16))]
    want = []
    for ch in chains:
        ch.logits.copy_(randn(ch.logits.shape, ch.logits.dtype, 6, scale=2.0))
        res = ch.run()
        want.append(ch.values() + [t.clone() for t in res])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in chains]
    for _ in range(5):
        for ch in chains:
            ch.out.zero_(), ch.q.zero_(), ch.lse.zero_()
        torch.cuda.synchronize()
        res = [ch.run(stream=s) for ch, s in zip(chains, streams)]
        torch.cuda.synchronize()
        for ch, r, w in zip(chains, res, want):
            for a, b in zip(ch.values() + list(r), w):
                assert torch.equal(a, b)


@pytest.mark.parametrize("tokens,n_heads", [([1, 1, 1, 1], 8), ([4, 3, 4, 2], 8), ([40, 64, 7, 33], 4)])
@pytest.mark.parametrize("dtype,cache", [(BF16, BF16), (F16, I8)])
def test_tokens_do_not_depend_on_the_other_sequences(tokens, n_heads, dtype, cache):
    """The same bits whatever the other sequences of the call hold: their contexts replaced by others' lengths and values."""
    ctx = [500, 20, 3000, 0]
    p = Place(tokens, ctx, n_kv=2, d=64, cache=cache, seen=tree(tokens)[0], table_pad=200)
    q = randn((p.n, n_heads * 64), dtype, 3)
    ws = B.window_workspace(p.cache, p.window, n_heads)
    a = B.moe_window_attention(p.cache, p.window, q, 0.2, ws=ws)
    p.window.ctx_len[1], p.window.ctx_len[3] = 0, 0
    q2 = q.clone()
    own = [i for s in (0, 2) for i in range(p.start[s], p.start[s + 1])]
    q2[[i for i in range(p.n) if i not in own]] = 1.5
    b = B.moe_window_attention(p.cache, p.window, q2, 0.2, ws=ws)
    assert torch.equal(a[own], b[own])


@pytest.mark.parametrize("n_seqs", [64, 65, 300])
def test_many_sequences(n_seqs):
    rng = np.random.default_rng(3)
    p = Place(rng.integers(0, 4, n_seqs), rng.integers(0, 90, n_seqs), n_kv=1, d=64, pad=2)
    q = randn((p.rows, 128), BF16, 5)
    out = B.moe_window_attention(p.cache, p.window, q, 0.125)
    want, _, tol, _ = attend_ref(p, q[:p.n], 2, 0.125)
    assert (np.abs(host(out)[:p.n] - want) <= tol).all() and p.window.errors() == 0
