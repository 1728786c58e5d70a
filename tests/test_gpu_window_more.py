"""Calls on windows that the other tests leave out: prompts in append, of up to 1536 tokens and of more (four tokens a workgroup), every
kind of attention's tiles captured and replayed, and logits far from 0. Tolerances are those of test_gpu_window."""
import copy

import numpy as np
import pytest
import torch

from moe_routed_expert_route_amd import binding as B
from moe_routed_expert_route_amd import synth
from tests.test_gpu_window import TYPES, check_append, check_logprobs, randn
from tests.test_gpu_window_tiles import TILES
from tests.window_util import BF16, DEV, F16, F32, I8, Place, attend_ref, host, tree

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("first", [300, 1324])
@pytest.mark.parametrize("cache", [BF16, F16, I8])
@pytest.mark.parametrize("d,n_rot,layout", [(64, 64, B.ROPE_HALF), (128, 128, B.ROPE_HALF), (128, 100, B.ROPE_PAIRS), (80, 36, B.ROPE_PAIRS),
                                            (16, 2, B.ROPE_HALF), (96, 0, B.ROPE_HALF), (112, 62, B.ROPE_HALF), (256, 250, B.ROPE_HALF),
                                            (240, 6, B.ROPE_PAIRS)])
def test_append_prompts(d, n_rot, layout, cache, first):
    """517 and 1541 tokens, in sequences that begin and end inside a workgroup's four, some of none."""
    p = Place([first, 0, 1, 17, 2, 194, 3], [5, 9, 0, 30, 16, 0, 1], d=d, cache=cache, pad=3, key=d + n_rot)
    check_append(p, 6, BF16 if cache is I8 else cache, F16 if cache is F16 else BF16, n_rot, layout, amp=1.0 if d < 100 else 1.25)


@pytest.mark.parametrize("in_type,out_type,w_type", [(F32, BF16, F32), (F32, F32, F32), (BF16, F32, F32), (F16, F16, BF16)])
@pytest.mark.parametrize("cache", [BF16, I8])
def test_append_prompts_types(in_type, out_type, w_type, cache):
    for n in (511, 1535):
        check_append(Place([n, 2], [7, 100], d=128, cache=cache, page=48, order="wide"), 4, in_type, out_type, 64, w_type=w_type)


@pytest.mark.parametrize("norm,in_place", [(False, True), (True, True), (False, False)])
def test_append_prompts_in_place_of_trees_and_many_sequences(norm, in_place):
    lengths = synth.rng(6).integers(0, 9, 450)
    bits, depth = tree(lengths, 4)
    assert sum(lengths) > 1536
    ctx = synth.rng(7).integers(0, 40, 450)
    pos = [c + e for c, e in zip(np.repeat(ctx, lengths), depth)]
    check_append(Place(lengths, ctx, n_kv=1, d=64, pad=1, pos=pos), 3, BF16, BF16, 64, norm=norm, in_place=in_place)


@pytest.mark.parametrize("n", [600, 1600])
def test_append_prompts_keys_alone(n):
    p = Place([n], [10], d=64, cache=F16)
    k, v = randn((n, 128), F16, 1), randn((n, 128), F16, 2)
    assert B.moe_window_append(p.cache, p.window, None, k, v) is None
    at = np.arange(n) + 10
    page, slot = torch.from_numpy(p.table[0, at // 16].astype(np.int64)).to(DEV), torch.from_numpy(at % 16).to(DEV)
    assert torch.equal(p.k[page, :, slot], k.view(n, 2, 64)) and torch.equal(p.v[page, :, slot], v.view(n, 2, 64))


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("n", [1537, 2051])
def test_append_prompts_whole_and_in_parts(n, dtype, cache):
    """The same bits in one call and in calls of 500 tokens behind one another."""
    q, k, v = randn((n, 512), dtype, 1), randn((n, 256), dtype, 2), randn((n, 256), dtype, 3)
    w, freq = randn((128,), dtype, 4) + 1, torch.rand(64, device=DEV)
    got = []
    for part in (n, 500):
        p = Place([n], [30], d=128, cache=cache)
        q_out = torch.zeros_like(q)
        for i in range(0, n, part):
            m = min(part, n - i)
            ints = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
            one = B.Window(ints(0, m), ints(30 + i), p.window.pages, m)
            B.moe_window_append(p.cache, one, q[i:i + m], k[i:i + m], v[i:i + m], freq=freq, q_weight=w, k_weight=w, q_out=q_out[i:i + m])
            assert one.errors() == 0
        got.append([q_out, p.k, p.v] + ([p.k_scale, p.v_scale] if cache is I8 else []))
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("d", [80, 128, 256])
@pytest.mark.parametrize("tokens,group", TILES)
def test_attention_captured_and_replayed(tokens, group, d, dtype, cache):
    """Lengths, pages, masks and queries change between replays; two graphs on one workspace, replayed one after the other."""
    lengths = [tokens, 2, tokens // 2]
    p = Place(lengths, [900, 40, 300], n_kv=2, d=d, cache=cache, seen=tree(lengths)[0], table_pad=3)
    q = randn((p.n, 2 * group * d), dtype, 8)
    ws, outs = B.window_workspace(p.cache, p.window, 2 * group), [torch.zeros_like(q) for _ in range(2)]
    lses = [torch.zeros((p.n, 2 * group), device=DEV) for _ in range(2)]
    run = lambda i, s: B.moe_window_attention(p.cache, p.window, q, s, out=outs[i], lse=lses[i], ws=ws)
    run(0, 0.1)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for i, g in enumerate(graphs):
        with torch.cuda.graph(g):
            run(i, 0.1 + i)
    for step in range(3):
        p.window.ctx_len.copy_(torch.tensor([900 - 280 * step, 3 * step, 300 - step], dtype=torch.int32))
        p.window.seen.bitwise_or_(1 << step)
        q.copy_(randn(q.shape, dtype, 20 + step))
        ws.fill_(255)
        for t in outs + lses:
            t.fill_(7)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs + lses]
        for i in range(2):
            run(i, 0.1 + i)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, outs + lses))
    assert p.window.errors() == 0


@pytest.mark.parametrize("n,offset", [(5000, 1000.0), (50021, -3000.0), (50021, 1000.0), (140000, 20000.0)])
def test_logits_far_from_zero(n, offset):
    """Float32 rows of a common offset: most values share their first 16 bits, so that a piece's best are among many."""
    x = randn((5, n), F32, n, 3, scale=2.0) + offset
    x[1] = torch.round(x[1] * 4) / 4         # and ties
    x[2, ::3] = float("-inf")
    check_logprobs(x, torch.tensor([[0, 7, n - 1]] * 5, dtype=torch.int32, device=DEV), 32)


def far_apart(rows, n, step, dtype, key):
    """Rows of n values `step` elements apart, in a buffer that is otherwise not written."""
    buf = torch.empty(rows * step, dtype=dtype, device=DEV).view(rows, step)[:, :n]
    buf.copy_(randn((rows, n), dtype, key))
    return buf


@pytest.mark.parametrize("dtype,cache", [(BF16, BF16), (F16, I8)])
def test_offsets_past_32_bits(dtype, cache):
    """Pages 2^28 bytes and more apart (their last 10 GB from the first), rows of queries and outputs 2^24 elements apart (the last 2^32 from
    the first), against the same calls on what lies close together."""
    pages, n_kv, page, d, n_heads, tokens = 40, 2, 16, 64, 4, [20, 1, 64]
    ctx = [300, 40, 0]
    near = Place(tokens, ctx, n_kv=n_kv, d=d, cache=cache)
    assert near.n_pages <= pages
    wide = torch.empty(2 * pages << 27, dtype=cache, device=DEV).view(pages, 2, 1 << 27)[:, :, :n_kv * page * d]
    spread = [pages - 1 - i for i in range(near.n_pages)]
    pools = []
    for i, pool in enumerate((near.k, near.v)):
        far = wide[:, i].view(pages, n_kv, page, d)
        far[spread] = pool
        pools.append(far)
    scales = [None, None]
    if cache is I8:
        scales = [torch.zeros((pages, n_kv, page), device=DEV) for _ in range(2)]
        for far, s in zip(scales, (near.k_scale, near.v_scale)):
            far[spread] = s
    far = B.KVCache(*pools, *scales)
    table = torch.full_like(near.window.pages, -7)
    for s, row in enumerate(near.table):
        for c, x in enumerate(row):
            if x >= 0:
                table[s, c] = spread[x]
    w = B.Window(near.window.row_start, near.window.ctx_len, table, near.rows, near.window.max_window)
    n = near.rows
    q, k, v = randn((n, n_heads * d), dtype, 1), randn((n, n_kv * d), dtype, 2), randn((n, n_kv * d), dtype, 3)
    outs = []
    for cache_, window in ((near.cache, near.window), (far, w)):
        q_out = B.moe_window_append(cache_, window, q, k, v, freq=torch.ones(32, device=DEV))
        outs.append([q_out, B.moe_window_attention(cache_, window, q_out, 0.1)])
        assert window.errors() == 0
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    for i, pool in enumerate((near.k, near.v)):
        assert torch.equal(pools[i][spread], pool)
    if cache is I8:
        return
    step, rows = 1 << 24, 260
    p = Place([rows - 10, 10], [3, 50], n_kv=1, d=d, cache=cache)
    small = B.Window(torch.tensor([250, 260], dtype=torch.int32, device=DEV), p.window.ctx_len[1:], p.window.pages[1:], rows, 10)
    q, q_out = far_apart(rows, 128, step, dtype, 4), far_apart(rows, 128, step, dtype, 5)
    kv = randn((rows, 64), dtype, 6)
    close_q = q.contiguous()
    want = B.moe_window_append(p.cache, p.window, close_q, kv, kv, freq=torch.ones(32, device=DEV))
    k0 = p.k.clone()
    B.moe_window_append(p.cache, p.window, q, kv, kv, freq=torch.ones(32, device=DEV), q_out=q_out)
    assert torch.equal(q_out, want) and torch.equal(p.k, k0) and p.window.errors() == 0
    got = far_apart(rows, 128, step, dtype, 7)
    before = got.clone()
    B.moe_window_attention(p.cache, small, q_out, 0.1, out=got)
    near_out = before.clone()
    B.moe_window_attention(p.cache, small, want, 0.1, out=near_out)
    assert small.errors() == 0 and torch.equal(got, near_out) and torch.equal(got[:250], before[:250]) and not torch.equal(got[250:], before[250:])


def test_logits_past_32_bits():
    x = far_apart(1100, 3000, 1 << 22, F16, 9)
    t = torch.arange(1100, dtype=torch.int32, device=DEV)[:, None]
    for a, b in zip(B.moe_token_logprobs(x, tokens=t, k=9, entropy=True), B.moe_token_logprobs(x.contiguous(), tokens=t, k=9, entropy=True)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("n,group", [(200, 4), (129, 1)])
def test_a_prompt_appended_whole_and_attended_in_parts(n, group, dtype, cache):
    """A prompt longer than attention's windows: appended in one call, then attended as sequences of up to 64 tokens that share its
    pages, each with the ones before it as its context."""
    p = Place([n], [30], n_kv=2, d=128, cache=cache, page=32)
    q, k, v = randn((n, 2 * group * 128), dtype, 1), randn((n, 256), dtype, 2), randn((n, 256), dtype, 3)
    q_out = B.moe_window_append(p.cache, p.window, q, k, v, freq=torch.ones(64, device=DEV) / 7)
    parts = copy.copy(p)
    parts.tokens = [min(64, n - i) for i in range(0, n, 64)]
    parts.ctx = [30 + i for i in range(0, n, 64)]
    parts.start = np.concatenate([[0], np.cumsum(parts.tokens)])
    parts.table = np.repeat(p.table, len(parts.tokens), 0)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    parts.window = B.Window(ints(parts.start), ints(parts.ctx), p.window.pages.expand(len(parts.tokens), -1).contiguous(), n, 64)
    lse = torch.zeros((n, 2 * group), device=DEV)
    out = B.moe_window_attention(p.cache, parts.window, q_out, 128 ** -0.5, lse=lse)
    want, want_lse, tol, lse_tol = attend_ref(parts, q_out, 2 * group, 128 ** -0.5)
    assert (np.abs(host(out) - want) <= tol).all() and (np.abs(host(lse) - want_lse) <= lse_tol).all()
    assert p.window.errors() == 0 and parts.window.errors() == 0
