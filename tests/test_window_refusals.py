"""Argument checks of moe_window_append, moe_window_attention and moe_token_logprobs: made on the host before anything is
enqueued, so no GPU is needed. Pointers are fakes that no call below gets to use."""
import ctypes
import os

import pytest
import torch

from moe_routed_expert_route_amd import binding as B

ARG, SHAPE, HIP, WS, OK = -1, -3, -4, -5, 0
P = [i << 40 for i in range(32)]   # far from each other
NAN, INF = float("nan"), float("inf")

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="library not built")
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="would launch kernels on pointers that are fakes")

CACHE = dict(dtype=2, n_pages=10, page_size=32, n_kv=2, head_dim=64, page_stride=4096, head_stride=2048, slot_stride=64, k=P[1],
             v=P[2], k_scale=None, v_scale=None)
I8 = dict(dtype=4, k_scale=P[3], v_scale=P[4])
WINDOW = dict(n_seqs=2, n_tokens=6, max_window=4, max_pages=5, ld_pages=5, row_start=P[5], ctx_len=P[6], pages=P[7], pos=P[8],
              seen=P[9], err=P[10])
APPEND = dict(dtype=2, q=P[11], ldq=256, k=P[12], ldk=128, v=P[13], ldv=128, n_heads=4, w_dtype=2, q_weight=P[14], k_weight=P[15],
              eps=1e-6, freq=P[16], n_rot=64, layout=1, amp=1.0, o_dtype=2, q_out=P[17], ldqo=256)
ATTEND = dict(dtype=2, q=P[11], ldq=256, n_heads=4, scale=0.125, out=P[12], ldo=256, lse=P[13], ws=P[14], ws_bytes=1 << 30)
SCORES = dict(dtype=2, logits=P[1], ld=1000, rows=5, n=1000, scale=1.0, tokens=P[2], given=2, logp=P[3], entropy=P[4], k=8, ids=P[5],
              top=P[6], ws=P[7], ws_bytes=1 << 30)
BASE = {"moe_window_append": APPEND, "moe_window_attention": ATTEND}


def over_cache(name, cache=None, window=None, **change):
    c, w, args = dict(CACHE, **(cache or {})), dict(WINDOW, **(window or {})), dict(BASE[name])
    assert set(c) == set(CACHE) and set(w) == set(WINDOW) and set(change) <= set(args)
    args.update(change)
    return getattr(B.lib(), name)(None, ctypes.byref(B.MoeKvCache(*c.values())), ctypes.byref(B.MoeWindow(*w.values())), *args.values())


BOTH = [
    (dict(cache=dict(dtype=1)), ARG), (dict(cache=dict(dtype=0)), ARG), (dict(cache=dict(n_pages=0)), SHAPE), (dict(cache=dict(page_size=8)), SHAPE),
    (dict(cache=dict(page_size=40)), SHAPE), (dict(cache=dict(page_size=1 << 17)), SHAPE), (dict(cache=dict(n_kv=0)), SHAPE),
    (dict(cache=dict(n_kv=1025)), SHAPE), (dict(cache=dict(head_dim=72)), SHAPE), (dict(cache=dict(head_dim=272)), SHAPE),
    (dict(cache=dict(k=None)), ARG), (dict(cache=dict(v=P[2] + 8)), ARG), (dict(cache=dict(slot_stride=48)), ARG),
    (dict(cache=dict(slot_stride=72)), ARG), (dict(cache=dict(head_stride=1024)), ARG), (dict(cache=dict(page_stride=2048)), ARG),
    (dict(cache=dict(page_stride=-4096)), ARG), (dict(cache=dict(page_stride=1 << 60)), ARG), (dict(cache=dict(slot_stride=1 << 25, page_stride=1 << 40, head_stride=1 << 36)), SHAPE),
    (dict(cache=dict(v=P[1] + 64)), ARG), (dict(cache=dict(v=P[1])), ARG), (dict(cache=dict(k_scale=P[3], v_scale=P[4])), ARG),
    (dict(cache=dict(I8, v_scale=None)), ARG), (dict(cache=dict(I8, k_scale=P[3] + 2)), ARG), (dict(cache=dict(I8, v_scale=P[3] + 64)), ARG),
    (dict(window=dict(n_seqs=-1)), ARG), (dict(window=dict(n_tokens=-1)), ARG), (dict(window=dict(n_seqs=4097)), SHAPE),
    (dict(window=dict(max_window=0)), SHAPE), (dict(window=dict(max_pages=0)), SHAPE), (dict(window=dict(max_pages=1 << 27, ld_pages=1 << 27)), SHAPE),
    (dict(window=dict(ld_pages=4)), ARG), (dict(window=dict(ld_pages=1 << 50)), ARG), (dict(window=dict(row_start=None)), ARG),
    (dict(window=dict(ctx_len=None)), ARG), (dict(window=dict(pages=None)), ARG), (dict(window=dict(err=None)), ARG),
    (dict(window=dict(seen=P[9] + 4)), ARG), (dict(window=dict(pos=P[8] + 2)), ARG), (dict(window=dict(err=P[10] + 1)), ARG),
    (dict(q=P[1] + 256), None), (dict(n_heads=3), SHAPE), (dict(n_heads=0), SHAPE), (dict(n_heads=1026), SHAPE), (dict(dtype=9), ARG),
    (dict(q=P[11] + 1), ARG), (dict(ldq=255), ARG), (dict(window=dict(n_seqs=0)), OK), (dict(window=dict(n_tokens=0)), OK),
]


@pytest.mark.parametrize("name", sorted(BASE))
@pytest.mark.parametrize("change,want", BOTH, ids=str)
def test_cache_and_window_refused(name, change, want):
    if want is None:   # queries within the cache: read only by attention, which a GPU would then run
        if name == "moe_window_append":
            assert over_cache(name, **change) == ARG
        return
    assert over_cache(name, **change) == want


@pytest.mark.parametrize("change,want", [
    (dict(k=None), ARG), (dict(v=None), ARG), (dict(q=None), ARG), (dict(q_out=None), ARG), (dict(o_dtype=4), ARG), (dict(w_dtype=0), ARG),
    (dict(eps=0.0), ARG), (dict(eps=NAN), ARG), (dict(eps=INF), ARG), (dict(amp=INF), ARG), (dict(amp=NAN), ARG), (dict(layout=0), ARG),
    (dict(layout=3), ARG), (dict(n_rot=63), SHAPE), (dict(n_rot=66), SHAPE), (dict(n_rot=-2), SHAPE), (dict(freq=None), ARG), (dict(ldk=127), ARG),
    (dict(ldv=127), ARG), (dict(ldqo=255), ARG), (dict(q_out=P[11] + 64), ARG), (dict(q_out=P[11], ldqo=512), ARG), (dict(q_out=P[11], o_dtype=3), ARG),
    (dict(q_out=P[12]), ARG), (dict(q_out=P[14] - 64), ARG), (dict(q_out=P[16] - 64), ARG), (dict(q_out=P[1] + 128), ARG), (dict(k=P[2] + 128), ARG),
    (dict(q_out=P[8]), ARG), (dict(freq=P[16] + 2), ARG), (dict(q_weight=P[14] + 1), ARG), (dict(k=P[10] - 64), ARG),
    (dict(window=dict(pos=P[1] + 64)), ARG), (dict(window=dict(err=P[7] + 4)), ARG)])
def test_append_refused(change, want):
    assert over_cache("moe_window_append", **change) == want


@pytest.mark.parametrize("change,want", [
    (dict(dtype=3), ARG), (dict(dtype=1), ARG), (dict(scale=NAN), ARG), (dict(scale=INF), ARG), (dict(out=None), ARG), (dict(q=None), ARG),
    (dict(out=P[12] + 1), ARG), (dict(lse=P[13] + 2), ARG), (dict(ldo=255), ARG), (dict(ws=None), WS), (dict(ws=P[14] + 8), WS), (dict(ws_bytes=15), WS),
    (dict(out=P[11] + 64), ARG), (dict(lse=P[12] + 64), ARG), (dict(out=P[1] + 64), ARG), (dict(ws=P[12]), ARG), (dict(lse=P[9]), ARG),
    (dict(window=dict(max_window=65)), SHAPE), (dict(window=dict(err=P[12])), ARG), (dict(ws_bytes=0), WS)])
def test_attention_refused(change, want):
    assert over_cache("moe_window_attention", **change) == want


@pytest.mark.parametrize("change,want", [
    (dict(dtype=4), ARG), (dict(rows=-1), ARG), (dict(given=-1), ARG), (dict(given=65), ARG), (dict(k=33), ARG), (dict(k=-1), ARG), (dict(scale=0.0), ARG),
    (dict(scale=-1.0), ARG), (dict(scale=NAN), ARG), (dict(scale=INF), ARG), (dict(rows=1 << 22), SHAPE), (dict(n=0), SHAPE), (dict(n=(1 << 22) + 1, ld=1 << 23), SHAPE),
    (dict(n=7), ARG), (dict(logits=None), ARG), (dict(ld=999), ARG), (dict(ld=1 << 50), ARG), (dict(tokens=None), ARG), (dict(logp=None), ARG),
    (dict(given=0), ARG), (dict(ids=None), ARG), (dict(top=None), ARG), (dict(k=0), ARG), (dict(logits=P[1] + 1), ARG), (dict(tokens=P[2] + 2), ARG),
    (dict(entropy=P[4] + 1), ARG), (dict(ws=None), WS), (dict(ws=P[7] + 8), WS), (dict(ws_bytes=100), WS), (dict(logp=P[1] + 64), ARG), (dict(top=P[5] + 16), ARG),
    (dict(ws=P[6] - 64), ARG), (dict(tokens=None, given=0, logp=None, entropy=None, k=0, ids=None, top=None), ARG),
    (dict(rows=0, logits=None, tokens=None, logp=None, ids=None, top=None, ws=None), OK)])
def test_logprobs_refused(change, want):
    assert set(change) <= set(SCORES)
    assert B.lib().moe_token_logprobs(None, *dict(SCORES, **change).values()) == want


@no_gpu
def test_sound_calls_reach_the_launch():
    """Without a GPU a call that passes its checks ends in the launch's own error."""
    for name in BASE:
        for cache in ({}, I8, dict(page_stride=8192, v=P[1] + 8192), dict(page_stride=64 * 64, slot_stride=128, head_stride=64)):
            assert over_cache(name, cache=cache) == HIP, (name, cache)
    assert over_cache("moe_window_append", q=None, q_out=None) == HIP
    assert over_cache("moe_window_append", q_out=P[11]) == HIP
    assert over_cache("moe_window_attention", q=P[1] + 256) == HIP
    assert B.lib().moe_token_logprobs(None, *SCORES.values()) == HIP


def test_workspace_sizes():
    c, w = B.MoeKvCache(*CACHE.values()), dict(WINDOW)
    size = lambda **k: B.lib().moe_window_attention_bytes(ctypes.byref(c), ctypes.byref(B.MoeWindow(*dict(w, **k).values())), 4)
    assert size() == 16 and size(max_window=65) == 0 and size(n_seqs=-1) == 0
    assert size(max_pages=1000, ld_pages=1000) == 6 * 4 * 64 * (64 + 2) * 4
    assert B.lib().moe_token_logprobs_bytes(5, 1000, 8) > 0 and B.lib().moe_token_logprobs_bytes(5, 1000, 33) == 0


def test_binding_refuses_tensors_of_the_cpu():
    k = torch.zeros(2, 1, 16, 16, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: B.KVCache(k, k.clone()), lambda: B.Window(i, i[:1], i[:1, None], 1), lambda: B.moe_token_logprobs(torch.zeros(2, 4), k=1)):
        with pytest.raises(ValueError, match="not on a GPU"):
            call()


def test_binding_structs_follow_header():
    import re
    src = open(os.path.join(os.path.dirname(B.HERE), "include", "moe_route.h")).read()
    for cname, py in (("moe_kv_cache", B.MoeKvCache), ("moe_window", B.MoeWindow)):
        body = re.sub(r"/\*.*?\*/", "", re.search(r"typedef struct %s \{(.*?)\} %s;" % (cname, cname), src, re.S).group(1), flags=re.S)
        names = [n.split()[-1].lstrip("*") for decl in body.split(";") if decl.strip() for n in decl.split(",")]
        assert [f[0] for f in py._fields_] == names
