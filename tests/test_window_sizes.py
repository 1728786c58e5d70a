"""Operands over each other in a cache, and the sizes at which the calls on windows begin to refuse, and the workspaces that they name up to there. On the host alone, with
pointers that are fakes: a call that passes its checks ends in the launch's own error where there is no GPU."""
import ctypes
import os

import pytest
import torch

from moe_routed_expert_route_amd import binding as B
from tests.test_window_refusals import ARG, CACHE, HIP, I8, OK, P, SCORES, SHAPE, WINDOW, no_gpu, over_cache

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="library not built")


def attention(n_tokens, n_heads, max_pages, **window):
    """The workspace that is named for these sizes, and what the call says."""
    w = dict(n_tokens=n_tokens, max_pages=max_pages, ld_pages=max_pages, **window)
    size = B.lib().moe_window_attention_bytes(ctypes.byref(B.MoeKvCache(*CACHE.values())), ctypes.byref(B.MoeWindow(*dict(WINDOW, **w).values())), n_heads)
    return size, lambda: over_cache("moe_window_attention", window=w, n_heads=n_heads, ldq=64 * n_heads, ldo=64 * n_heads, ws_bytes=size)


def test_rows_that_a_join_has():
    """Four rows a workgroup of 256 threads, fewer than 2^32 threads in a launch; without several runs there is no join."""
    size, call = attention(65536, 1024, 20)
    assert size == 0 and call() == SHAPE
    size, call = attention(1 << 22, 1024, 5)
    assert size == 0 and call() == SHAPE      # more rows than any call takes
    for n_tokens, max_pages, want in ((65535, 20, 65535 * 1024 * 2 * 66 * 4), (65536, 16, 16), (1 << 18, 8, 16)):
        assert attention(n_tokens, 1024, max_pages)[0] == want
    assert attention(4096 * 64, 64, 64, n_seqs=4096, max_window=64)[0] > 0


@no_gpu
def test_rows_that_a_join_has_reach_the_launch():
    for args in ((65535, 1024, 20), (65536, 1024, 16), (1 << 18, 64, 20)):
        assert attention(*args)[1]() == HIP, args
    assert attention(4096 * 64, 64, 64, n_seqs=4096, max_window=64)[1]() == HIP


def test_calls_without_tokens_name_a_workspace_that_they_accept():
    for window in (dict(n_seqs=0), dict(n_seqs=0, max_pages=-5), dict(n_tokens=0, max_pages=0), dict(n_seqs=0, max_pages=1 << 20, ld_pages=1 << 20)):
        w = B.MoeWindow(*dict(WINDOW, **window).values())
        assert B.lib().moe_window_attention_bytes(ctypes.byref(B.MoeKvCache(*CACHE.values())), ctypes.byref(w), 4) == 16, window
        assert over_cache("moe_window_attention", window=window, ws_bytes=16) == OK


@pytest.mark.parametrize("rows,n,refused", [(4194303, 32768, False), (4194303, 32769, True), (4194304, 10, True), (65535, 1 << 22, False),
                                            (65536, 1 << 22, True), (3, (1 << 22) + 1, True)])
def test_pieces_of_log_probabilities(rows, n, refused):
    assert (B.lib().moe_token_logprobs_bytes(rows, n, 8) == 0) == refused
    args = dict(SCORES, rows=rows, n=n, ld=n, ws_bytes=1 << 40)
    if refused:
        assert B.lib().moe_token_logprobs(None, *args.values()) == SHAPE


@no_gpu
def test_pieces_of_log_probabilities_reach_the_launch():
    assert B.lib().moe_token_logprobs(None, *dict(SCORES, rows=4194303, n=32768, ld=32768, ws_bytes=1 << 40).values()) == HIP


# the rows of k and of v: 10 pages x 4096 bytes; a scale array: 640 x 4 bytes
@pytest.mark.parametrize("name", ["moe_window_append", "moe_window_attention"])
@pytest.mark.parametrize("change", [dict(k_scale=P[1]), dict(k_scale=P[2] + 40956), dict(v_scale=P[1] + 4096), dict(v_scale=P[2] - 2556),
                                    dict(k_scale=P[1] + 8 + 4096, v=P[1] + 4096, page_stride=8192)])
def test_scales_over_the_rows_of_a_cache(name, change):
    assert over_cache(name, cache=dict(I8, **change)) == ARG


@no_gpu
@pytest.mark.parametrize("change", [dict(k_scale=P[1] + 40960), dict(v_scale=P[1] - 2560), dict(k_scale=P[2] - 2560, v_scale=P[2] + 40960)])
def test_scales_beside_the_rows_of_a_cache(change):
    for name in ("moe_window_append", "moe_window_attention"):
        assert over_cache(name, cache=dict(I8, **change)) == HIP


@pytest.mark.parametrize("scale,ok", [(2.0 ** 127, True), (2.0 ** 127 * (1 + 2.0 ** -23), False), (2.4e38, False), (3.4e38, False), (1e-45, True)])
def test_largest_scales(scale, ok):
    """Above 2^127 the unit of the exponentials, scale times log2(e), need not be a float32."""
    calls = [lambda: over_cache("moe_window_attention", scale=scale), lambda: over_cache("moe_window_attention", scale=-scale),
             lambda: B.lib().moe_token_logprobs(None, *dict(SCORES, scale=scale).values())]
    if not ok:
        assert [c() for c in calls] == [ARG] * 3
    elif not torch.cuda.is_available():
        assert [c() for c in calls] == [HIP] * 3
